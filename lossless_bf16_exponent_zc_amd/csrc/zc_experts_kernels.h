// zc_experts_kernels.h -- argument blocks and launchers of the expert
// operators (include/zc_experts.h), and the small device helpers they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zc_experts.h"

namespace zc {

constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxTopk = 64;
constexpr uint32_t kFp8Block = 128;  // values per scale, along the contracted dimension

// ------------------------------------------------------------ launchers
struct RouteArgs {
    const int32_t* ids;
    uint32_t nslots;
    uint32_t experts;
    uint32_t align;
    uint32_t capacity;  // rows d_slot holds
    int32_t* offsets;
    int32_t* counts;
    int32_t* row;
    int32_t* slot;
    uint32_t* ws;       // per expert, per tile: slots of the expert in the tile
    uint32_t tiles;
};

struct RowArgs {  // dispatch, combine and the gradient of combine
    const void* x;         // dispatch: tokens; combine: rows; gradient: dy
    const void* rows;      // gradient: rows (or null)
    void* out;             // dispatch: rows; combine: tokens; gradient: drows (or null)
    const float* weights;  // or null
    float* dweights;       // or null
    const int32_t* offsets;
    const int32_t* counts; // or null: no padding rows
    const int32_t* row;
    uint64_t x_stride, rows_stride, out_stride;  // in bytes
    uint32_t tokens, topk, experts;
    uint32_t width;        // elements per row
    uint32_t capacity;
};

struct CastRowsArgs {
    const void* x;
    uint64_t x_stride;     // elements
    uint8_t* data;
    uint8_t* scale;
    const int32_t* row;    // null: row t goes to row t
    const int32_t* offsets;
    const int32_t* counts;
    const int32_t* used;   // null, or rows in use
    uint32_t tokens, topk, experts, width;
    uint32_t data_stride, scale_stride;
    uint32_t capacity;
};

struct CastTileArgs {
    const void* x;
    uint64_t x_stride;     // elements (columns form)
    uint8_t* data;
    uint8_t* scale;
    const int32_t* used;
    uint32_t rows, cols;   // weights: n, k of the result; columns: rows, cols of x
    uint32_t experts;
    uint32_t data_stride, scale_stride;  // columns: scale_stride alone
    uint32_t transpose;
};

struct ProductArgs {
    const uint8_t* a;        // tokens: [rows, k] bytes
    const uint8_t* a_scale;
    const uint8_t* w;
    const uint8_t* w_scale;
    const int32_t* offsets;  // null: one expert
    const int32_t* counts;   // null: whole segments
    void* out;
    uint64_t out_stride;     // elements
    uint32_t rows, experts, n, k;  // k: stored, a multiple of 128
    uint32_t a_scale_stride, w_scale_stride;
    uint32_t out_dtype;
};

struct WeightGradArgs {
    const uint8_t* y;        // [rows / 128][n][128] bytes
    const uint8_t* y_scale;  // [rows / 128][y_scale_stride]
    const uint8_t* x;        // [rows / 128][k][128]
    const uint8_t* x_scale;
    const int32_t* offsets;
    void* dw;
    uint32_t rows;           // stored, a multiple of 128
    uint32_t experts, n, k;
    uint32_t y_scale_stride, x_scale_stride;
    uint32_t out_dtype;
};

// How a weight gradient is cut: tiles of side x side, each segment summed in up
// to `parts` parts that are joined afterwards (parts > 1 needs a workspace of
// parts * experts * n * k floats).  split: whether parts are allowed.
struct WeightGradPlan {
    uint32_t side, parts;
};
WeightGradPlan plan_weight_grad(uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, bool split);

// Each enqueues its kernels, or returns ZC_ERR_UNSUPPORTED and enqueues none
// where the launch would have more workgroups than a launch may (2^32 threads).
uint64_t route_tiles(uint64_t nslots);
zc_status launch_route(const RouteArgs& a, hipStream_t stream);
zc_status launch_dispatch(const RowArgs& a, uint32_t dtype, hipStream_t stream);
zc_status launch_combine(const RowArgs& a, uint32_t dtype, hipStream_t stream);
zc_status launch_combine_backward(const RowArgs& a, uint32_t dtype, hipStream_t stream);
zc_status launch_cast_rows(const CastRowsArgs& a, uint32_t dtype, hipStream_t stream);
zc_status launch_cast_weights(const CastTileArgs& a, uint32_t dtype, hipStream_t stream);
zc_status launch_cast_columns(const CastTileArgs& a, uint32_t dtype, hipStream_t stream);
zc_status launch_product(const ProductArgs& a, hipStream_t stream);
zc_status launch_weight_grad(const WeightGradArgs& a, const WeightGradPlan& plan, void* ws, hipStream_t stream);

// Whether a launch may have this many workgroups of 256 threads.
inline bool fits(uint64_t workgroups) { return workgroups < (1ull << 24); }

// -------------------------------------------------------- device helpers
typedef uint32_t xu32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t xu32x2 __attribute__((ext_vector_type(2)));

__host__ __device__ constexpr uint32_t up_to(uint32_t n, uint32_t m) { return (n + m - 1) / m * m; }

__device__ __forceinline__ float to_float(__bf16 v) { return (float)v; }
__device__ __forceinline__ float to_float(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_float(float v) { return v; }

// A value that the compiler may keep in a scalar register: every lane of the
// wave has it.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// 16 bytes of values at any element's address, zeros past the first n (n <= 0:
// all): a short word comes in parts of 8, 4 and 2 bytes.
template <typename T>
__device__ __forceinline__ xu32x4 load_word(const T* p, int32_t n) {
    typedef xu32x4 __attribute__((aligned(2))) Four;
    typedef xu32x2 __attribute__((aligned(2))) Two;
    typedef uint32_t __attribute__((aligned(2))) One;
    if (n >= 16 / (int32_t)sizeof(T)) return *reinterpret_cast<const Four*>(p);
    if (n <= 0) return xu32x4{};
    const uint32_t bytes = (uint32_t)n * sizeof(T);
    xu32x2 two = {0, 0};
    uint32_t one = 0, half = 0;
    if (bytes & 8) two = *reinterpret_cast<const Two*>(p);
    if (bytes & 4) one = *reinterpret_cast<const One*>(p + (bytes & 8) / sizeof(T));
    if (sizeof(T) == 2 && bytes & 2) half = *reinterpret_cast<const uint16_t*>(p + (bytes & 12) / sizeof(T));
    const uint32_t next = bytes & 4 ? one : half, past = bytes & 4 ? half : 0;
    return bytes & 8 ? xu32x4{two[0], two[1], next, past} : xu32x4{next, past, 0, 0};
}

// The byte of the least scale s = 2^(b-127) with top <= 448 s, top given as
// the bits of a finite float >= 0: 448 = 1.75 * 2^8, so the exponent of top
// less 8, one more where its mantissa passes 1.75; at least 2^-126 (so that
// 1/s and s are normal floats), 1 for top = 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int b = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return top == 0 ? 127u : (uint32_t)(b < 1 ? 1 : b);
}
// 1/s; b is at most 254 - 7, so the result is a normal float.
__device__ __forceinline__ float inverse_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// |x| as ordered bits, 0 for what is not finite.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u < 0x7F800000u ? u : 0u;
}

// x / s as it is to be rounded; infinity where x is not finite, which the
// conversion turns into the one NaN 0x7F.
__device__ __forceinline__ float scaled(float x, float inv) {
    return (__float_as_uint(x) & 0x7FFFFFFFu) < 0x7F800000u ? x * inv : __uint_as_float(0x7F800000u);
}

// Four E4M3 bytes, rounded to nearest even.  |x| <= 448 or infinity.
__device__ __forceinline__ uint32_t four_fp8(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

}  // namespace zc
