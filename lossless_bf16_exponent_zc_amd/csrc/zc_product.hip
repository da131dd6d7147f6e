// zc_product.hip -- the experts' products of 8-bit blocks.
//
//   out[r, j] = sum over b of sA[r,b] sW[j,b] <A[r,b], W[j,b]>
//
// on v_mfma_scale_f32_16x16x128_f8f6f4: one instruction takes 16 rows of each
// side over a whole block of 128 and applies both blocks' scale exponents, so
// the scales cost no arithmetic and the sum over blocks stays in the unit's
// 32-bit accumulators.  The weight side is the instruction's first operand:
// a lane then has four neighbouring columns j of one row r.
#include "zc_experts_kernels.h"

namespace zc {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x8 two(xu32x4 lo, xu32x4 hi) {
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// One tile of a product, whichever product it is.
struct Tile {
    const uint8_t* a;        // first row of the token side, at its first block
    const uint8_t* as;       // its scales
    const uint8_t* w;        // first row of the weight side
    const uint8_t* ws;       // scales of the weight side's row 0
    uint32_t a_rows, w_rows; // rows that exist from there on
    uint32_t w0;             // index of the weight side's first row (for its scales)
    uint32_t blocks;
    uint64_t a_stride, w_stride;
    uint32_t as_stride, ws_stride;
    uint32_t w_shift;        // rows per scale row of the weight side, as a shift: 7 or 0
};

// Expert and first row of the `index`-th tile of `m` rows, over all experts'
// segments in order.  Every wave finds it for itself: a lane has one expert.
struct Found {
    uint32_t expert, row, count, end;  // count: rows of the segment from `row`; end: where padding ends
    bool any;
};

__device__ __forceinline__ uint32_t clamp_to(int32_t v, uint32_t lo, uint32_t hi) {
    return v < (int32_t)lo ? lo : (uint32_t)v > hi ? hi : (uint32_t)v;
}

__device__ __forceinline__ Found find_tile(const ProductArgs& p, uint32_t index, uint32_t m) {
    if (!p.offsets) {
        const uint64_t r = (uint64_t)index * m;
        const bool any = r < p.rows;
        return Found{0, (uint32_t)r, any ? p.rows - (uint32_t)r : 0, p.rows, any};
    }
    const uint32_t lane = __lane_id();
    uint32_t before = 0;
    for (uint32_t e0 = 0; e0 < p.experts; e0 += 64) {
        const uint32_t e = e0 + lane;
        uint32_t lo = 0, count = 0, end = 0;
        if (e < p.experts) {
            lo = clamp_to(p.offsets[e], 0, p.rows);
            end = clamp_to(p.offsets[e + 1], lo, p.rows);
            count = p.counts ? clamp_to(p.counts[e], 0, end - lo) : end - lo;
        }
        uint32_t tiles = (count + m - 1) / m;
        if (end > lo && tiles == 0) tiles = 1;  // a segment of padding only
        uint32_t sum = tiles;
        for (uint32_t d = 1; d < 64; d <<= 1) {
            const uint32_t t = __shfl_up(sum, d);
            if (lane >= d) sum += t;
        }
        const uint64_t past = __ballot(before + sum > index);
        if (past) {
            const uint32_t at = __ffsll((unsigned long long)past) - 1;
            const uint32_t in = uniform(index - before - (uint32_t)__shfl((int)(sum - tiles), at));
            Found f;
            f.expert = uniform(e0 + at);
            const uint32_t l = uniform(__shfl((int)lo, at)), c = uniform(__shfl((int)count, at));
            f.end = uniform(__shfl((int)end, at));
            f.row = l + in * m;
            f.count = c > in * m ? c - in * m : 0;
            f.any = true;
            return f;
        }
        before += uniform(__shfl((int)sum, 63));
    }
    return Found{0, 0, 0, 0, false};
}

template <typename T>
__device__ __forceinline__ void store4(T* out, const f32x4& v, uint32_t n) {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (i < n) out[i] = (T)v[i];
}

__device__ __forceinline__ void store_out(void* out, uint32_t dtype, uint64_t at, const f32x4& v, uint32_t n) {
    if (dtype == ZC_BF16) store4(static_cast<__bf16*>(out) + at, v, n);
    else if (dtype == ZC_FP16) store4(static_cast<_Float16*>(out) + at, v, n);
    else store4(static_cast<float*>(out) + at, v, n);
}

// 16 weight rows by 64 token rows of a tile, from memory to the unit.
__device__ __forceinline__ void wave_tile(const Tile& t, uint32_t w_first, f32x4* acc) {
    const uint32_t lane = __lane_id(), r = lane & 15, g = lane >> 4;
    const uint32_t wr = w_first + r < t.w_rows ? w_first + r : t.w_rows - 1;
    const uint8_t* w = t.w + wr * t.w_stride + g * 32;
    const uint8_t* ws = t.ws + (uint64_t)((t.w0 + wr) >> t.w_shift) * t.ws_stride;
    const uint8_t* a[4];
    const uint8_t* as[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t ar = i * 16 + r < t.a_rows ? i * 16 + r : t.a_rows - 1;
        a[i] = t.a + ar * t.a_stride + g * 32;
        as[i] = t.as + (uint64_t)ar * t.as_stride;
        acc[i] = f32x4{0, 0, 0, 0};
    }
    for (uint32_t b = 0; b < t.blocks; ++b) {
        const xu32x4* wp = reinterpret_cast<const xu32x4*>(w + (uint64_t)b * 128);
        const i32x8 wv = two(wp[0], wp[1]);
        const int sw = ws[b];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const xu32x4* ap = reinterpret_cast<const xu32x4*>(a[i] + (uint64_t)b * 128);
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, two(ap[0], ap[1]), acc[i], 0, 0, 0, sw, 0,
                                                                     (int)as[i][b]);
        }
    }
}

__global__ __launch_bounds__(256) void product(ProductArgs p) {
    const uint32_t lane = __lane_id(), r = lane & 15, g = lane >> 4, wave = uniform(threadIdx.x >> 6);
    const Found f = find_tile(p, blockIdx.y, 64);
    if (!f.any) return;
    const uint32_t n0 = blockIdx.x * 64 + wave * 16;
    if (n0 >= p.n) return;
    f32x4 acc[4] = {};
    if (f.count) {
        const uint32_t wrows = (p.n + 127) / 128;
        const Tile t{p.a + (uint64_t)f.row * p.k, p.a_scale + (uint64_t)f.row * p.a_scale_stride,
                     p.w + (uint64_t)f.expert * p.n * p.k, p.w_scale + (uint64_t)f.expert * wrows * p.w_scale_stride,
                     f.count, p.n, 0, p.k / 128, p.k, p.k, p.a_scale_stride, p.w_scale_stride, 7};
        wave_tile(t, n0, acc);
    }
    const uint32_t j = n0 + g * 4;
    if (j >= p.n) return;
    const uint32_t left = p.n - j;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (i * 16 + r < f.count) store_out(p.out, p.out_dtype, (uint64_t)(f.row + i * 16 + r) * p.out_stride + j, acc[i], left);
    if (f.count <= 64)
        for (uint32_t q = f.row + f.count + r; q < f.end; q += 16)
            store_out(p.out, p.out_dtype, (uint64_t)q * p.out_stride + j, f32x4{0, 0, 0, 0}, left);
}

__global__ __launch_bounds__(256) void weight_grad(WeightGradArgs p) {
    const uint32_t lane = __lane_id(), r = lane & 15, g = lane >> 4, wave = uniform(threadIdx.x >> 6);
    const uint32_t e = blockIdx.z, i0 = blockIdx.y * 64, j0 = blockIdx.x * 64 + wave * 16;
    if (j0 >= p.k) return;
    uint32_t b0 = 0, b1 = p.rows / 128;
    if (p.offsets) {
        b0 = clamp_to(p.offsets[e], 0, p.rows) / 128;
        b1 = (clamp_to(p.offsets[e + 1], b0 * 128, p.rows) + 127) / 128;
    }
    const Tile t{p.y + (uint64_t)i0 * p.rows + b0 * 128, p.y_scale + (uint64_t)i0 * p.scale_stride + b0,
                 p.x + b0 * 128, p.x_scale + b0, p.n - i0, p.k, 0, b1 - b0, p.rows, p.rows, p.scale_stride,
                 p.scale_stride, 0};
    f32x4 acc[4];
    wave_tile(t, j0, acc);
    const uint32_t j = j0 + g * 4;
    if (j >= p.k) return;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (i0 + i * 16 + r < p.n)
            store_out(p.dw, p.out_dtype, ((uint64_t)e * p.n + i0 + i * 16 + r) * p.k + j, acc[i], p.k - j);
}

}  // namespace

void launch_product(const ProductArgs& a, hipStream_t stream) {
    const uint32_t tiles = a.rows / 64 + (a.offsets ? a.experts : 1);
    hipLaunchKernelGGL(product, dim3((a.n + 63) / 64, tiles), dim3(256), 0, stream, a);
}

void launch_weight_grad(const WeightGradArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(weight_grad, dim3((a.k + 63) / 64, (a.n + 63) / 64, a.experts), dim3(256), 0, stream, a);
}

}  // namespace zc
