// zc_experts_api.hip -- the C ABI of include/zc_experts.h: argument checks and
// launches.  Every call enqueues on the caller's stream and returns.
#include "zc_experts_kernels.h"

using namespace zc;

namespace {

constexpr uint64_t kMaxRows = 0x7FFFFFFFull;
constexpr uint32_t kMaxWidth = 1u << 24;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
uint64_t up64(uint64_t n, uint64_t m) { return (n + m - 1) / m * m; }
uint32_t stored(uint32_t cols) { return up_to(cols, kFp8Block); }
uint32_t scales(uint32_t cols) { return up_to((cols + kFp8Block - 1) / kFp8Block, 4); }
uint32_t elem_bytes(uint32_t dtype) { return dtype == ZC_FP32 ? 4 : 2; }

bool route_limits(uint64_t tokens, uint32_t topk, uint32_t experts, uint32_t align) {
    if (!topk || topk > kMaxTopk || !experts || experts > kMaxExperts) return false;
    if (!align || align > 1024 || (align & (align - 1))) return false;
    return tokens <= kMaxRows && tokens * topk <= kMaxRows;
}

uint64_t route_rows(uint64_t tokens, uint32_t topk, uint32_t experts, uint32_t align) {
    const uint64_t slots = tokens * topk, used = slots < experts ? slots : experts;
    return up64(slots + used * (align - 1), align);
}

zc_status finished(zc_status launched) {
    return launched != ZC_OK ? launched : hipGetLastError() == hipSuccess ? ZC_OK : ZC_ERR_HIP;
}

// Shapes that every row call shares; ZC_OK, or why not.
zc_status check_rows(uint32_t dtype, uint64_t tokens, uint32_t topk, uint32_t hidden, uint64_t row_capacity) {
    if (dtype > ZC_FP32 || !hidden) return ZC_ERR_INVALID_ARG;
    if (!topk || topk > kMaxTopk || hidden >= kMaxWidth || tokens > kMaxRows || tokens * topk > kMaxRows ||
        row_capacity > kMaxRows)
        return ZC_ERR_UNSUPPORTED;
    return ZC_OK;
}

bool bad_matrix(const void* p, uint64_t stride, uint32_t width, uint32_t dtype) {
    return !p || !aligned(p, elem_bytes(dtype)) || stride < width || stride > (1ull << 40);
}

bool bad_words(const void* p) { return !p || !aligned(p, 4); }

// offsets are read for the padding rows alone, which counts stand for
bool bad_segments(const int32_t* offsets, const int32_t* counts) {
    return counts && (!aligned(counts, 4) || bad_words(offsets));
}

}  // namespace

extern "C" {

uint64_t zc_route_rows(uint64_t tokens, uint32_t topk, uint32_t experts, uint32_t align) {
    if (!route_limits(tokens, topk, experts, align)) return 0;
    const uint64_t r = route_rows(tokens, topk, experts, align);
    return r <= kMaxRows ? r : 0;
}

uint64_t zc_route_workspace_bytes(uint64_t tokens, uint32_t topk, uint32_t experts) {
    if (!route_limits(tokens, topk, experts, 1)) return 0;
    return up64((route_tiles(tokens * topk) + 1) * experts * 4, 256);
}

zc_status zc_route(const int32_t* d_ids, uint64_t tokens, uint32_t topk, uint32_t experts, uint32_t align,
                   int32_t* d_offsets, int32_t* d_counts, int32_t* d_row, int32_t* d_slot, uint64_t row_capacity,
                   void* d_ws, uint64_t ws_bytes, hipStream_t stream) {
    if (!route_limits(tokens, topk, experts, align)) return ZC_ERR_UNSUPPORTED;
    const uint64_t need = route_rows(tokens, topk, experts, align);
    if (need > kMaxRows || row_capacity > kMaxRows) return ZC_ERR_UNSUPPORTED;
    if (bad_words(d_offsets) || bad_words(d_counts) || !d_ws || !aligned(d_ws, 256)) return ZC_ERR_INVALID_ARG;
    if (tokens && (bad_words(d_ids) || bad_words(d_row))) return ZC_ERR_INVALID_ARG;
    if (row_capacity && bad_words(d_slot)) return ZC_ERR_INVALID_ARG;
    if (row_capacity < need || ws_bytes < zc_route_workspace_bytes(tokens, topk, experts)) return ZC_ERR_CAPACITY;
    const uint32_t n = (uint32_t)(tokens * topk);
    const RouteArgs a{d_ids, n, experts, align, (uint32_t)row_capacity, d_offsets, d_counts, d_row, d_slot,
                      static_cast<uint32_t*>(d_ws), (uint32_t)route_tiles(n)};
    return finished(launch_route(a, stream));
}

zc_status zc_dispatch(const void* d_x, uint64_t x_stride, uint32_t dtype, uint64_t tokens, uint32_t topk,
                      uint32_t experts, uint32_t hidden, const int32_t* d_offsets, const int32_t* d_counts,
                      const int32_t* d_row, void* d_rows, uint64_t rows_stride, uint64_t row_capacity,
                      hipStream_t stream) {
    if (zc_status e = check_rows(dtype, tokens, topk, hidden, row_capacity)) return e;
    if (!experts || experts > kMaxExperts) return ZC_ERR_UNSUPPORTED;
    if (!tokens || !row_capacity) return ZC_OK;
    if (bad_matrix(d_x, x_stride, hidden, dtype) || bad_matrix(d_rows, rows_stride, hidden, dtype) ||
        bad_words(d_row) || bad_segments(d_offsets, d_counts))
        return ZC_ERR_INVALID_ARG;
    const uint32_t eb = elem_bytes(dtype);
    RowArgs a{};
    a.x = d_x;
    a.out = d_rows;
    a.offsets = d_offsets;
    a.counts = d_counts;
    a.row = d_row;
    a.x_stride = x_stride * eb;
    a.out_stride = rows_stride * eb;
    a.tokens = (uint32_t)tokens;
    a.topk = topk;
    a.experts = experts;
    a.width = hidden;
    a.capacity = (uint32_t)row_capacity;
    return finished(launch_dispatch(a, dtype, stream));
}

zc_status zc_dispatch_fp8(const void* d_x, uint64_t x_stride, uint32_t dtype, uint64_t tokens, uint32_t topk,
                          uint32_t experts, uint32_t hidden, const int32_t* d_offsets, const int32_t* d_counts,
                          const int32_t* d_row, void* d_data, void* d_scale, uint64_t row_capacity,
                          hipStream_t stream) {
    if (zc_status e = check_rows(dtype, tokens, topk, hidden, row_capacity)) return e;
    if (!experts || experts > kMaxExperts) return ZC_ERR_UNSUPPORTED;
    if (!tokens || !row_capacity) return ZC_OK;
    if (bad_matrix(d_x, x_stride, hidden, dtype) || !d_data || !aligned(d_data, 16) || !d_scale ||
        !aligned(d_scale, 16) || bad_words(d_row) || bad_segments(d_offsets, d_counts))
        return ZC_ERR_INVALID_ARG;
    const CastRowsArgs a{d_x, x_stride, static_cast<uint8_t*>(d_data), static_cast<uint8_t*>(d_scale), d_row,
                         d_offsets, d_counts, nullptr, (uint32_t)tokens, topk, experts, hidden, stored(hidden),
                         scales(hidden), (uint32_t)row_capacity};
    return finished(launch_cast_rows(a, dtype, stream));
}

zc_status zc_combine(const void* d_rows, uint64_t rows_stride, const float* d_weights, uint32_t dtype,
                     uint64_t tokens, uint32_t topk, uint32_t hidden, const int32_t* d_row, uint64_t row_capacity,
                     void* d_y, uint64_t y_stride, hipStream_t stream) {
    if (zc_status e = check_rows(dtype, tokens, topk, hidden, row_capacity)) return e;
    if (!tokens) return ZC_OK;
    if (bad_matrix(d_y, y_stride, hidden, dtype) || bad_words(d_row) ||
        (row_capacity && bad_matrix(d_rows, rows_stride, hidden, dtype)) || (d_weights && !aligned(d_weights, 4)))
        return ZC_ERR_INVALID_ARG;
    const uint32_t eb = elem_bytes(dtype);
    RowArgs a{};
    a.x = d_rows;
    a.out = d_y;
    a.weights = d_weights;
    a.row = d_row;
    a.x_stride = rows_stride * eb;
    a.out_stride = y_stride * eb;
    a.tokens = (uint32_t)tokens;
    a.topk = topk;
    a.width = hidden;
    a.capacity = (uint32_t)row_capacity;
    return finished(launch_combine(a, dtype, stream));
}

zc_status zc_combine_backward(const void* d_dy, uint64_t dy_stride, const void* d_rows, uint64_t rows_stride,
                              const float* d_weights, uint32_t dtype, uint64_t tokens, uint32_t topk,
                              uint32_t experts, uint32_t hidden, const int32_t* d_offsets, const int32_t* d_counts,
                              const int32_t* d_row, uint64_t row_capacity, void* d_drows, uint64_t drows_stride,
                              float* d_dweights, hipStream_t stream) {
    if (zc_status e = check_rows(dtype, tokens, topk, hidden, row_capacity)) return e;
    if (!experts || experts > kMaxExperts) return ZC_ERR_UNSUPPORTED;
    if (!d_drows && !d_dweights) return ZC_ERR_INVALID_ARG;
    if (!tokens) return ZC_OK;
    if (bad_matrix(d_dy, dy_stride, hidden, dtype) || bad_words(d_row) || (d_weights && !aligned(d_weights, 4)))
        return ZC_ERR_INVALID_ARG;
    if (d_drows && (bad_matrix(d_drows, drows_stride, hidden, dtype) || bad_segments(d_offsets, d_counts)))
        return ZC_ERR_INVALID_ARG;
    if (d_dweights &&
        (!aligned(d_dweights, 4) || (row_capacity && bad_matrix(d_rows, rows_stride, hidden, dtype))))
        return ZC_ERR_INVALID_ARG;
    const uint32_t eb = elem_bytes(dtype);
    RowArgs a{};
    a.x = d_dy;
    a.rows = d_rows;
    a.out = d_drows;
    a.weights = d_weights;
    a.dweights = d_dweights;
    a.offsets = d_offsets;
    a.counts = d_counts;
    a.row = d_row;
    a.x_stride = dy_stride * eb;
    a.rows_stride = rows_stride * eb;
    a.out_stride = drows_stride * eb;
    a.tokens = (uint32_t)tokens;
    a.topk = topk;
    a.experts = experts;
    a.width = hidden;
    a.capacity = (uint32_t)row_capacity;
    return finished(launch_combine_backward(a, dtype, stream));
}

zc_status zc_quantize_rows(const void* d_x, uint64_t x_stride, uint32_t dtype, uint64_t rows, uint32_t cols,
                           const int32_t* d_used, void* d_data, void* d_scale, hipStream_t stream) {
    if (dtype > ZC_FP32 || !cols) return ZC_ERR_INVALID_ARG;
    if (cols >= kMaxWidth || rows > kMaxRows) return ZC_ERR_UNSUPPORTED;
    if (!rows) return ZC_OK;
    if (bad_matrix(d_x, x_stride, cols, dtype) || !d_data || !aligned(d_data, 16) || !d_scale ||
        !aligned(d_scale, 16) || !aligned(d_used, 4))
        return ZC_ERR_INVALID_ARG;
    const CastRowsArgs a{d_x, x_stride, static_cast<uint8_t*>(d_data), static_cast<uint8_t*>(d_scale), nullptr,
                         nullptr, nullptr, d_used, (uint32_t)rows, 1, 0, cols, stored(cols), scales(cols),
                         (uint32_t)rows};
    return finished(launch_cast_rows(a, dtype, stream));
}

zc_status zc_quantize_weights(const void* d_w, uint32_t dtype, uint32_t experts, uint32_t n, uint32_t k,
                              int transpose, void* d_data, void* d_scale, hipStream_t stream) {
    if (dtype > ZC_FP32 || !n || !k || !experts) return ZC_ERR_INVALID_ARG;
    if (experts > kMaxExperts || n >= kMaxWidth || k >= kMaxWidth) return ZC_ERR_UNSUPPORTED;
    if ((uint64_t)experts * (stored(n) / 128) * (stored(k) / 128) > kMaxRows) return ZC_ERR_UNSUPPORTED;
    if (bad_matrix(d_w, k, k, dtype) || !d_data || !aligned(d_data, 16) || !d_scale || !aligned(d_scale, 16))
        return ZC_ERR_INVALID_ARG;
    const CastTileArgs a{d_w, 0, static_cast<uint8_t*>(d_data), static_cast<uint8_t*>(d_scale), nullptr, n, k,
                         experts, stored(k), scales(k), transpose ? 1u : 0u};
    return finished(launch_cast_weights(a, dtype, stream));
}

zc_status zc_quantize_columns(const void* d_x, uint64_t x_stride, uint32_t dtype, uint64_t rows, uint32_t cols,
                              const int32_t* d_used, void* d_data, void* d_scale, hipStream_t stream) {
    if (dtype > ZC_FP32 || !cols) return ZC_ERR_INVALID_ARG;
    if (cols >= kMaxWidth || rows >= kMaxWidth) return ZC_ERR_UNSUPPORTED;
    if (!rows) return ZC_OK;
    if (bad_matrix(d_x, x_stride, cols, dtype) || !d_data || !aligned(d_data, 16) || !d_scale ||
        !aligned(d_scale, 16) || !aligned(d_used, 4))
        return ZC_ERR_INVALID_ARG;
    const CastTileArgs a{d_x, x_stride, static_cast<uint8_t*>(d_data), static_cast<uint8_t*>(d_scale), d_used,
                         (uint32_t)rows, cols, 1, 128, up_to(cols, 4), 0};
    return finished(launch_cast_columns(a, dtype, stream));
}

zc_status zc_expert_product(const void* d_a, const void* d_a_scale, uint64_t rows, const void* d_w,
                            const void* d_w_scale, uint32_t experts, uint32_t n, uint32_t k,
                            const int32_t* d_offsets, const int32_t* d_counts, void* d_out, uint64_t out_stride,
                            uint32_t out_dtype, hipStream_t stream) {
    if (out_dtype > ZC_FP32 || !experts || !n || !k) return ZC_ERR_INVALID_ARG;
    if (!d_offsets && (experts != 1 || d_counts)) return ZC_ERR_INVALID_ARG;
    if (experts > kMaxExperts || n >= kMaxWidth || k >= kMaxWidth || rows > kMaxRows) return ZC_ERR_UNSUPPORTED;
    if (!rows) return ZC_OK;
    if (!d_a || !aligned(d_a, 16) || !d_a_scale || !aligned(d_a_scale, 16) || !d_w || !aligned(d_w, 16) ||
        !d_w_scale || !aligned(d_w_scale, 16) || bad_matrix(d_out, out_stride, n, out_dtype) ||
        !aligned(d_offsets, 4) || !aligned(d_counts, 4))
        return ZC_ERR_INVALID_ARG;
    const ProductArgs a{static_cast<const uint8_t*>(d_a), static_cast<const uint8_t*>(d_a_scale),
                        static_cast<const uint8_t*>(d_w), static_cast<const uint8_t*>(d_w_scale), d_offsets, d_counts,
                        d_out, out_stride, (uint32_t)rows, experts, n, stored(k), scales(k), scales(k), out_dtype};
    return finished(launch_product(a, stream));
}

uint64_t zc_expert_weight_grad_workspace_bytes(uint64_t rows, uint32_t experts, uint32_t n, uint32_t k) {
    if (!experts || !n || !k || experts > kMaxExperts || n >= kMaxWidth || k >= kMaxWidth || rows >= kMaxWidth) return 0;
    const uint32_t parts = plan_weight_grad(stored((uint32_t)rows), experts, n, k, true).parts;
    return parts == 1 ? 0 : up64((uint64_t)parts * experts * n * k * 4, 256);
}

zc_status zc_expert_weight_grad(const void* d_y, const void* d_y_scale, const void* d_x, const void* d_x_scale,
                                uint64_t rows, uint32_t experts, uint32_t n, uint32_t k, const int32_t* d_offsets,
                                void* d_dw, uint32_t out_dtype, void* d_ws, uint64_t ws_bytes, hipStream_t stream) {
    if (out_dtype > ZC_FP32 || !experts || !n || !k) return ZC_ERR_INVALID_ARG;
    if (!d_offsets && experts != 1) return ZC_ERR_INVALID_ARG;
    if (experts > kMaxExperts || n >= kMaxWidth || k >= kMaxWidth || rows >= kMaxWidth) return ZC_ERR_UNSUPPORTED;
    if (bad_matrix(d_dw, k, k, out_dtype) || !aligned(d_offsets, 4)) return ZC_ERR_INVALID_ARG;
    if (rows && (!d_y || !aligned(d_y, 16) || !d_y_scale || !aligned(d_y_scale, 16) || !d_x || !aligned(d_x, 16) ||
                 !d_x_scale || !aligned(d_x_scale, 16)))
        return ZC_ERR_INVALID_ARG;
    if (d_ws && !aligned(d_ws, 256)) return ZC_ERR_INVALID_ARG;
    if (d_ws && ws_bytes < zc_expert_weight_grad_workspace_bytes(rows, experts, n, k)) return ZC_ERR_CAPACITY;
    const WeightGradArgs a{static_cast<const uint8_t*>(d_y), static_cast<const uint8_t*>(d_y_scale),
                           static_cast<const uint8_t*>(d_x), static_cast<const uint8_t*>(d_x_scale), d_offsets, d_dw,
                           stored((uint32_t)rows), experts, n, k, up_to(n, 4), up_to(k, 4), out_dtype};
    const WeightGradPlan plan = plan_weight_grad(a.rows, experts, n, k, d_ws != nullptr);
    return finished(launch_weight_grad(a, plan, d_ws, stream));
}

}  // extern "C"
