/*
 * zc_experts.h -- rows of a mixture of experts on AMD MI355X (gfx950): C ABI.
 *
 * What happens around the compressed all-to-all of zc.h: tokens are sorted by
 * expert (zc_route, zc_dispatch), optionally as 8-bit blocks, the experts'
 * matrix products run on the sorted rows (zc_expert_product), rows go back to
 * their tokens with the router's weights applied (zc_combine), and the
 * gradients of all of these (zc_combine with no weights is the gradient of
 * zc_dispatch; zc_combine_backward; zc_expert_product on transposed weights;
 * zc_expert_weight_grad).
 *
 * Rows.  A slot is one (token, choice) pair, i = token * topk + choice, with
 * an expert id.  An id outside [0, experts) has no row here (another GPU's
 * expert, a dropped token).  c_e slots go to expert e; its segment is
 *   rows [offset_e, offset_e + c_e),   offset_(e+1) = offset_e + up(c_e, align)
 * in slot order, where up rounds up to a multiple of align.  Padding rows
 * (between offset_e + c_e and offset_(e+1)) are written as zeros by every call
 * that writes rows; rows from offset_E on are not written.
 *
 * 8-bit blocks.  Values are E4M3 (OCP, largest 448); every block of 128 has
 * one power-of-two scale, held as its biased exponent b in a byte (E8M0, the
 * scale is 2^(b-127)).  The scale is the least power of two s with
 * max|x| <= 448 s over the block's finite values, at least 2^-126, and 1 for
 * a block without any nonzero; x/s is then rounded once (to nearest even),
 * with no overflow.  Infinities and NaN are stored as NaN and do not enter
 * the maximum, so they stay in their own place.
 * A blocked matrix [rows, cols] is stored as data [rows, up(cols,128)] bytes
 * (zeros past cols) and scales [rows of blocks, up(ceil(cols/128),4)] bytes
 * (ones past the last block).  Blocks are
 *   1 x 128     (zc_quantize_rows, zc_dispatch_fp8)      one scale row per row,
 *   128 x 128   (zc_quantize_weights)                    one per 128 rows,
 *   128 rows of one column (zc_quantize_columns), stored block by block: for
 *               128 rows each, data [cols, 128] (a column's 128 values side by
 *               side) and up(cols,4) scales, so that a product over the rows
 *               reads whole strips.
 *
 * Conventions are zc.h's: device memory is the caller's; calls only enqueue
 * work on `stream` (no allocation, no synchronisation, no device memory read
 * on the host); argument errors are returned synchronously and enqueue
 * nothing; calls sharing a workspace must not overlap, nor may what a call
 * writes overlap what it reads.  Strides are in
 * elements between rows, the last dimension is contiguous.  Row-like buffers
 * need their element's alignment only (16-byte aligned pointers and strides
 * are faster); 8-bit data and scales need 16 bytes, workspaces 256.
 * row_capacity is the number of rows the row buffers hold; a slot whose row
 * is outside [0, row_capacity) counts as one without a row.
 * Results do not depend on timing: nothing is summed by atomics.
 */
#ifndef ZC_EXPERTS_H
#define ZC_EXPERTS_H

#include "zc.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum zc_dtype { ZC_BF16 = 0, ZC_FP16 = 1, ZC_FP32 = 2 } zc_dtype;

/* Limits: experts 1..1024, topk 1..64, align a power of two 1..1024, rows
 * below 2^31 (below 2^24 in blocks of 128 rows of one column:
 * zc_quantize_columns, zc_expert_weight_grad), row widths below 2^24.
 * zc_route_rows gives the rows that hold
 * every possible routing, up(slots + min(experts, slots) * (align - 1), align),
 * or 0 where a limit is passed.  A call whose launch would pass 2^32 threads is
 * refused with ZC_ERR_UNSUPPORTED. */
uint64_t zc_route_rows(uint64_t tokens, uint32_t topk, uint32_t experts, uint32_t align);
uint64_t zc_route_workspace_bytes(uint64_t tokens, uint32_t topk, uint32_t experts);

/*
 * Sorts the slots of d_ids (int32 [tokens, topk]) by expert, stably.  Writes
 * d_offsets (experts + 1), d_counts (experts), d_row (row of each slot, -1
 * without one; tokens * topk) and d_slot (slot of each row, -1 for a padding
 * row and past the last segment; row_capacity >= zc_route_rows).
 * ZC_ERR_CAPACITY where row_capacity or ws_bytes is too small,
 * ZC_ERR_UNSUPPORTED past a limit.
 */
zc_status zc_route(const int32_t *d_ids, uint64_t tokens, uint32_t topk, uint32_t experts,
                   uint32_t align, int32_t *d_offsets, int32_t *d_counts, int32_t *d_row,
                   int32_t *d_slot, uint64_t row_capacity, void *d_ws, uint64_t ws_bytes,
                   hipStream_t stream);

/* d_rows[row of (t, k)] = d_x[t] for every slot with a row; padding rows are
 * zeros.  d_offsets, d_counts, d_row: as zc_route wrote them.  d_counts NULL,
 * here and in the calls below: there are no padding rows (zc_route with align
 * 1), and nothing looks for them. */
zc_status zc_dispatch(const void *d_x, uint64_t x_stride, uint32_t dtype, uint64_t tokens,
                      uint32_t topk, uint32_t experts, uint32_t hidden, const int32_t *d_offsets,
                      const int32_t *d_counts, const int32_t *d_row, void *d_rows,
                      uint64_t rows_stride, uint64_t row_capacity, hipStream_t stream);

/* zc_dispatch with the rows stored as 8-bit blocks of 1 x 128 (each token is
 * cast once): d_data [rows, up(hidden,128)], d_scale [rows,
 * up(ceil(hidden/128),4)].  Padding rows: zeros, scale 1. */
zc_status zc_dispatch_fp8(const void *d_x, uint64_t x_stride, uint32_t dtype, uint64_t tokens,
                          uint32_t topk, uint32_t experts, uint32_t hidden,
                          const int32_t *d_offsets, const int32_t *d_counts, const int32_t *d_row,
                          void *d_data, void *d_scale, uint64_t row_capacity, hipStream_t stream);

/* d_y[t] = sum over the token's slots with a row of weight(t,k) * d_rows[row],
 * in 32 bits in order of k, rounded once; d_weights float [tokens, topk] or
 * NULL for ones (the gradient of zc_dispatch).  A token without rows gets
 * zeros. */
zc_status zc_combine(const void *d_rows, uint64_t rows_stride, const float *d_weights,
                     uint32_t dtype, uint64_t tokens, uint32_t topk, uint32_t hidden,
                     const int32_t *d_row, uint64_t row_capacity, void *d_y, uint64_t y_stride,
                     hipStream_t stream);

/* The gradient of zc_combine: d_drows[row] = weight * d_dy[t] (padding rows
 * zeros), d_dweights[t,k] = <d_dy[t], d_rows[row]> in 32 bits, 0 for a slot
 * without a row.  d_weights NULL: ones.  d_drows or d_dweights may be NULL
 * (not both); d_rows is needed for d_dweights only. */
zc_status zc_combine_backward(const void *d_dy, uint64_t dy_stride, const void *d_rows,
                              uint64_t rows_stride, const float *d_weights, uint32_t dtype,
                              uint64_t tokens, uint32_t topk, uint32_t experts, uint32_t hidden,
                              const int32_t *d_offsets, const int32_t *d_counts,
                              const int32_t *d_row, uint64_t row_capacity, void *d_drows,
                              uint64_t drows_stride, float *d_dweights, hipStream_t stream);

/* Casts x [rows, cols] to blocks of 1 x 128.  d_used: NULL, or a device
 * int32: rows from *d_used on are neither read nor written. */
zc_status zc_quantize_rows(const void *d_x, uint64_t x_stride, uint32_t dtype, uint64_t rows,
                           uint32_t cols, const int32_t *d_used, void *d_data, void *d_scale,
                           hipStream_t stream);

/* Casts [experts, n, k] weights (contiguous) to blocks of 128 x 128, stored
 * per expert as [n, k].  transpose: d_w is [experts, k, n] instead, and the
 * result is the blocked [n, k] of its transpose; both directions of one
 * weight have the same 8-bit values. */
zc_status zc_quantize_weights(const void *d_w, uint32_t dtype, uint32_t experts, uint32_t n,
                              uint32_t k, int transpose, void *d_data, void *d_scale,
                              hipStream_t stream);

/* Casts x [rows, cols] in blocks of 128 rows of one column: d_data
 * [ceil(rows/128), cols, 128], d_scale [ceil(rows/128), up(cols,4)]; rows past
 * the last are zeros.  d_used: as above; blocks that begin there or later are
 * neither read nor written, rows of the last one past it count as zeros. */
zc_status zc_quantize_columns(const void *d_x, uint64_t x_stride, uint32_t dtype, uint64_t rows,
                              uint32_t cols, const int32_t *d_used, void *d_data, void *d_scale,
                              hipStream_t stream);

/*
 * out[r, j] = sum over blocks b of sA[r,b] sW[e,j/128,b] <A[r,b], W[e,j,b]>
 * for the rows r of expert e's segment: A blocked [rows, k] (1 x 128), W
 * blocked [experts, n, k] (128 x 128), out [rows, n] of out_dtype.  The
 * matrix unit adds products of 8 neighbours in k at a time, each cut toward
 * zero to a multiple of 2^-13 of the group's largest power of two, and all
 * groups and blocks in 32 bits: about 2e-5 of the sum's root mean square off
 * on Gaussian data, whatever k, and at most 7 * 2^-13 of each group's
 * largest product.  Results in 16 bits hardly show it beside their own
 * rounding (1.7e-3 in bf16, 2e-4 in fp16); results in 32 bits are that far from
 * a product in 32-bit arithmetic.  zc_expert_weight_grad adds in the same way.
 * d_offsets NULL: one expert, all rows (experts must be 1, d_counts NULL).
 * d_counts NULL: segments are whole, offset_e to offset_(e+1).  Padding rows
 * are written as zeros.  Offsets and counts that leave [0, rows] are clamped.
 */
zc_status zc_expert_product(const void *d_a, const void *d_a_scale, uint64_t rows, const void *d_w,
                            const void *d_w_scale, uint32_t experts, uint32_t n, uint32_t k,
                            const int32_t *d_offsets, const int32_t *d_counts, void *d_out,
                            uint64_t out_stride, uint32_t out_dtype, hipStream_t stream);

/*
 * dW[e][i, j] = sum over the blocks b of 128 rows in expert e's segment of
 * sY[i,b] sX[j,b] <Y[b,i], X[b,j]>: Y and X as zc_quantize_columns makes them
 * from [rows, n] and [rows, k], dW contiguous [experts, n, k] of
 * out_dtype; an expert without rows gets zeros.  Segments begin at multiples
 * of 128 (zc_route with such an align), padding rows are zeros; a segment that
 * shares a block of 128 rows with another one gets NaN.  d_offsets NULL: one
 * expert, all rows.
 * Long segments of small weights are summed in parts, joined in their order,
 * where d_ws holds them: zc_expert_weight_grad_workspace_bytes (0: none would
 * be used, or a limit is passed).  d_ws NULL: every sum in one piece.  Which parts are taken goes by
 * the arguments alone.
 */
uint64_t zc_expert_weight_grad_workspace_bytes(uint64_t rows, uint32_t experts, uint32_t n, uint32_t k);
zc_status zc_expert_weight_grad(const void *d_y, const void *d_y_scale, const void *d_x,
                                const void *d_x_scale, uint64_t rows, uint32_t experts, uint32_t n,
                                uint32_t k, const int32_t *d_offsets, void *d_dw,
                                uint32_t out_dtype, void *d_ws, uint64_t ws_bytes,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* ZC_EXPERTS_H */
