// zc_blocks.hip -- casts to 8-bit blocks of 128 with power-of-two scales.
//
//   s = least power of two with max|x| <= 448 s,   q = E4M3(x / s)
//
// Division by a power of two is exact, so each value is rounded once and the
// result does not depend on how a block is split over lanes.
//
// Bound by memory: the input is read once, into registers, and every block's
// maximum found there.  Measured, of bytes read and written: rows 16384 x 7168
// 53 us (6.7 TB/s), weights 64 x 2048 x 1408 101 us (5.5), transposed 106 (5.2),
// columns 16384 x 7168 66 us (5.3), dispatch of 8192 tokens to 8 rows of 7168 as
// blocks 92 us (6.4).
#include "zc_experts_kernels.h"

namespace zc {

namespace {

constexpr uint32_t kWaveCols = 1024;  // columns of one wave: 16 per lane, 8 blocks

template <typename T>
struct Pack16 {
    static constexpr int N = 16 / (int)sizeof(T);     // values per word
    typedef xu32x4 __attribute__((aligned(2))) Word;  // at any element's address
    union {
        xu32x4 w[sizeof(T)];  // 16 values
        T v[16];
    };
};

constexpr uint32_t kPadSplit = 4;  // workgroups for the padding rows of an expert

// Blocks of 1 x 128.  A wave casts 1024 columns of one token, 16 per lane (or,
// where a row has 4 blocks at most, L = 8, 16 or 32 lanes do a token), so a
// block is 8 lanes and its bytes leave in one 16-byte store per lane; the
// stores go to every row of the token, past the caches (PAST) where the rows
// are more than the L2s hold.  The workgroups of the padding rows come first.
template <typename T, int L, bool PAST>
__global__ __launch_bounds__(256) void cast_rows(CastRowsArgs a, uint32_t pieces, uint32_t pad_blocks) {
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6);
    if (blockIdx.x < pad_blocks) {
        const uint32_t e = blockIdx.x / kPadSplit, first = blockIdx.x % kPadSplit * 4 + wave;
        const uint32_t lo = (uint32_t)a.offsets[e] + (uint32_t)a.counts[e];
        uint32_t hi = (uint32_t)a.offsets[e + 1];
        hi = hi < a.capacity ? hi : a.capacity;
        for (uint32_t r = lo + first; r < hi; r += kPadSplit * 4) {
            for (uint32_t c = lane * 16; c < a.data_stride; c += 1024)
                *reinterpret_cast<xu32x4*>(a.data + (uint64_t)r * a.data_stride + c) = xu32x4{};
            for (uint32_t c = lane * 4; c < a.scale_stride; c += 256)
                *reinterpret_cast<uint32_t*>(a.scale + (uint64_t)r * a.scale_stride + c) = 0x7F7F7F7Fu;
        }
        return;
    }
    const uint64_t item = (uint64_t)(blockIdx.x - pad_blocks) * 4 + wave;
    const uint32_t piece = L < 64 ? 0 : (uint32_t)(item % pieces), in = lane % L;
    const uint64_t t = L < 64 ? item * (64 / L) + lane / L : item / pieces;
    uint32_t tokens = a.tokens;
    if (a.used) {
        const int32_t u = *a.used;
        tokens = u < 0 ? 0 : (uint32_t)u < tokens ? (uint32_t)u : tokens;
    }
    if (t >= tokens) return;
    const uint32_t c = piece * kWaveCols + in * 16;
    const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
    Pack16<T> p;
    if (c + 16 <= a.width) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) p.w[i] = reinterpret_cast<const typename Pack16<T>::Word*>(x + c)[i];
    } else {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i)
            p.w[i] = load_word(x + c + i * Pack16<T>::N, (int32_t)(a.width - c) - i * Pack16<T>::N);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, finite_bits(to_float(p.v[i])));
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    const uint32_t b = scale_byte(top);
    const float inv = inverse_scale(b);
    xu32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = four_fp8(scaled(to_float(p.v[4 * i]), inv), scaled(to_float(p.v[4 * i + 1]), inv),
                        scaled(to_float(p.v[4 * i + 2]), inv), scaled(to_float(p.v[4 * i + 3]), inv));
    // four blocks' bytes per word, in the first of their lanes; blocks past the last
    // are all zeros and so get scale 1
    uint32_t s = b << (8 * ((in >> 3) & 3));
    if (L >= 16) s |= (uint32_t)__shfl_xor((int)s, 8);
    if (L >= 32) s |= (uint32_t)__shfl_xor((int)s, 16);
    if (L < 32) s |= 0x7F7F7F7Fu << L;
    const uint32_t sc = piece * 8 + (in >> 5) * 4;
    const bool has_scale = (in & 31) == 0 && sc < a.scale_stride;
    auto store = [&](uint64_t r) {
        xu32x4* out = reinterpret_cast<xu32x4*>(a.data + r * a.data_stride + c);
        if (c < a.data_stride) {
            if (PAST) __builtin_nontemporal_store(q, out);
            else *out = q;
        }
        if (has_scale) *reinterpret_cast<uint32_t*>(a.scale + r * a.scale_stride + sc) = s;
    };
    if (!a.row) {
        store(t);
        return;
    }
    for (uint32_t k = 0; k < a.topk; ++k) {
        const uint32_t r = (uint32_t)a.row[t * a.topk + k];
        if (r < a.capacity) store(r);
    }
}

enum CastMode { kWeights, kWeightsTransposed, kColumns };

// One 128 x 128 tile of x per workgroup; a thread has 8 rows by 8 columns, so
// that turned over its 8 rows are 8 neighbouring bytes.
template <typename T, CastMode MODE>
__global__ __launch_bounds__(256) void cast_tile(CastTileArgs a, uint32_t row_tiles, uint32_t col_tiles) {
    constexpr bool TURN = MODE != kWeights;
    // Turned over, 128 rows of 128 bytes.  Rows 8 cg + j, written by 16 cg at a
    // time, change places in pairs by cg's lowest bit and their 16-byte pieces
    // by the other three, so that a write, and a read of whole rows, uses all
    // 64 banks (against rows 144 bytes apart, conflicts 85 -> 39% of LDS cycles,
    // columns of 32,768 x 1024 26 -> 21 us).
    __shared__ __align__(16) uint8_t turn[TURN ? 128 * 128 : 16];
    auto turned = [](uint32_t row, uint32_t piece) {
        const uint32_t g = row >> 3;
        return (row ^ (g & 1)) * 128 + ((piece ^ (g >> 1)) << 4);
    };
    __shared__ uint32_t tops[MODE == kColumns ? 16 * 128 : 4];
    const uint32_t tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
    uint32_t bt = blockIdx.x;
    const uint32_t ct = bt % col_tiles;
    bt /= col_tiles;
    const uint32_t rt = bt % row_tiles, e = bt / row_tiles;
    // x as it lies: [xrows, xcols]
    const uint32_t xrows = MODE == kWeightsTransposed ? a.cols : a.rows;
    const uint32_t xcols = MODE == kWeightsTransposed ? a.rows : a.cols;
    uint32_t limit = xrows;
    if (MODE == kColumns && a.used) {
        const int32_t u = *a.used;
        limit = u < 0 ? 0 : (uint32_t)u < limit ? (uint32_t)u : limit;
        if (rt * 128 >= limit) return;
    }
    const T* x = static_cast<const T*>(a.x) + (MODE == kColumns ? 0 : (uint64_t)e * xrows * xcols);
    const uint64_t stride = MODE == kColumns ? a.x_stride : xcols;
    const uint32_t c0 = ct * 128 + cg * 8, r0 = rt * 128 + rg * 8;
    union {
        xu32x4 w[sizeof(T) / 2];
        T v[8];
    } p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const T* xr = x + (r0 + i) * stride + c0;
        const int32_t n = r0 + i < limit ? (int32_t)(xcols - c0) : 0;
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h) p[i].w[h] = load_word(xr + h * Pack16<T>::N, n - h * Pack16<T>::N);
    }
    uint32_t sbyte[8];
    float inv[8];
    if (MODE == kColumns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, finite_bits(to_float(p[i].v[j])));
            tops[rg * 128 + cg * 8 + j] = top;
        }
        __syncthreads();
        if (tid < 128) {
            uint32_t top = 0;
            for (int g = 0; g < 16; ++g) top = max(top, tops[g * 128 + tid]);
            tops[tid] = scale_byte(top);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) inv[j] = inverse_scale(sbyte[j] = tops[cg * 8 + j]);
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, finite_bits(to_float(p[i].v[j])));
        for (int m = 32; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
        if ((tid & 63) == 0) tops[tid >> 6] = top;
        __syncthreads();
        const uint32_t b = scale_byte(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
#pragma unroll
        for (int j = 0; j < 8; ++j) inv[j] = inverse_scale(sbyte[j] = b);
    }
    // the result's rows and columns of blocks, and its tile
    const uint32_t orow_tiles = MODE == kWeights ? row_tiles : col_tiles;
    const uint32_t or0 = (MODE == kWeights ? rt : ct) * 128, ob = MODE == kWeights ? ct : rt;
    const uint32_t orows = MODE == kColumns ? a.cols : a.rows;
    const uint32_t blocks = MODE == kWeights ? col_tiles : row_tiles;
    // columns: block ob is [cols][128] bytes
    uint8_t* data = MODE == kColumns ? a.data + (uint64_t)ob * orows * 128 : a.data + (uint64_t)e * orows * a.data_stride;
    if (MODE == kWeights) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const xu32x2 q = {four_fp8(scaled(to_float(p[i].v[0]), inv[0]), scaled(to_float(p[i].v[1]), inv[1]),
                                       scaled(to_float(p[i].v[2]), inv[2]), scaled(to_float(p[i].v[3]), inv[3])),
                              four_fp8(scaled(to_float(p[i].v[4]), inv[4]), scaled(to_float(p[i].v[5]), inv[5]),
                                       scaled(to_float(p[i].v[6]), inv[6]), scaled(to_float(p[i].v[7]), inv[7]))};
            if (r0 + i < orows) *reinterpret_cast<xu32x2*>(data + (uint64_t)(r0 + i) * a.data_stride + c0) = q;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const xu32x2 q = {four_fp8(scaled(to_float(p[0].v[j]), inv[j]), scaled(to_float(p[1].v[j]), inv[j]),
                                       scaled(to_float(p[2].v[j]), inv[j]), scaled(to_float(p[3].v[j]), inv[j])),
                              four_fp8(scaled(to_float(p[4].v[j]), inv[j]), scaled(to_float(p[5].v[j]), inv[j]),
                                       scaled(to_float(p[6].v[j]), inv[j]), scaled(to_float(p[7].v[j]), inv[j]))};
            *reinterpret_cast<xu32x2*>(turn + turned(cg * 8 + j, rg >> 1) + (rg & 1) * 8) = q;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = i * 32 + (tid >> 3), c = (tid & 7) * 16;
            if (or0 + r < orows)
                *reinterpret_cast<xu32x4*>(data + (MODE == kColumns ? (uint64_t)(or0 + r) * 128 : (uint64_t)(or0 + r) * a.data_stride + ob * 128) + c) =
                    *reinterpret_cast<const xu32x4*>(turn + turned(r, tid & 7));
        }
    }
    // scales; ones past the last block, or past the last column
    if (MODE == kColumns) {
        if (rg == 0) {
            const uint32_t c = or0 + cg * 8;
            uint8_t* s = a.scale + (uint64_t)ob * a.scale_stride + c;
#pragma unroll
            for (int h = 0; h < 2; ++h)  // columns past the last are zeros, and so have scale 1
                if (c + h * 4 < a.scale_stride)
                    *reinterpret_cast<uint32_t*>(s + h * 4) = sbyte[h * 4] | sbyte[h * 4 + 1] << 8 | sbyte[h * 4 + 2] << 16 |
                                                              sbyte[h * 4 + 3] << 24;
        }
    } else if (tid == 0) {
        uint8_t* s = a.scale + ((uint64_t)e * orow_tiles + or0 / 128) * a.scale_stride;
        s[ob] = (uint8_t)sbyte[0];
        if (ob == blocks - 1)
            for (uint32_t b = blocks; b < a.scale_stride; ++b) s[b] = 127;
    }
}

template <typename T, int L>
zc_status rows_by(const CastRowsArgs& a, hipStream_t stream) {
    const uint32_t pieces = (a.data_stride + kWaveCols - 1) / kWaveCols;
    const uint64_t items = L < 64 ? ((uint64_t)a.tokens * L + 63) / 64 : (uint64_t)a.tokens * pieces, blocks = (items + 3) / 4;
    const uint32_t pads = a.counts ? a.experts * kPadSplit : 0;
    if (!fits(blocks + pads)) return ZC_ERR_UNSUPPORTED;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks + pads), dim3(256), 0, stream, a, pieces, pads);
        return ZC_OK;
    };
    const bool past = (uint64_t)a.tokens * a.topk * a.data_stride >= (64ull << 20);
    return past ? launch(cast_rows<T, L, true>) : launch(cast_rows<T, L, false>);
}

// 39,836 rows of 98 and 100,000 of 300 values: by 64 lanes a token 17 and 39 us,
// by 8 and 32 of them 6 and 25.
template <typename T>
zc_status rows_type(const CastRowsArgs& a, hipStream_t stream) {
    if (a.data_stride <= 128) return rows_by<T, 8>(a, stream);
    if (a.data_stride <= 256) return rows_by<T, 16>(a, stream);
    return a.data_stride <= 512 ? rows_by<T, 32>(a, stream) : rows_by<T, 64>(a, stream);
}

template <typename T>
zc_status weights_type(const CastTileArgs& a, hipStream_t stream) {
    const uint32_t nt = (a.rows + 127) / 128, kt = (a.cols + 127) / 128;
    if (!fits((uint64_t)nt * kt * a.experts)) return ZC_ERR_UNSUPPORTED;
    if (a.transpose)
        hipLaunchKernelGGL((cast_tile<T, kWeightsTransposed>), dim3(nt * kt * a.experts), dim3(256), 0, stream, a, kt, nt);
    else
        hipLaunchKernelGGL((cast_tile<T, kWeights>), dim3(nt * kt * a.experts), dim3(256), 0, stream, a, nt, kt);
    return ZC_OK;
}

template <typename T>
zc_status columns_type(const CastTileArgs& a, hipStream_t stream) {
    const uint32_t rt = (a.rows + 127) / 128, ct = (a.cols + 127) / 128;
    if (!fits((uint64_t)rt * ct)) return ZC_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((cast_tile<T, kColumns>), dim3(rt * ct), dim3(256), 0, stream, a, rt, ct);
    return ZC_OK;
}

}  // namespace

zc_status launch_cast_rows(const CastRowsArgs& a, uint32_t dtype, hipStream_t stream) {
    if (dtype == ZC_BF16) return rows_type<__bf16>(a, stream);
    if (dtype == ZC_FP16) return rows_type<_Float16>(a, stream);
    return rows_type<float>(a, stream);
}

zc_status launch_cast_weights(const CastTileArgs& a, uint32_t dtype, hipStream_t stream) {
    if (dtype == ZC_BF16) return weights_type<__bf16>(a, stream);
    if (dtype == ZC_FP16) return weights_type<_Float16>(a, stream);
    return weights_type<float>(a, stream);
}

zc_status launch_cast_columns(const CastTileArgs& a, uint32_t dtype, hipStream_t stream) {
    if (dtype == ZC_BF16) return columns_type<__bf16>(a, stream);
    if (dtype == ZC_FP16) return columns_type<_Float16>(a, stream);
    return columns_type<float>(a, stream);
}

}  // namespace zc
