// zc_rows.hip -- rows to experts and back, with weights, and the gradient.
//
//   dispatch:  R[row(t,k)] = x[t]
//   combine:   y[t] = sum over k of w(t,k) R[row(t,k)]
//   gradient:  dR[row(t,k)] = w(t,k) dy[t],  dw(t,k) = <dy[t], R[row(t,k)]>
//
// All three go by token: a token's row is read once and its topk rows are
// written or read from there, so nothing is fetched twice and every sum has a
// fixed order.  Bound by memory: dispatch moves (1 + topk) rows per token,
// combine the same, the gradient 1 + 2 topk.
//
// Rows are moved in 16-byte words wherever they start (the memory takes words
// at any element's address; a copy of odd rows of 7169 16-bit values runs at
// 4.1 TB/s so and at 3.2 by elements); the last, shorter word of a row goes
// by elements.
#include "zc_experts_kernels.h"

namespace zc {

namespace {

template <typename T>
struct Pack {
    static constexpr int N = 16 / (int)sizeof(T);
    typedef xu32x4 __attribute__((aligned(2))) Word;
    union {
        xu32x4 w;
        T v[N];
    };
};

// What a launch moves past the caches (nontemporal), by its size:
//   stores of dispatched rows and of gradients from 256 MB on (with the rows
//     read for dweights), which the Infinity Cache (256 MB) cannot hold for a
//     reader (537 MB of dispatched rows 116 -> 103 us; 268 MB 50 -> 52; 134 MB
//     25 -> 27; 420 MB of rows' gradients 93 -> 67);
//   combine's loads from 512 MB on, which it cannot hold from their writer
//     (940 MB combined 190 -> 174 us; 33 MB 7.7 -> 9.7).
// Such stores want whole sectors of 64 bytes: where rows do not begin at
// multiples of 64, a wave that starts at a row's start leaves part of a sector
// at both its ends, and each costs several whole ones (8192 tokens to 8 rows
// each, 4096 / 4104 / 4112 / 4128 values: 103 / 151 / 146 / 112 us).  So there
// every word is taken at a multiple of 16 bytes of the row it goes to, the
// wave's first at a multiple of 64, and the first and last word of a row are
// moved to its ends, over their neighbours, which store the same there (4104
// values 151 -> 118 us, 7170 values 265 -> 201).  Rows below 4 KB have too
// many ends and stay in the caches (1000 values, 20,000 tokens: 78; past them
// 88, shifted 91).  The gradient with dweights gains nothing from the shift,
// which reads dy for every row again (4104 values: 259; 285).
enum Mode { kCached, kPast, kPastShifted };

// Element of a row of `width` where the word for column `col` begins.
struct Shifted {
    int32_t at;
    bool any;
};
template <typename T>
__device__ __forceinline__ Shifted shifted(const T* row, uint32_t col, uint32_t width) {
    constexpr int32_t N = 16 / (int)sizeof(T);
    const int32_t w = (int32_t)width;
    const int32_t nominal = (int32_t)col - (int32_t)(((uint32_t)(uintptr_t)row & 63) / sizeof(T));
    const int32_t lo = nominal < 0 ? 0 : nominal;
    return Shifted{lo > w - N ? w - N : lo, nominal > -N && nominal < w};
}

// A word of a row, or its last `n` values.
template <typename T, bool PAST>
__device__ __forceinline__ Pack<T> load(const T* p, uint32_t n) {
    typedef Pack<T> P;
    P x;
    if (n >= P::N) {
        if (PAST) x.w = __builtin_nontemporal_load(reinterpret_cast<const typename P::Word*>(p));
        else x.w = *reinterpret_cast<const typename P::Word*>(p);
    } else {
#pragma unroll
        for (uint32_t i = 0; i < P::N; ++i) x.v[i] = i < n ? p[i] : (T)0.0f;
    }
    return x;
}

template <typename T, bool PAST>
__device__ __forceinline__ void store(T* p, const Pack<T>& x, uint32_t n) {
    typedef Pack<T> P;
    if (n >= P::N) {
        if (PAST) __builtin_nontemporal_store(x.w, reinterpret_cast<typename P::Word*>(p));
        else *reinterpret_cast<typename P::Word*>(p) = x.w;
    } else {
#pragma unroll
        for (uint32_t i = 0; i < P::N; ++i)
            if (i < n) p[i] = x.v[i];
    }
}

template <typename T>
__device__ __forceinline__ T* row_of(const void* base, uint64_t row, uint64_t stride_bytes) {
    return reinterpret_cast<T*>(const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) + row * stride_bytes);
}

// How a launch is cut: workgroups of tx columns (words) by 256 / tx tokens, tx
// a power of two; the column blocks of a token go to one XCD (every eighth
// workgroup), whose L2 joins what they share of a line (4097 values: combine
// 115 -> 106 us, dispatch 167 -> 152).  From 64
// columns on a wave has one token, whose rows and weights are then scalar
// loads.
struct Split {
    uint32_t log_tx;
    uint32_t col_blocks;
    uint32_t blocks;
    uint32_t pad_blocks;  // workgroups of the padding rows, before the others
};

struct Place {
    uint32_t token, col;  // col: first element
};

template <typename T, bool WAVE>
__device__ __forceinline__ Place place_of(const Split& s) {
    const uint32_t block = blockIdx.x - s.pad_blocks;
    const uint32_t ty = threadIdx.x >> s.log_tx, tx = threadIdx.x & ((1u << s.log_tx) - 1);
    const uint32_t n = block >> 3, tb = n / s.col_blocks * 8 + (block & 7), cb = n % s.col_blocks;
    return Place{tb * (256u >> s.log_tx) + (WAVE ? uniform(ty) : ty), ((cb << s.log_tx) + tx) * Pack<T>::N};
}

// Zeros in the padding rows, kPadSplit workgroups for each expert, a wave for
// a row.  They are the launch's first workgroups: as its last they ran alone
// at the end (4756 padding rows of 10 KB added 34 us to a dispatch of 80).
constexpr uint32_t kPadSplit = 4;

template <typename T>
__device__ __forceinline__ void zero_padding(const RowArgs& a) {
    const uint32_t e = blockIdx.x / kPadSplit, first = blockIdx.x % kPadSplit * 4 + uniform(threadIdx.x >> 6);
    const uint32_t lo = (uint32_t)a.offsets[e] + (uint32_t)a.counts[e];
    uint32_t hi = (uint32_t)a.offsets[e + 1];
    hi = hi < a.capacity ? hi : a.capacity;
    Pack<T> zero;
    zero.w = xu32x4{};
    for (uint32_t r = lo + first; r < hi; r += kPadSplit * 4) {
        T* out = row_of<T>(a.out, r, a.out_stride);
        for (uint32_t c = __lane_id() * Pack<T>::N; c < a.width; c += 64 * Pack<T>::N)
            store<T, false>(out + c, zero, a.width - c);
    }
}

template <typename T, bool WAVE, Mode MODE>
__global__ __launch_bounds__(256) void dispatch_rows(RowArgs a, Split s) {
    if (blockIdx.x < s.pad_blocks) {
        zero_padding<T>(a);
        return;
    }
    const Place at = place_of<T, WAVE>(s);
    if (at.token >= a.tokens) return;
    const T* in = row_of<const T>(a.x, at.token, a.x_stride);
    const int32_t* row = a.row + (uint64_t)at.token * a.topk;
    if constexpr (MODE == kPastShifted) {
#pragma unroll 4
        for (uint32_t k = 0; k < a.topk; ++k) {
            const uint32_t r = (uint32_t)row[k];
            if (r >= a.capacity) continue;
            T* out = row_of<T>(a.out, r, a.out_stride);
            const Shifted c = shifted(out, at.col, a.width);
            if (c.any) store<T, true>(out + c.at, load<T, false>(in + c.at, Pack<T>::N), Pack<T>::N);
        }
    } else {
        if (at.col >= a.width) return;
        const Pack<T> x = load<T, false>(in + at.col, a.width - at.col);
        for (uint32_t k = 0; k < a.topk; ++k) {
            const uint32_t r = (uint32_t)row[k];
            if (r < a.capacity) store<T, MODE == kPast>(row_of<T>(a.out, r, a.out_stride) + at.col, x, a.width - at.col);
        }
    }
}

template <typename T, bool WAVE, bool PAST>
__global__ __launch_bounds__(256) void combine_rows(RowArgs a, Split s) {
    typedef Pack<T> P;
    const Place at = place_of<T, WAVE>(s);
    if (at.token >= a.tokens || at.col >= a.width) return;
    const uint32_t n = a.width - at.col;
    float acc[P::N] = {};
    const int32_t* row = a.row + (uint64_t)at.token * a.topk;
    const float* weight = a.weights ? a.weights + (uint64_t)at.token * a.topk : nullptr;
#pragma unroll 4
    for (uint32_t k = 0; k < a.topk; ++k) {
        const uint32_t r = (uint32_t)row[k];
        if (r >= a.capacity) continue;
        const float w = weight ? weight[k] : 1.0f;
        const P x = load<T, PAST>(row_of<const T>(a.x, r, a.x_stride) + at.col, n);
#pragma unroll
        for (int i = 0; i < P::N; ++i) acc[i] = __builtin_fmaf(w, to_float(x.v[i]), acc[i]);
    }
    P y;
#pragma unroll
    for (int i = 0; i < P::N; ++i) y.v[i] = (T)acc[i];
    store<T, PAST>(row_of<T>(a.out, at.token, a.out_stride) + at.col, y, n);
}

// L threads per token (a workgroup or less); kGroup slots at a time (dy is
// read again, from the cache, for every further group).
constexpr int kGroup = 8;

template <typename T, int L, Mode MODE>
__global__ __launch_bounds__(256) void combine_rows_backward(RowArgs a, uint32_t pad_blocks) {
    typedef Pack<T> P;
    if (blockIdx.x < pad_blocks) {
        zero_padding<T>(a);
        return;
    }
    const uint32_t thread = threadIdx.x % L, sub = threadIdx.x / L;
    const uint64_t t = (uint64_t)(blockIdx.x - pad_blocks) * (256 / L) + (L >= 64 ? uniform(sub) : sub);
    if (t >= a.tokens) return;  // L = 256: no workgroup
    const T* dy = row_of<const T>(a.x, t, a.x_stride);
    for (uint32_t k0 = 0; k0 < a.topk; k0 += kGroup) {
        uint32_t r[kGroup];
        float w[kGroup], acc[kGroup];
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
            const uint32_t k = k0 + g;
            r[g] = k < a.topk ? (uint32_t)a.row[t * a.topk + k] : ~0u;
            w[g] = k < a.topk && a.weights ? a.weights[t * a.topk + k] : 1.0f;
            acc[g] = 0.0f;
        }
        const uint32_t end = a.width + (MODE == kPastShifted ? 63 / sizeof(T) : 0);
        for (uint32_t c = thread * P::N; c < end; c += L * P::N) {
            const uint32_t n = a.width - c;
            P d;
            if (MODE != kPastShifted) d = load<T, false>(dy + c, n);
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                if (r[g] >= a.capacity) continue;
                if constexpr (MODE == kPastShifted) {  // no dweights
                    T* out = row_of<T>(a.out, r[g], a.out_stride);
                    const Shifted s = shifted(out, c, a.width);
                    if (!s.any) continue;
                    d = load<T, false>(dy + s.at, P::N);
                    P o;
#pragma unroll
                    for (int i = 0; i < P::N; ++i) o.v[i] = (T)(w[g] * to_float(d.v[i]));
                    store<T, true>(out + s.at, o, P::N);
                } else {
                    if (a.dweights) {
                        const P x = load<T, false>(row_of<const T>(a.rows, r[g], a.rows_stride) + c, n);
#pragma unroll
                        for (int i = 0; i < P::N; ++i)
                            acc[g] = __builtin_fmaf(to_float(d.v[i]), to_float(x.v[i]), acc[g]);
                    }
                    if (a.out) {
                        P o;
#pragma unroll
                        for (int i = 0; i < P::N; ++i) o.v[i] = (T)(w[g] * to_float(d.v[i]));
                        store<T, MODE == kPast>(row_of<T>(a.out, r[g], a.out_stride) + c, o, n);
                    }
                }
            }
        }
        if (MODE == kPastShifted || !a.dweights) continue;
        float mine = 0.0f;
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
            for (int m = L < 64 ? L / 2 : 32; m; m >>= 1) acc[g] += __shfl_xor(acc[g], m);
            if ((int)thread == g) mine = acc[g];
        }
        if constexpr (L > 64) {
            __shared__ float part[4][kGroup];
            if (k0) __syncthreads();  // the last group's sums have been read
            if (__lane_id() == 0)
#pragma unroll
                for (int g = 0; g < kGroup; ++g) part[threadIdx.x >> 6][g] = acc[g];
            __syncthreads();
            if (thread < kGroup) mine = (part[0][thread] + part[1][thread]) + (part[2][thread] + part[3][thread]);
        }
        if (thread < kGroup && k0 + thread < a.topk) a.dweights[t * a.topk + k0 + thread] = mine;
    }
}

// The widest tx that leaves at most an eighth of the threads without a word,
// or else the fewest.
Split split(uint32_t words, uint32_t tokens, uint32_t pad_blocks) {
    uint32_t best = 0, waste = ~0u;
    for (uint32_t lt = 0; lt <= 8; ++lt) {
        const uint32_t w = up_to(words, 1u << lt) - words;
        if (w * 8 <= words || w <= waste) {
            best = lt;
            waste = w;
        }
    }
    const uint32_t ty = 256u >> best, cols = (words + (1u << best) - 1) >> best;
    const uint64_t blocks = (uint64_t)up_to((tokens + ty - 1) / ty, 8) * cols;
    return Split{best, cols, (uint32_t)(blocks < ~0u ? blocks : ~0u), pad_blocks};
}

uint32_t pad_blocks(const RowArgs& a) { return a.counts ? a.experts * kPadSplit : 0; }

template <typename T>
uint64_t rows_bytes(const RowArgs& a) { return (uint64_t)a.tokens * a.topk * a.width * sizeof(T); }

constexpr uint64_t kStoresPast = 256ull << 20, kLoadsPast = 512ull << 20;

template <typename T>
Mode store_mode(const RowArgs& a) {
    if (!a.out || rows_bytes<T>(a) * (a.dweights ? 2 : 1) < kStoresPast) return kCached;
    if (a.dweights || !(((uintptr_t)a.out | a.out_stride) & 63)) return kPast;
    return a.width * sizeof(T) >= 4096 ? kPastShifted : kCached;
}

template <typename T>
zc_status dispatch_as(const RowArgs& a, hipStream_t stream) {
    const Mode mode = store_mode<T>(a);
    const uint32_t values = a.width + (mode == kPastShifted ? 63 / sizeof(T) : 0);
    const Split s = split((values + Pack<T>::N - 1) / Pack<T>::N, a.tokens, pad_blocks(a));
    if (!fits((uint64_t)s.blocks + s.pad_blocks)) return ZC_ERR_UNSUPPORTED;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(s.blocks + s.pad_blocks), dim3(256), 0, stream, a, s);
        return ZC_OK;
    };
    if (mode == kPastShifted)
        return s.log_tx >= 6 ? launch(dispatch_rows<T, true, kPastShifted>) : launch(dispatch_rows<T, false, kPastShifted>);
    if (mode == kPast) return s.log_tx >= 6 ? launch(dispatch_rows<T, true, kPast>) : launch(dispatch_rows<T, false, kPast>);
    return s.log_tx >= 6 ? launch(dispatch_rows<T, true, kCached>) : launch(dispatch_rows<T, false, kCached>);
}

template <typename T>
zc_status combine_as(const RowArgs& a, hipStream_t stream) {
    const Split s = split((a.width + Pack<T>::N - 1) / Pack<T>::N, a.tokens, 0);
    if (!fits(s.blocks)) return ZC_ERR_UNSUPPORTED;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(s.blocks), dim3(256), 0, stream, a, s);
        return ZC_OK;
    };
    const bool past = rows_bytes<T>(a) >= kLoadsPast;
    if (s.log_tx >= 6) return past ? launch(combine_rows<T, true, true>) : launch(combine_rows<T, true, false>);
    return past ? launch(combine_rows<T, false, true>) : launch(combine_rows<T, false, false>);
}

template <typename T, int L>
zc_status backward_by(const RowArgs& a, hipStream_t stream) {
    const uint32_t pads = a.out ? pad_blocks(a) : 0, per = 256 / L, groups = (a.tokens + per - 1) / per;
    if (!fits((uint64_t)groups + pads)) return ZC_ERR_UNSUPPORTED;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(groups + pads), dim3(256), 0, stream, a, pads);
        return ZC_OK;
    };
    switch (store_mode<T>(a)) {
        case kPastShifted: return launch(combine_rows_backward<T, L, kPastShifted>);
        case kPast: return launch(combine_rows_backward<T, L, kPast>);
        default: return launch(combine_rows_backward<T, L, kCached>);
    }
}

// Threads per token, in us (4096 tokens, 4 rows each, unless stated):
//            16 / 64 / 256 threads
//    200 values    6.9 /  7.6 /  14
//    400          11.8 /  8.8 /  16
//   1001          23.5 / 16.4 /  24
//   1500            32 /   23 /  27
//   2048 (8192 tokens, 8 rows)  171 / 157 / 112
template <typename T>
zc_status backward_as(const RowArgs& a, hipStream_t stream) {
    const uint32_t words = (a.width + Pack<T>::N - 1) / Pack<T>::N;
    if (words <= 32) return backward_by<T, 16>(a, stream);
    return words <= 192 ? backward_by<T, 64>(a, stream) : backward_by<T, 256>(a, stream);
}

}  // namespace

zc_status launch_dispatch(const RowArgs& a, uint32_t dtype, hipStream_t stream) {
    // a copy: 16-bit values of either type are the same
    return dtype == ZC_FP32 ? dispatch_as<float>(a, stream) : dispatch_as<_Float16>(a, stream);
}

zc_status launch_combine(const RowArgs& a, uint32_t dtype, hipStream_t stream) {
    if (dtype == ZC_BF16) return combine_as<__bf16>(a, stream);
    if (dtype == ZC_FP16) return combine_as<_Float16>(a, stream);
    return combine_as<float>(a, stream);
}

zc_status launch_combine_backward(const RowArgs& a, uint32_t dtype, hipStream_t stream) {
    if (dtype == ZC_BF16) return backward_as<__bf16>(a, stream);
    if (dtype == ZC_FP16) return backward_as<_Float16>(a, stream);
    return backward_as<float>(a, stream);
}

}  // namespace zc
