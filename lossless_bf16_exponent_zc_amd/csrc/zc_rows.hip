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
// 4.1 TB/s so and at 3.2 by elements); the last, shorter word of a row is moved
// to the row's end, over its neighbour.
//
// 8192 tokens, 8 rows each, 7168 16-bit values: dispatch 180 us (5.9 TB/s; 211
// and 5.0, a copy's rate, where x is not in the Infinity Cache), combine 174
// (6.1 TB/s), gradient 394 (5.1 TB/s).  8 tokens: 3.5 us each, the launch.
#include "zc_experts_kernels.h"

#include <type_traits>

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

// A row's last word moved to the row's end, over its neighbour, so that it is
// whole (where the row has a word).
struct Last {
    uint32_t at, n;
};
template <typename T>
__device__ __forceinline__ Last last_moved(uint32_t col, uint32_t width) {
    constexpr uint32_t N = Pack<T>::N;
    if (width < N) return Last{0, width};
    return Last{col + N <= width ? col : width - N, N};
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
        const Last c = last_moved<T>(at.col, a.width);
        const Pack<T> x = load<T, false>(in + c.at, c.n);
        for (uint32_t k = 0; k < a.topk; ++k) {
            const uint32_t r = (uint32_t)row[k];
            if (r < a.capacity) store<T, MODE == kPast>(row_of<T>(a.out, r, a.out_stride) + c.at, x, c.n);
        }
    }
}

template <typename T, bool WAVE, bool PAST>
__global__ __launch_bounds__(256) void combine_rows(RowArgs a, Split s) {
    typedef Pack<T> P;
    const Place at = place_of<T, WAVE>(s);
    if (at.token >= a.tokens || at.col >= a.width) return;
    const Last c = last_moved<T>(at.col, a.width);
    float acc[P::N] = {};
    const int32_t* row = a.row + (uint64_t)at.token * a.topk;
    const float* weight = a.weights ? a.weights + (uint64_t)at.token * a.topk : nullptr;
    // GROUP rows at a time are asked for before any is used (a slot without a
    // row reads row 0 and adds nothing): two where latency counts (64 tokens, 8
    // rows of 7168 values, by 1 / 2 / 4 / 8: 4.1 / 3.9 / 3.7 / 3.5 us; 4096 tokens,
    // 2 rows of 2048: 9.2 / 8.9 / 10.1 / 12.9); one for the largest (8192 tokens,
    // 8 rows of 7168, by 1 / 2 / 4: 177 / 183 / 182)
    constexpr int GROUP = PAST ? 1 : 2;
    const uint32_t rows = a.capacity ? a.topk : 0;
    auto add = [&](auto count, uint32_t k0) {
        constexpr int G = decltype(count)::value;
        P x[G];
        float w[G];
        bool any[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint32_t r = (uint32_t)row[k0 + g];
            any[g] = r < a.capacity;
            w[g] = weight ? weight[k0 + g] : 1.0f;
            x[g] = load<T, PAST>(row_of<const T>(a.x, any[g] ? r : 0, a.x_stride) + c.at, c.n);
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < P::N; ++i) acc[i] = any[g] ? __builtin_fmaf(w[g], to_float(x[g].v[i]), acc[i]) : acc[i];
    };
    uint32_t k = 0;
    for (; k + GROUP <= rows; k += GROUP) add(std::integral_constant<int, GROUP>{}, k);
    if (k < rows) add(std::integral_constant<int, 1>{}, k);
    P y;
#pragma unroll
    for (int i = 0; i < P::N; ++i) y.v[i] = (T)acc[i];
    store<T, PAST>(row_of<T>(a.out, at.token, a.out_stride) + c.at, y, c.n);
}

// The gradient for G slots of a token from k0 on, by L threads.  The rows of
// all G are asked for before any is used: a load behind a branch waits for the
// one before it (one token of 8 rows of 7168 values: 13.4 us; so 7.5).  So a
// slot without a row reads dy, and its sum is dropped.
template <typename T, int L, Mode MODE, int G>
__device__ __forceinline__ void backward_group(const RowArgs& a, uint64_t t, uint32_t thread, uint32_t k0,
                                               float (*part)[8]) {
    typedef Pack<T> P;
    const T* dy = row_of<const T>(a.x, t, a.x_stride);
    const T* in[G];
    T* out[G];
    float w[G], acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint32_t k = k0 + g < a.topk ? k0 + g : a.topk - 1;
        const uint32_t r = (uint32_t)a.row[t * a.topk + k];
        const bool any = k0 + g < a.topk && r < a.capacity;
        w[g] = a.weights ? a.weights[t * a.topk + k] : 1.0f;
        acc[g] = 0.0f;
        in[g] = any && a.dweights ? row_of<const T>(a.rows, r, a.rows_stride) : dy;
        out[g] = any && a.out ? row_of<T>(a.out, r, a.out_stride) : nullptr;
    }
    if constexpr (MODE == kPastShifted) {  // no dweights
        for (uint32_t c = thread * P::N; c < a.width + 63 / sizeof(T); c += L * P::N) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const Shifted s = shifted(out[g], c, a.width);
                if (!out[g] || !s.any) continue;
                const P d = load<T, false>(dy + s.at, P::N);
                P o;
#pragma unroll
                for (int i = 0; i < P::N; ++i) o.v[i] = (T)(w[g] * to_float(d.v[i]));
                store<T, true>(out[g] + s.at, o, P::N);
            }
        }
        return;
    }
    // n values from c on, of which the first `skip` are another word's
    auto word = [&](uint32_t c, uint32_t n, uint32_t skip) {
        const P d = load<T, false>(dy + c, n);
        P x[G];
        if (a.dweights)
#pragma unroll
            for (int g = 0; g < G; ++g) x[g] = load<T, false>(in[g] + c, n);
        if (a.out)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                P o;
#pragma unroll
                for (int i = 0; i < P::N; ++i) o.v[i] = (T)(w[g] * to_float(d.v[i]));
                if (out[g]) store<T, MODE == kPast>(out[g] + c, o, n);
            }
        if (!a.dweights) return;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < P::N; ++i)
                if (i >= (int)skip) acc[g] = __builtin_fmaf(to_float(d.v[i]), to_float(x[g].v[i]), acc[g]);
    };
    if (a.width < P::N) {
        if (thread == 0) word(0, a.width, 0);
    } else {
        for (uint32_t c = thread * P::N; c < a.width; c += L * P::N) {
            // the last word is moved to the row's end, over its neighbour,
            // which stores the same there
            const uint32_t at = c + P::N <= a.width ? c : a.width - P::N;
            word(at, P::N, c - at);
        }
    }
    if (!a.dweights) return;
    float mine = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        for (int m = L < 64 ? L / 2 : 32; m; m >>= 1) acc[g] += __shfl_xor(acc[g], m);
        if ((int)thread == g) mine = acc[g];
    }
    if constexpr (L > 64) {
        if (k0) __syncthreads();  // the last group's sums have been read
        if (__lane_id() == 0)
#pragma unroll
            for (int g = 0; g < G; ++g) part[threadIdx.x >> 6][g] = acc[g];
        __syncthreads();
        if (thread < G) mine = (part[0][thread] + part[1][thread]) + (part[2][thread] + part[3][thread]);
    }
    if (thread < G && k0 + thread < a.topk) {
        const uint64_t slot = t * a.topk + k0 + thread;
        a.dweights[slot] = (uint32_t)a.row[slot] < a.capacity ? mine : 0.0f;
    }
}

// L threads per token (a workgroup or less); 8, 4 or 2 slots at a time (dy is
// read again, from the cache, for every further group).
template <typename T, int L, Mode MODE>
__global__ __launch_bounds__(256) void combine_rows_backward(RowArgs a, uint32_t pad_blocks) {
    __shared__ float part[L > 64 ? 4 : 1][8];
    if (blockIdx.x < pad_blocks) {
        zero_padding<T>(a);
        return;
    }
    const uint32_t thread = threadIdx.x % L, sub = threadIdx.x / L;
    const uint64_t t = (uint64_t)(blockIdx.x - pad_blocks) * (256 / L) + (L >= 64 ? uniform(sub) : sub);
    if (t >= a.tokens) return;  // L = 256: no workgroup
    uint32_t k = 0;
    // 16 threads a token keep the addresses of 8 slots in general registers,
    // too many (20,000 tokens, 12 rows of 100 values, without dweights: 14.6 us
    // by 8, 13.0 by 4)
    constexpr uint32_t MOST = L < 64 ? 4 : 8;
    for (; k + MOST / 2 < a.topk; k += MOST) backward_group<T, L, MODE, MOST>(a, t, thread, k, part);
    if (MOST == 8 && k + 2 < a.topk) backward_group<T, L, MODE, 4>(a, t, thread, k, part);
    else if (k < a.topk) backward_group<T, L, MODE, 2>(a, t, thread, k, part);
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
//    200 values    5.0 /  6.0 / 12
//   1001          16.1 / 15.8 / 20
//   1500          22.8 / 22.3 / 26
//   2048 (8192 tokens, 8 rows)  133 / 107 /  94
//   1001 (512 tokens)           9.9 / 6.2 / 5.4
template <typename T>
zc_status backward_as(const RowArgs& a, hipStream_t stream) {
    const uint32_t words = (a.width + Pack<T>::N - 1) / Pack<T>::N;
    if (words <= 32) return backward_by<T, 16>(a, stream);
    return words <= 192 && a.tokens > 1024 ? backward_by<T, 64>(a, stream) : backward_by<T, 256>(a, stream);
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
