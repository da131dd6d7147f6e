// zc_choose.hip -- the router: each token's choice of experts, the balance
// loss, and the gradient of both.
//
// A token belongs to L neighbouring lanes of one wave, lane l holding experts
// l * V to l * V + V - 1 in registers from the load of the logits on, so that
// they are read once: scores, the shares' sums and the choice all come from
// there.  16 experts a lane (fewer where there are few) keep the number of
// steps between lanes, which a wave waits for, at four for up to 256 experts.
//
// The choice is bound by instructions, not by memory: 65,536 tokens on 256
// experts, topk 8, take 33 us (49 with a bias), of which the logits are 7 (bf16)
// to 14 (32 bits), about 250 vector instructions a token: a third of them the
// sorted keys, a third the joins of 16 lanes' best.  Its gradient takes 25 us
// (bf16; of sigmoids 28) to 36 (32 bits), 67 to 134 MB at 2.6 to 3.8 TB/s.  Few
// tokens are bound by their chain of round trips: 8 tokens 4.7 us (7.1 with a
// bias), gradient 5.3; 8192 tokens 12 to 13 (18) and 10 to 11.
#include "zc_experts_kernels.h"

#include <type_traits>

namespace zc {

namespace {

constexpr float kInf = __builtin_inff();

// A lane's number that the compiler does not look through: what follows from it
// is made anew for every token instead of being held over the loop (16
// comparisons alone would take 32 scalar registers).
__device__ __forceinline__ uint32_t anew(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The lane d further in a group: within 16 lanes a turn of the row by DPP.
template <int D>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
    if constexpr (D < 16) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + D, 0xF, 0xF, true);
    else return __shfl_xor(v, D);
}
template <int D>
__device__ __forceinline__ float turned(float v) {
    return __uint_as_float(turned<D>(__float_as_uint(v)));
}
template <int D>
__device__ __forceinline__ double turned(double v) {
    const xu32x2 w = __builtin_bit_cast(xu32x2, v);
    return __builtin_bit_cast(double, xu32x2{turned<D>(w[0]), turned<D>(w[1])});
}
struct Best {
    double key;
    uint32_t of;
};
template <int D>
__device__ __forceinline__ Best turned(const Best& v) {
    return Best{turned<D>(v.key), turned<D>(v.of)};
}
// f over all lanes of a group, the same result in each (f commutes, and turns
// by 1, 2, 4, 8 add in the same pairs in every lane).
template <int L, int D = 1, typename T, typename F>
__device__ __forceinline__ T over_group(T v, F f) {
    if constexpr (D < L) return over_group<L, D * 2>(f(v, turned<D>(v)), f);
    else return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
    return over_group<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L, typename T>
__device__ __forceinline__ T group_sum(T v) {
    // by exchange, so that every lane adds the same pairs
#pragma unroll
    for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// The larger and the smaller of two keys, none of them NaN.
__device__ __forceinline__ double larger(double a, double b) {
#if defined(__HIP_DEVICE_COMPILE__)
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
#else
    return a > b ? a : b;
#endif
}
__device__ __forceinline__ double smaller(double a, double b) {
#if defined(__HIP_DEVICE_COMPILE__)
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
#else
    return a < b ? a : b;
#endif
}

// What LDS holds of one wave is seen by its other lanes.
__device__ __forceinline__ void wave_sees() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// e^x and 1/x in the hardware's rounding (x log2 e rounded once: |x| 2^-24 of
// the result; 1 unit in the last place).
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }
// 1/x, 0 for 0, NaN for NaN.
__device__ __forceinline__ float share_of(float x) { return x == 0.0f ? 0.0f : inverse(x); }

template <typename T, int V>
__device__ __forceinline__ void load_as(const T* row, uint32_t e0, uint32_t experts, bool whole, float (&x)[V]) {
    typedef xu32x4 __attribute__((aligned(2))) Four;
    typedef xu32x2 __attribute__((aligned(2))) Two;
    constexpr int kWord = 16 / sizeof(T), kEach = kWord < V ? kWord : V;
    const int32_t left = (int32_t)experts - (int32_t)e0;
#pragma unroll
    for (int j = 0; j < V; j += kEach) {
        T v[kWord];
        xu32x4 w{};
        if (!whole) {
            w = load_word(row + (left > j ? e0 + j : 0), left - j < kEach ? left - j : kEach);
        } else if constexpr (kEach == kWord) {
            w = *reinterpret_cast<const Four*>(row + e0 + j);
        } else {
            const xu32x2 h = *reinterpret_cast<const Two*>(row + e0 + j);
            w = xu32x4{h[0], h[1], 0, 0};
        }
        __builtin_memcpy(v, &w, 16);
#pragma unroll
        for (int q = 0; q < kEach; ++q) x[j + q] = to_float(v[q]);
    }
    if (!whole) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = j < left ? x[j] : -kInf;
    }
}

// V logits of a lane, -inf past the last expert.  whole: no lane has one.
template <int V>
__device__ __forceinline__ void load_logits(const void* logits, uint64_t at, uint32_t dtype, uint32_t e0, uint32_t experts,
                                            bool whole, float (&x)[V]) {
    if (dtype == ZC_BF16) load_as(static_cast<const __bf16*>(logits) + at, e0, experts, whole, x);
    else if (dtype == ZC_FP16) load_as(static_cast<const _Float16*>(logits) + at, e0, experts, whole, x);
    else load_as(static_cast<const float*>(logits) + at, e0, experts, whole, x);
}
__device__ __forceinline__ float one_logit(const void* logits, uint64_t at, uint32_t dtype) {
    if (dtype == ZC_BF16) return to_float(static_cast<const __bf16*>(logits)[at]);
    if (dtype == ZC_FP16) return to_float(static_cast<const _Float16*>(logits)[at]);
    return static_cast<const float*>(logits)[at];
}

// Scores of a token, all times one factor: softmax e^(x - base), base the
// largest; sigmoid e^(x - base) / (1 + e^x), base = min(largest, 0), so that the
// largest neither overflows nor underflows.  The score itself is s * back.
// Infinite or NaN logits but -inf make softmax's NaN.
__device__ __forceinline__ float sigmoid_of(float x) {
    const float t = exp_of(-fabsf(x)), down = inverse(1.0f + t);
    return (x < 0.0f ? t : 1.0f) * down;
}
// the same times e^-base, every x being below 0
__device__ __forceinline__ float low_sigmoid_of(float x, float base) { return exp_of(x - base) * inverse(1.0f + exp_of(x)); }
__device__ __forceinline__ float score_of(float x, float base, bool sigmoid) {
    return !sigmoid ? exp_of(x - base) : base < 0.0f ? low_sigmoid_of(x, base) : sigmoid_of(x);
}

__device__ __forceinline__ float base_of(float largest, bool sigmoid) {
    return largest == -kInf || (sigmoid && largest > 0.0f) ? 0.0f : largest;
}

struct Scored {
    float base, total, part, back;  // part: 1 / total
};
template <int L, int V>
__device__ __forceinline__ Scored scores(const float (&x)[V], float (&s)[V], bool sigmoid) {
    float top = -kInf;
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
    top = group_max<L>(top);
    Scored r;
    r.base = base_of(top, sigmoid);
    float sum = 0.0f;
    if (!sigmoid) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = exp_of(x[j] - r.base);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = sigmoid_of(x[j]);
        if (r.base < 0.0f) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = low_sigmoid_of(x[j], r.base);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) sum += s[j];
    r.total = group_sum<L>(sum);
    r.part = share_of(r.total);
    r.back = sigmoid ? exp_of(r.base) : r.part;
    return r;
}

// With a bias the largest logits need not be among the chosen, and the scores of
// these, relative to the largest of all, lose their digits where they are far
// below it.  Where their sum is below kFar (2^-126 is the smallest number that
// the exponential makes), they are made anew, relative to the largest chosen one.
// Returns their sum.
constexpr float kFar = 0x1p-24f;
template <int L>
__device__ __forceinline__ float among_chosen(const void* logits, uint64_t at, uint32_t dtype, const int32_t (&id)[64 / L],
                                              bool sigmoid, float (&s)[64 / L]) {
    float top = -kInf, sum = 0.0f;
#pragma unroll
    for (int h = 0; h < 64 / L; ++h) {
        s[h] = id[h] >= 0 ? one_logit(logits, at + id[h], dtype) : -kInf;
        top = fmaxf(top, s[h]);
    }
    const float base = base_of(group_max<L>(top), sigmoid);
#pragma unroll
    for (int h = 0; h < 64 / L; ++h) {
        s[h] = score_of(s[h], base, sigmoid);
        sum += s[h];
    }
    return group_sum<L>(sum);
}

// A comparison's value and its expert in one double that orders as they do,
// larger values first and lower indices first among equals: a float leaves 29
// bits of a double's mantissa free.  NaN and -inf become kClosed, or less by
// their index.
constexpr double kClosed = -0x1p128, kNone = -0x1p130;
__device__ __forceinline__ double key_of(float v, uint32_t e) {
    const double d = smaller(larger((double)(v + 0.0f), kClosed), -kClosed);  // -0 is 0
    xu32x2 w = __builtin_bit_cast(xu32x2, d);
    w[0] |= (kMaxExperts - 1 - e) ^ ((uint32_t)((int32_t)w[1] >> 31) & (kMaxExperts - 1));
    return __builtin_bit_cast(double, w);
}
__device__ __forceinline__ int32_t expert_of(double key) {
    const xu32x2 w = __builtin_bit_cast(xu32x2, key);
    const uint32_t c = (w[0] ^ (uint32_t)((int32_t)w[1] >> 31)) & (kMaxExperts - 1);
    return key <= kClosed ? -1 : (int32_t)(kMaxExperts - 1 - c);
}
__device__ __forceinline__ double value_of(double key) {
    xu32x2 w = __builtin_bit_cast(xu32x2, key);
    w[0] &= ~(kMaxExperts - 1);
    return __builtin_bit_cast(double, w);
}

__device__ __forceinline__ void order(double& a, double& b) {
    const double x = larger(a, b);
    b = smaller(a, b);
    a = x;
}
// Sorts N keys, largest first (Batcher's odd-even merges).
template <int N, int STRIDE = 1, int M>
__device__ __forceinline__ void merge(double (&k)[M], int at) {
    if constexpr (STRIDE * 2 < N) {
        merge<N, STRIDE * 2>(k, at);
        merge<N, STRIDE * 2>(k, at + STRIDE);
#pragma unroll
        for (int i = STRIDE; i + STRIDE < N; i += STRIDE * 2) order(k[at + i], k[at + i + STRIDE]);
    } else {
        order(k[at], k[at + STRIDE]);
    }
}
template <int N, int M>
__device__ __forceinline__ void sort(double (&k)[M], int at = 0) {
    if constexpr (N > 1) {
        sort<N / 2>(k, at);
        sort<N / 2>(k, at + N / 2);
        merge<N>(k, at);
    }
}

// Sorts N keys that go up and then down, or down and then up, largest first.
template <int N>
__device__ __forceinline__ void sort_bitonic(double (&k)[N]) {
#pragma unroll
    for (int d = N / 2; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!(i & d)) order(k[i], k[i + d]);
}

// The best D of a lane's V keys, largest first, kNone past the V-th.
template <int V, int D>
__device__ __forceinline__ void best_of(double (&k)[V], double (&best)[D]) {
    if constexpr (D < V) {
        static_assert(V == 2 * D, "two sorted halves");
        sort<D>(k, 0);
        sort<D>(k, D);
#pragma unroll
        for (int i = 0; i < D; ++i) best[i] = larger(k[i], k[2 * D - 1 - i]);
        sort_bitonic(best);
    } else {
        sort<V>(k);
#pragma unroll
        for (int i = 0; i < D; ++i) best[i] = i < V ? k[i < V ? i : 0] : kNone;
    }
}

// The best D of all lanes of a group, in each of them.
template <int L, int D, int STEP = 1>
__device__ __forceinline__ void best_of_group(double (&best)[D]) {
    if constexpr (STEP < L) {
        double other[D];
#pragma unroll
        for (int i = 0; i < D; ++i) other[i] = turned<STEP>(best[D - 1 - i]);
#pragma unroll
        for (int i = 0; i < D; ++i) best[i] = larger(best[i], other[i]);
        sort_bitonic(best);
        best_of_group<L, D, STEP * 2>(best);
    }
}

// Scores with a bias, compared in 64 bits one choice after the other: the way
// for the few tokens whose scores 32 bits do not tell apart and that
// in_exact_order does not take: a wave that gets here ends some 8 us later.  The
// exponentials go four by four, by way of LDS (a lane's values 256 apart): all
// side by side they would take all registers.
template <int L, int V>
__device__ __forceinline__ void choose_exactly(const ChooseArgs& a, uint64_t at, uint32_t e0, uint32_t l, double* keys,
                                               int32_t (&ids)[64 / L]) {
    float x[V];
    load_logits<V>(a.logits, at, a.dtype, e0, a.experts, a.experts == L * V, x);
    float top = -kInf;
    uint32_t open = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        top = fmaxf(top, x[j]);
        keys[j * 256] = (double)x[j];
        if (x[j] > -kInf) open |= 1u << j;  // neither closed nor NaN
    }
    top = group_max<L>(top);
    double sum = 0.0;
#pragma unroll 4
    for (int j = 0; j < V; ++j) {
        const double v = keys[j * 256], e = exp(a.sigmoid ? -v : v - (double)top), score = a.sigmoid ? 1.0 / (1.0 + e) : e;
        keys[j * 256] = score;
        sum += score;
    }
    sum = group_sum<L>(sum);
#pragma unroll 4
    for (int j = 0; j < V; ++j) {
        const double v = (a.sigmoid ? keys[j * 256] : keys[j * 256] / sum) + (e0 + j < a.experts ? (double)a.bias[e0 + j] : 0.0);
        keys[j * 256] = v;
        if (!(v > -(double)kInf)) open &= ~(1u << j);
    }
    double key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = keys[j * 256];
#pragma unroll
    for (int h = 0; h < 64 / L; ++h) ids[h] = -1;
#pragma unroll 1
    for (uint32_t k = 0; k < a.topk; ++k) {
        Best best{-(double)kInf, ~0u};
#pragma unroll
        for (int j = 0; j < V; ++j)
            if ((open >> j & 1) && key[j] > best.key) best = Best{key[j], e0 + j};
        best = over_group<L>(best, [](const Best& p, const Best& q) {
            return q.key > p.key || (q.key == p.key && q.of < p.of) ? q : p;
        });
        const uint32_t of = best.of;
        if (of - e0 < (uint32_t)V) open &= ~(1u << (of - e0));
#pragma unroll
        for (int h = 0; h < 64 / L; ++h)
            if (k == h * L + l) ids[h] = (int32_t)of;
    }
}

// The same for sigmoids, which are each by itself, where what is chosen and the
// next one are all that come into question: lane k's is `mine` (-1: none), and
// lane k gets the expert that has rank k among them.  One exponential a lane
// instead of 16 and no rounds: with a bias 8192 tokens 26.7 -> 19.1 us, 65,536
// 55 -> 47, as of both some tokens need it.
template <int L>
__device__ __forceinline__ int32_t in_exact_order(const ChooseArgs& a, uint64_t at, int32_t mine, uint32_t l, int candidates) {
    double v = -(double)kInf;
    if (mine >= 0) v = 1.0 / (1.0 + exp(-(double)one_logit(a.logits, at + mine, a.dtype))) + (double)a.bias[mine];
    uint32_t rank = 0;
#pragma unroll 1
    for (int i = 0; i < candidates; ++i) {
        const double w = __shfl(v, i, L);
        const int32_t of = __shfl(mine, i, L);
        rank += of >= 0 && (w > v || (w == v && of < mine));
    }
    int32_t id = -1;
#pragma unroll 1
    for (int i = 0; i < candidates; ++i) {
        const uint32_t of_rank = __shfl(rank, i, L);
        const int32_t of = __shfl(mine, i, L);
        if (of >= 0 && of_rank == l) id = of;
    }
    return id;
}

// Sum over a workgroup, in every thread; `shared` has room for 4.
__device__ __forceinline__ double workgroup_sum(double v, double* shared) {
    v = group_sum<64>(v);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = shared[0] + shared[1] + shared[2] + shared[3];
    __syncthreads();
    return v;
}

__device__ __forceinline__ float loss_of(const ChooseArgs& a, double dot, uint32_t live) {
    const double t = (double)live;
    return live ? (float)((double)a.balance * a.experts * dot / ((double)a.topk * t * t)) : 0.0f;
}

// Up to kFew choices are taken from the lanes' best kFew, joined pair by pair of
// lanes; more of them one after the other from all.  Without a bias there is
// nothing to do again: 92 registers instead of 168, and 8 tokens take 4.6 us, not
// 5.4, 65,536 33, not 35.
constexpr int kFew = 8;
template <int L, int V, bool MANY, bool BIASED>
__global__ __launch_bounds__(256, MANY ? 2 : BIASED ? 3 : 4) void choose(ChooseArgs a) {
    constexpr int D = MANY ? V : kFew;  // keys that a lane keeps
    constexpr uint32_t G = 256 / L;  // tokens at a time
    __shared__ double keys_in_lds[(BIASED ? 256 : 128) * V];  // choose_exactly's; at the end, the sums
    __shared__ uint32_t hist[kMaxExperts];
    __shared__ uint32_t live_tokens;
    __shared__ double shared[4];
    const uint32_t tid = threadIdx.x, l = tid % L, g = tid / L;
    for (uint32_t e = tid; e < a.experts; e += 256) hist[e] = 0;
    if (tid == 0) live_tokens = 0;
    if (blockIdx.x == 0 && tid == 0) *a.arrived = 0;
    __syncthreads();
    const bool sigmoid = a.sigmoid;
    float* const held = reinterpret_cast<float*>(keys_in_lds);
    float sums[V], bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sums[j] = 0.0f;
        bias[j] = BIASED && l * V + j < a.experts ? a.bias[l * V + j] : 0.0f;
    }
    uint32_t live = 0;
    for (uint32_t t = blockIdx.x * G + g; t < a.tokens; t += gridDim.x * G) {
        int32_t* ids = a.ids + (uint64_t)t * a.topk;
        float* weights = a.weights + (uint64_t)t * a.topk;
        if (a.mask && !a.mask[t]) {
            for (uint32_t k = l; k < a.topk; k += L) {
                ids[k] = -1;
                weights[k] = 0.0f;
            }
            continue;
        }
        live += l == 0;
        const uint64_t at = t * a.stride;
        const uint32_t e0 = anew(l * V);
        float x[V], s[V];
        load_logits<V>(a.logits, at, a.dtype, e0, a.experts, a.experts == L * V, x);
        const Scored r = scores<L, V>(x, s, sigmoid);
        double keys[V], best[D];
#pragma unroll
        for (int j = 0; j < V; ++j) sums[j] += s[j] * r.part;
        if constexpr (BIASED) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = x[j] > -kInf ? s[j] * r.back + bias[j] : -kInf;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) keys[j] = key_of(x[j], e0 + j);
        best_of<V, D>(keys, best);
        int32_t id[64 / L];
        // What two 32-bit scores have to be apart for their order to be sure, in
        // units of 2^-24: a sigmoid is off by at most 5 (its exponential by 1.5 |x|
        // + 2 of itself), a softmax by 3 and by 27 that its sum has, of what two
        // scores differ by; the sum with the bias is rounded by as many as its size.
        const double tells = sigmoid ? 0x1p-20 : 0x1p-18;
        bool unsure = false;
        auto near = [&](double before, double next) {
            const double v = value_of(next), gap = value_of(before) - v;
            return before > kClosed && !(gap > tells * (1.0 + fabs(v)));
        };
        if constexpr (!MANY) {
            best_of_group<L>(best);
            double own = kNone;
#pragma unroll
            for (int i = 0; i < D; ++i) own = (uint32_t)i == l ? best[i] : own;
            id[0] = l < a.topk ? expert_of(own) : -1;
#pragma unroll
            for (int h = 1; h < 64 / L; ++h) id[h] = -1;
            if constexpr (BIASED) {
                double past = kNone;  // the first one not among them
#pragma unroll
                for (int j = 0; j < V; ++j) past = larger(past, keys[j] < best[D - 1] ? keys[j] : kNone);
                past = over_group<L>(past, larger);
                // lane k compares choice k with the next
                double next = past;
#pragma unroll
                for (int i = 1; i < D; ++i) next = (uint32_t)i == l + 1 ? best[i] : next;
                const bool close = l < a.topk && near(own, next);
                if (close) {  // unless the two are one score: the same logit and bias
                    const int32_t e = expert_of(own), f = expert_of(next);
                    unsure = f < 0 || one_logit(a.logits, at + e, a.dtype) != one_logit(a.logits, at + f, a.dtype) || a.bias[e] != a.bias[f];
                }
                auto in_group = [](bool v) {
                    const uint64_t of_wave = __ballot(v);
                    return (L == 64 ? of_wave : of_wave >> (__lane_id() & ~(L - 1)) & ((1ull << (L & 63)) - 1)) != 0;
                };
                unsure = in_group(unsure);
                if (unsure ? sigmoid : in_group(close && l + 1 == a.topk)) {
                    // Those left out that may belong among the chosen: at least all
                    // that are near the last choice.  Where that and the next one are
                    // one score, the lower index stands first, but another one behind
                    // them may be larger than both.
                    const double last = __shfl(own, (int)a.topk - 1, L);
                    const double from = larger(last - 1.01 * tells * (1.0 + fabs(last)), kClosed);
                    uint32_t others = 0;
#pragma unroll
                    for (int j = 0; j < V; ++j) others += keys[j] < last && keys[j] > from;
                    const uint32_t all = group_sum<L>(others);
                    if (!unsure && all > 1) {  // unless they all are that one score
                        const int32_t e = expert_of(last);
                        const float its_logit = one_logit(a.logits, at + e, a.dtype), its_bias = a.bias[e];
                        uint32_t same = 0;
#pragma unroll 4
                        for (int32_t f = e0; f < (int32_t)(e0 + V); ++f)
                            same += f > e && f < (int32_t)a.experts && one_logit(a.logits, at + f, a.dtype) == its_logit && a.bias[f] == its_bias;
                        unsure = group_sum<L>(same) < all;
                    }
                    if (unsure && sigmoid && all <= 1) {
                        const int32_t of = in_exact_order<L>(a, at, l > a.topk ? -1 : expert_of(l == D ? past : own), l, (int)a.topk + 1);
                        id[0] = l < a.topk ? of : -1;
                        unsure = false;
                    }
                }
            }
        } else {
            // the group's best, again and again; the lane that had it moves up
            double before = kNone;
#pragma unroll
            for (int h = 0; h < 64 / L; ++h) {
                id[h] = -1;
                for (uint32_t q = 0; q < L && h * L + q < a.topk; ++q) {
                    const double top = over_group<L>(best[0], larger);
                    if constexpr (BIASED) unsure |= near(before, top);
                    before = top;
                    if (q == l) id[h] = expert_of(top);
                    if (best[0] == top) {
#pragma unroll
                        for (int i = 0; i + 1 < D; ++i) best[i] = best[i + 1];
                        best[D - 1] = kNone;
                    }
                }
            }
            if constexpr (BIASED) unsure |= near(before, over_group<L>(best[0], larger));  // the first one not among them
        }
        if (BIASED && unsure) choose_exactly<L, V>(a, at, e0, l, keys_in_lds + tid, id);
        float mine[64 / L], chosen = 0.0f;
#pragma unroll
        for (int h = 0; h < 64 / L; ++h) {
            mine[h] = 0.0f;
            if (h * L + l < a.topk) {
                ids[h * L + l] = id[h];
                if (id[h] >= 0) {
                    mine[h] = score_of(one_logit(a.logits, at + id[h], a.dtype), r.base, sigmoid);
                    atomicAdd(&hist[id[h]], 1u);
                }
            }
            chosen += mine[h];
        }
        float factor = a.scale * r.back;
        if (a.normalize) {
            chosen = group_sum<L>(chosen);
            if (BIASED && chosen < kFar) chosen = among_chosen<L>(a.logits, at, a.dtype, id, sigmoid, mine);
            factor = a.scale * share_of(chosen);
        }
        // a NaN among the token's logits reaches its weights wherever it was chosen
        if (r.total != r.total) factor = r.total;
#pragma unroll
        for (int h = 0; h < 64 / L; ++h)
            if (h * L + l < a.topk) weights[h * L + l] = mine[h] * factor;
    }
    __syncthreads();
    if (live) atomicAdd(&live_tokens, live);
#pragma unroll
    for (int j = 0; j < V; ++j) held[g * (L * V) + l * V + j] = sums[j];
    __syncthreads();
    const bool alone = gridDim.x == 1;  // nothing is left to add up
    double dot = 0.0;
    for (uint32_t e = tid; e < a.experts; e += 256) {
        float s = 0.0f;
        for (uint32_t q = 0; q < G; ++q) s += held[q * (L * V) + e];
        if (alone) {
            a.sums[e] = s;
            a.counts[e] = (int32_t)hist[e];
            dot += (double)s * hist[e];
        } else {
            a.part_sums[(uint64_t)blockIdx.x * a.experts + e] = s;
            a.part_counts[(uint64_t)blockIdx.x * a.experts + e] = hist[e];
        }
    }
    if (alone) {
        dot = workgroup_sum(dot, shared);
        if (tid == 0) {
            *a.counted = (int32_t)live_tokens;
            *a.loss = loss_of(a, dot, live_tokens);
        }
    } else if (tid == 0) {
        a.part_live[blockIdx.x] = live_tokens;
    }
}

// Sums of what the workgroups of `choose` left, kOf experts a workgroup, and by
// the last of them the loss.  Its time is that of one round trip to memory, as
// long as there are enough workgroups: 8192 tokens, 256 experts, 512 parts:
// with 8 experts each 6.1 us, with 16 7.3.
constexpr uint32_t kOf = 8;
__global__ __launch_bounds__(256) void finish_choice(ChooseArgs a, uint32_t parts) {
    __shared__ double sum[256], shared[4];
    __shared__ uint32_t count[256], last;
    const uint32_t c = threadIdx.x % kOf, first = threadIdx.x / kOf, e = blockIdx.x * kOf + c;
    double s = 0.0;
    uint32_t n = 0;
    if (e < a.experts) {
#pragma unroll 16
        for (uint32_t q = first; q < parts; q += 256 / kOf) {
            s += a.part_sums[(uint64_t)q * a.experts + e];
            n += a.part_counts[(uint64_t)q * a.experts + e];
        }
    }
    double live = 0.0;  // whole numbers below 2^31; every workgroup, so that the last one need not wait for them
    for (uint32_t q = threadIdx.x; q < parts; q += 256) live += a.part_live[q];
    sum[threadIdx.x] = s;
    count[threadIdx.x] = n;
    __syncthreads();
    if (threadIdx.x < 64) {  // of four parts of each sum, then of eight lanes
        for (uint32_t q = 1; q < 4; ++q) {
            s += sum[q * 64 + threadIdx.x];
            n += count[q * 64 + threadIdx.x];
        }
#pragma unroll
        for (int d = kOf; d < 64; d <<= 1) {
            s += __shfl_xor(s, d);
            n += __shfl_xor(n, d);
        }
        if (threadIdx.x < kOf && e < a.experts) {
            a.sums[e] = (float)s;
            a.counts[e] = (int32_t)n;
        }
        const double dot = group_sum<kOf>(s * n);
        if (threadIdx.x == 0) {
            __hip_atomic_store(&a.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    double dot = 0.0;
    if (threadIdx.x < gridDim.x) dot = __hip_atomic_load(&a.dots[threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    live = workgroup_sum(live, shared);
    dot = workgroup_sum(dot, shared);
    if (threadIdx.x == 0) {
        *a.counted = (int32_t)live;
        *a.loss = loss_of(a, dot, (uint32_t)live);
    }
}
static_assert(kMaxExperts / kOf <= 256, "one thread per workgroup");

template <typename T, int V>
__device__ __forceinline__ void store_as(T* p, const float (&d)[V], int32_t left) {
    constexpr int kWord = 16 / sizeof(T), kEach = kWord < V ? kWord : V;
    typedef xu32x4 __attribute__((aligned(2))) Word;
    typedef xu32x2 __attribute__((aligned(2))) Half;
    T v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = (T)d[j];
    if (left >= V) {
#pragma unroll
        for (int j = 0; j < V; j += kEach) {
            if constexpr (kEach * sizeof(T) == 16) {
                xu32x4 w;
                __builtin_memcpy(&w, v + j, 16);
                *reinterpret_cast<Word*>(p + j) = w;
            } else {
                xu32x2 w;
                __builtin_memcpy(&w, v + j, 8);
                *reinterpret_cast<Half*>(p + j) = w;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left) p[j] = v[j];
    }
}

template <int L, int V>
__global__ __launch_bounds__(256, 4) void choose_backward(ChooseGradArgs a) {
    constexpr uint32_t G = 256 / L, H = 64 / L;
    constexpr int kPitch = V + 4;  // lanes' runs begin in different banks
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ __align__(16) float held[256 * kPitch], given[256 * kPitch];  // scores; what comes by way of the weights
    const uint32_t tid = threadIdx.x, l = tid % L, g = tid / L;
    const bool sigmoid = a.sigmoid;
    auto place = [&](uint32_t id) { return (g * L + id / V) * kPitch + id % V; };
    // the loss's gradient for p, the same for every token
    float of_loss[V];
    {
        const double n = (double)*a.counted;
        const double f = n > 0.0 ? (double)a.balance * a.experts * (a.dloss ? (double)*a.dloss : 1.0) / ((double)a.topk * n * n) : 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) of_loss[j] = l * V + j < a.experts ? (float)(f * a.counts[l * V + j]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<f32x4*>(given + tid * kPitch + j) = f32x4{0, 0, 0, 0};
    for (uint32_t t = blockIdx.x * G + g; t < a.tokens; t += gridDim.x * G) {
        const uint32_t e0 = anew(l * V);
        const int32_t left = (int32_t)a.experts - (int32_t)e0;
        // all that is read of a token is asked for at once
        float x[V], s[V], d[V], dw[H];
        int32_t id[H];
        load_logits<V>(a.logits, t * a.stride, a.dtype, e0, a.experts, a.experts == L * V, x);
#pragma unroll
        for (int h = 0; h < (int)H; ++h) {
            const uint32_t k = h * L + l;
            id[h] = a.dweights && k < a.topk ? a.ids[(uint64_t)t * a.topk + k] : -1;
            dw[h] = a.dweights && k < a.topk ? a.dweights[(uint64_t)t * a.topk + k] * a.scale : 0.0f;
        }
        const bool live = !a.mask || a.mask[t];
        const Scored r = scores<L, V>(x, s, sigmoid);
#pragma unroll
        for (int j = 0; j < V; j += 4) *reinterpret_cast<f32x4*>(held + tid * kPitch + j) = f32x4{s[j], s[j + 1], s[j + 2], s[j + 3]};
        wave_sees();
        // d / d s of the chosen by way of the weights, for s as it is held here
        float chosen = 0.0f, both = 0.0f;
#pragma unroll
        for (int h = 0; h < (int)H; ++h) {
            if ((uint32_t)id[h] >= a.experts) id[h] = -1;
            if (id[h] < 0) dw[h] = 0.0f;
            if (a.normalize && id[h] >= 0) {
                const float v = held[place(id[h])];
                chosen += v;
                both += v * dw[h];
            }
        }
        bool far = false;
        if (a.normalize) {
            chosen = group_sum<L>(chosen);
            both = group_sum<L>(both);
            far = chosen < kFar;
            chosen = far ? 0.0f : share_of(chosen);
            both *= chosen;
        }
#pragma unroll
        for (int h = 0; h < (int)H; ++h)
            if (id[h] >= 0) given[place(id[h])] = a.normalize ? (dw[h] - both) * chosen : dw[h] * r.back;
        wave_sees();
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const f32x4 w = *reinterpret_cast<const f32x4*>(given + tid * kPitch + j);
#pragma unroll
            for (int q = 0; q < 4; ++q) d[j + q] = w[q];
        }
        wave_sees();
#pragma unroll
        for (int h = 0; h < (int)H; ++h)
            if (id[h] >= 0) given[place(id[h])] = 0.0f;  // as it was, for the next token
        float dot = 0.0f;
        if (sigmoid) {
#pragma unroll
            for (int j = 0; j < V; ++j) dot += of_loss[j] * s[j];
            dot = group_sum<L>(dot) * r.part;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // 1 - sigmoid(x)
                const float u = exp_of(-fabsf(x[j])), down = inverse(1.0f + u);
                d[j] = (d[j] + (of_loss[j] - dot) * r.part) * s[j] * (x[j] > 0.0f ? u * down : down);
            }
        } else {
            // d / d p: what is given is for s = p * total
#pragma unroll
            for (int j = 0; j < V; ++j) {
                d[j] = d[j] * r.total + of_loss[j];
                dot += d[j] * s[j];
            }
            dot = group_sum<L>(dot) * r.part;
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = (d[j] - dot) * (s[j] * r.part);
        }
        if (far && live && a.dweights) {  // what comes by way of the weights, times the chosen's shares
            float share[H], mean = 0.0f;
#pragma unroll
            for (int h = 0; h < (int)H; ++h) {
                const uint32_t k = h * L + l;
                id[h] = k < a.topk ? a.ids[(uint64_t)t * a.topk + k] : -1;
                if ((uint32_t)id[h] >= a.experts) id[h] = -1;
                dw[h] = id[h] >= 0 ? a.dweights[(uint64_t)t * a.topk + k] * a.scale : 0.0f;
            }
            const float sum = among_chosen<L>(a.logits, t * a.stride, a.dtype, id, sigmoid, share), part = share_of(sum);
#pragma unroll
            for (int h = 0; h < (int)H; ++h) {
                share[h] *= part;
                mean += share[h] * dw[h];
            }
            mean = group_sum<L>(mean);
#pragma unroll
            for (int h = 0; h < (int)H; ++h)
                if (id[h] >= 0) given[place(id[h])] = (dw[h] - mean) * share[h];
            wave_sees();
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = exp_of(-fabsf(x[j])), down = inverse(1.0f + u);
                d[j] += given[tid * kPitch + j] * (!sigmoid ? 1.0f : x[j] > 0.0f ? u * down : down);
                given[tid * kPitch + j] = 0.0f;
            }
            wave_sees();
        }
        if (!live) {
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = 0.0f;
        }
        const uint64_t out = t * a.out_stride + e0;
        if (a.dtype == ZC_BF16) store_as(static_cast<__bf16*>(a.dlogits) + out, d, left);
        else if (a.dtype == ZC_FP16) store_as(static_cast<_Float16*>(a.dlogits) + out, d, left);
        else store_as(static_cast<float*>(a.dlogits) + out, d, left);
    }
}

// Workgroups of a choice, and of its gradient: what the CUs hold at once, which go
// on to the next tokens.  65,536 tokens on 256 experts, in us: choices in 768 / 1024
// / 1280 workgroups 33/31/33, with a bias 49/51/53 (8192 tokens on 1024 experts with
// a bias 35/42/42); gradients in 1024 / 2048 / 4096 25/32/42.  More of them for a
// choice where a lane would add up more than kInLane tokens' shares, which are
// summed in 32 bits there and in 64 from workgroup to workgroup; at most
// kMostParts, which one launch may have (up to 2^29 tokens with kInLane a lane:
// past that they would have more logits than memory holds).
constexpr uint32_t kParts = 768, kBackward = 1024, kInLane = 16, kMostParts = 1u << 23;

uint32_t tokens_at_a_time(uint32_t experts) { return experts <= 256 ? 16 : experts <= 512 ? 8 : 4; }

// f(L, V) for a number of experts.
template <typename F>
void with_shape(uint32_t experts, F f) {
    if (experts <= 64) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
    else if (experts <= 128) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
    else if (experts <= 256) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
    else if (experts <= 512) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
    else f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

}  // namespace

uint32_t choose_parts(uint64_t tokens, uint32_t experts) {
    const uint32_t g = tokens_at_a_time(experts);
    const uint64_t n = (tokens + g - 1) / g;
    const uint64_t most = (n + kInLane - 1) / kInLane;
    return n < 1 ? 1 : n <= kParts ? (uint32_t)n : most <= kParts ? kParts : most < kMostParts ? (uint32_t)most : kMostParts;
}

zc_status launch_choose(const ChooseArgs& a, hipStream_t stream) {
    const uint32_t parts = choose_parts(a.tokens, a.experts);
    with_shape(a.experts, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        auto launch = [&](auto many, auto biased) {
            hipLaunchKernelGGL((choose<L, V, decltype(many)::value, decltype(biased)::value>), dim3(parts), dim3(256), 0, stream, a);
        };
        const std::true_type yes;
        const std::false_type no;
        if (a.topk <= kFew) a.bias ? launch(no, yes) : launch(no, no);
        else a.bias ? launch(yes, yes) : launch(yes, no);
    });
    if (parts > 1) hipLaunchKernelGGL(finish_choice, dim3((a.experts + kOf - 1) / kOf), dim3(256), 0, stream, a, parts);
    return ZC_OK;
}

zc_status launch_choose_backward(const ChooseGradArgs& a, hipStream_t stream) {
    const uint32_t g = tokens_at_a_time(a.experts), n = (a.tokens + g - 1) / g;
    with_shape(a.experts, [&](auto l, auto v) {
        hipLaunchKernelGGL((choose_backward<decltype(l)::value, decltype(v)::value>), dim3(n < kBackward ? n : kBackward), dim3(256), 0, stream, a);
    });
    return ZC_OK;
}

}  // namespace zc
