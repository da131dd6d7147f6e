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
#include "zc_experts_kernels.h"

namespace zc {

namespace {

// Threads of a workgroup: tx columns (in words) by 256 / tx tokens, tx a
// power of two.  From 64 columns on a wave has one token, whose rows and
// weights are then scalar loads.
struct Split {
    uint32_t log_tx;
    uint32_t words;         // words per row
    uint32_t token_blocks;  // workgroups along x before those of the padding rows
};

template <bool WAVE>
__device__ __forceinline__ uint32_t token_of(const Split& s) {
    const uint32_t ty = threadIdx.x >> s.log_tx;
    return blockIdx.x * (256u >> s.log_tx) + (WAVE ? uniform(ty) : ty);
}

// Zeros in the padding rows of expert e.  A workgroup per (expert, column
// block), as the launch's last workgroups.
template <typename W>
__device__ __forceinline__ void zero_padding(const RowArgs& a, const Split& s, uint32_t e, int unroll) {
    const uint32_t tx = 1u << s.log_tx, ty = threadIdx.x >> s.log_tx, nty = 256u >> s.log_tx;
    const uint32_t lo = (uint32_t)a.offsets[e] + (uint32_t)a.counts[e];
    uint32_t hi = (uint32_t)a.offsets[e + 1];
    hi = hi < a.capacity ? hi : a.capacity;
    for (uint32_t r = lo + ty; r < hi; r += nty) {
        W* out = reinterpret_cast<W*>(static_cast<uint8_t*>(a.out) + r * a.out_stride);
        for (int u = 0; u < unroll; ++u) {
            const uint32_t j = (blockIdx.y * unroll + u) * tx + (threadIdx.x & (tx - 1));
            if (j < s.words) out[j] = W{};
        }
    }
}

template <int VB, int U, bool WAVE>
__global__ __launch_bounds__(256) void dispatch_rows(RowArgs a, Split s) {
    typedef typename Word<VB>::type W;
    if (blockIdx.x >= s.token_blocks) {
        zero_padding<W>(a, s, blockIdx.x - s.token_blocks, U);
        return;
    }
    const uint32_t t = token_of<WAVE>(s), tx = 1u << s.log_tx;
    if (t >= a.tokens) return;
    const W* x = reinterpret_cast<const W*>(static_cast<const uint8_t*>(a.x) + t * a.x_stride);
    const uint32_t j0 = blockIdx.y * U * tx + (threadIdx.x & (tx - 1));
    W v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (j0 + u * tx < s.words) v[u] = x[j0 + u * tx];
    const int32_t* row = a.row + (uint64_t)t * a.topk;
    for (uint32_t k = 0; k < a.topk; ++k) {
        const uint32_t r = (uint32_t)row[k];
        if (r >= a.capacity) continue;
        W* out = reinterpret_cast<W*>(static_cast<uint8_t*>(a.out) + r * a.out_stride);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j0 + u * tx < s.words) out[j0 + u * tx] = v[u];
    }
}

template <typename T, int VB>
struct Pack {
    static constexpr int N = VB / (int)sizeof(T);
    typedef typename Word<VB>::type W;
    union {
        W w;
        T v[N];
    };
};

template <typename T, int VB, int U, bool WAVE>
__global__ __launch_bounds__(256) void combine_rows(RowArgs a, Split s) {
    typedef Pack<T, VB> P;
    const uint32_t t = token_of<WAVE>(s), tx = 1u << s.log_tx;
    if (t >= a.tokens) return;
    const uint32_t j0 = blockIdx.y * U * tx + (threadIdx.x & (tx - 1));
    float acc[U][P::N] = {};
    const int32_t* row = a.row + (uint64_t)t * a.topk;
    const float* weight = a.weights ? a.weights + (uint64_t)t * a.topk : nullptr;
#pragma unroll 4
    for (uint32_t k = 0; k < a.topk; ++k) {
        const uint32_t r = (uint32_t)row[k];
        if (r >= a.capacity) continue;
        const float w = weight ? weight[k] : 1.0f;
        const typename P::W* x =
            reinterpret_cast<const typename P::W*>(static_cast<const uint8_t*>(a.x) + r * a.x_stride);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j0 + u * tx < s.words) {
                P p;
                p.w = x[j0 + u * tx];
#pragma unroll
                for (int i = 0; i < P::N; ++i) acc[u][i] = __builtin_fmaf(w, to_float(p.v[i]), acc[u][i]);
            }
    }
    typename P::W* y = reinterpret_cast<typename P::W*>(static_cast<uint8_t*>(a.out) + t * a.out_stride);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (j0 + u * tx < s.words) {
            P p;
#pragma unroll
            for (int i = 0; i < P::N; ++i) p.v[i] = (T)acc[u][i];
            y[j0 + u * tx] = p.w;
        }
}

// One workgroup per token; kGroup slots at a time (dy is read again, from
// the cache, for every further group).
constexpr int kGroup = 8;

template <typename T, int VB>
__global__ __launch_bounds__(256) void combine_rows_backward(RowArgs a, Split s) {
    typedef Pack<T, VB> P;
    typedef typename P::W W;
    __shared__ float part[4][kGroup];
    if (blockIdx.x >= s.token_blocks) {
        for (uint32_t y = 0; y * 256 < s.words; ++y) {
            const uint32_t e = blockIdx.x - s.token_blocks;
            const uint32_t lo = (uint32_t)a.offsets[e] + (uint32_t)a.counts[e];
            uint32_t hi = (uint32_t)a.offsets[e + 1];
            hi = hi < a.capacity ? hi : a.capacity;
            const uint32_t j = y * 256 + threadIdx.x;
            if (j < s.words)
                for (uint32_t r = lo; r < hi; ++r)
                    reinterpret_cast<W*>(static_cast<uint8_t*>(a.out) + r * a.out_stride)[j] = W{};
        }
        return;
    }
    const uint64_t t = blockIdx.x;
    const W* dy = reinterpret_cast<const W*>(static_cast<const uint8_t*>(a.x) + t * a.x_stride);
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
        for (uint32_t j = threadIdx.x; j < s.words; j += 256) {
            P d;
            d.w = dy[j];
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                if (r[g] >= a.capacity) continue;
                if (a.dweights) {
                    P x;
                    x.w = reinterpret_cast<const W*>(static_cast<const uint8_t*>(a.rows) + r[g] * a.rows_stride)[j];
#pragma unroll
                    for (int i = 0; i < P::N; ++i)
                        acc[g] = __builtin_fmaf(to_float(d.v[i]), to_float(x.v[i]), acc[g]);
                }
                if (a.out) {
                    P o;
#pragma unroll
                    for (int i = 0; i < P::N; ++i) o.v[i] = (T)(w[g] * to_float(d.v[i]));
                    reinterpret_cast<W*>(static_cast<uint8_t*>(a.out) + r[g] * a.out_stride)[j] = o.w;
                }
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
            for (int m = 32; m; m >>= 1) acc[g] += __shfl_xor(acc[g], m);
        if (k0) __syncthreads();  // the last group's sums have been read
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int g = 0; g < kGroup; ++g) part[threadIdx.x >> 6][g] = acc[g];
        __syncthreads();
        const uint32_t k = k0 + threadIdx.x;
        if (threadIdx.x < kGroup && k < a.topk)
            a.dweights[t * a.topk + k] = (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                                         (part[2][threadIdx.x] + part[3][threadIdx.x]);
    }
}

// Widest word (16, 8, 4 or 2 bytes) that every row start and the row width
// are multiples of.
uint32_t word_bytes(uint64_t bits) {
    return bits & 15 ? bits & 7 ? bits & 3 ? 2 : 4 : 8 : 16;
}

uint64_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

Split split(uint32_t words, uint32_t tokens, uint32_t unroll) {
    // the widest tx that leaves the fewest threads without a word
    uint32_t best = 3, waste = ~0u;
    for (uint32_t lt = 3; lt <= 8; ++lt) {
        const uint32_t w = up_to(words, unroll << lt) - words;
        if (w <= waste) {
            best = lt;
            waste = w;
        }
    }
    const uint32_t ty = 256u >> best;
    return Split{best, words, (tokens + ty - 1) / ty};
}

template <int VB, int U>
void dispatch_as(const RowArgs& a, uint32_t bytes, hipStream_t stream) {
    const Split s = split(bytes / VB, a.tokens, U);
    const dim3 grid(s.token_blocks + a.experts, (s.words + (U << s.log_tx) - 1) / (U << s.log_tx));
    if (s.log_tx >= 6) hipLaunchKernelGGL((dispatch_rows<VB, U, true>), grid, dim3(256), 0, stream, a, s);
    else hipLaunchKernelGGL((dispatch_rows<VB, U, false>), grid, dim3(256), 0, stream, a, s);
}

template <typename T, int VB, int U>
void combine_as(const RowArgs& a, hipStream_t stream) {
    const Split s = split(a.width * (uint32_t)sizeof(T) / VB, a.tokens, U);
    const dim3 grid(s.token_blocks, (s.words + (U << s.log_tx) - 1) / (U << s.log_tx));
    if (s.log_tx >= 6) hipLaunchKernelGGL((combine_rows<T, VB, U, true>), grid, dim3(256), 0, stream, a, s);
    else hipLaunchKernelGGL((combine_rows<T, VB, U, false>), grid, dim3(256), 0, stream, a, s);
}

template <typename T>
void combine_type(const RowArgs& a, hipStream_t stream) {
    const uint64_t bits = addr(a.x) | addr(a.out) | a.x_stride | a.out_stride | (a.width * sizeof(T));
    switch (word_bytes(bits)) {
        case 16: combine_as<T, 16, 1>(a, stream); break;
        case 8: combine_as<T, 8, 2>(a, stream); break;
        case 4: combine_as<T, 4, 4>(a, stream); break;
        default:
            if constexpr (sizeof(T) == 2) combine_as<T, 2, 4>(a, stream);
    }
}

template <typename T, int VB>
void backward_as(const RowArgs& a, hipStream_t stream) {
    const Split s{8, a.width * (uint32_t)sizeof(T) / VB, a.tokens};
    const dim3 grid(a.tokens + (a.out ? a.experts : 0));
    hipLaunchKernelGGL((combine_rows_backward<T, VB>), grid, dim3(256), 0, stream, a, s);
}

template <typename T>
void backward_type(const RowArgs& a, hipStream_t stream) {
    uint64_t bits = addr(a.x) | a.x_stride | (a.width * sizeof(T));
    if (a.out) bits |= addr(a.out) | a.out_stride;
    if (a.dweights) bits |= addr(a.rows) | a.rows_stride;
    switch (word_bytes(bits)) {
        case 16: backward_as<T, 16>(a, stream); break;
        case 8: backward_as<T, 8>(a, stream); break;
        case 4: backward_as<T, 4>(a, stream); break;
        default:
            if constexpr (sizeof(T) == 2) backward_as<T, 2>(a, stream);
    }
}

}  // namespace

void launch_dispatch(const RowArgs& a, uint32_t elem_bytes, hipStream_t stream) {
    const uint32_t bytes = a.width * elem_bytes;
    switch (word_bytes(addr(a.x) | addr(a.out) | a.x_stride | a.out_stride | bytes)) {
        case 16: dispatch_as<16, 1>(a, bytes, stream); break;
        case 8: dispatch_as<8, 2>(a, bytes, stream); break;
        case 4: dispatch_as<4, 4>(a, bytes, stream); break;
        default: dispatch_as<2, 4>(a, bytes, stream); break;
    }
}

void launch_combine(const RowArgs& a, uint32_t dtype, hipStream_t stream) {
    if (dtype == ZC_BF16) combine_type<__bf16>(a, stream);
    else if (dtype == ZC_FP16) combine_type<_Float16>(a, stream);
    else combine_type<float>(a, stream);
}

void launch_combine_backward(const RowArgs& a, uint32_t dtype, hipStream_t stream) {
    if (dtype == ZC_BF16) backward_type<__bf16>(a, stream);
    else if (dtype == ZC_FP16) backward_type<_Float16>(a, stream);
    else backward_type<float>(a, stream);
}

}  // namespace zc
