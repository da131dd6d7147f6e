// zc_choose.hip -- the router: each token's choice of experts, the balance
// loss, and the gradient of both.
#include "zc_experts_kernels.h"

#include <type_traits>

namespace zc {

namespace {

constexpr float kInf = __builtin_inff();

// A token belongs to L neighbouring lanes of one wave, lane l holding experts
// l * V to l * V + V - 1.
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int d = 1; d < L; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// What LDS holds of one wave is seen by its other lanes.
__device__ __forceinline__ void wave_sees() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// V logits of a lane, -inf past the last expert.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, uint32_t e0, uint32_t experts, float (&x)[V]) {
    constexpr int kEach = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
#pragma unroll
    for (int j = 0; j < V; j += kEach) {
        const int32_t left = (int32_t)experts - (int32_t)(e0 + j);
        T v[16 / sizeof(T)];
        const xu32x4 w = load_word(row + (left > 0 ? e0 + j : 0), left < kEach ? left : 16 / (int32_t)sizeof(T) > kEach ? kEach : left);
        __builtin_memcpy(v, &w, 16);
#pragma unroll
        for (int q = 0; q < kEach; ++q) x[j + q] = q < left ? to_float(v[q]) : -kInf;
    }
}

// Scores of a token, all times one factor: softmax e^(x - max), sigmoid
// e^(x - low) / (1 + e^x) with low = min(max, 0), so that the largest neither
// overflows nor underflows; the score itself is s * back.  Infinite or NaN
// logits but -inf make them NaN.
template <int V, int L, bool SIGMOID>
__device__ __forceinline__ float scores(const float (&x)[V], float (&s)[V], float& total) {
    float top = -kInf;
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
    top = group_max<L>(top);
    float sum = 0.0f, low = 0.0f;
    if (SIGMOID) {
        low = top < 0.0f && top > -kInf ? top : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = low < 0.0f ? expf(x[j] - low) / (1.0f + expf(x[j])) : 1.0f / (1.0f + expf(-x[j]));
            sum += s[j];
        }
    } else {
        const float m = top == -kInf ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = expf(x[j] - m);
            sum += s[j];
        }
    }
    total = group_sum<L>(sum);
    return SIGMOID ? expf(low) : total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
}

template <typename T, int L, int V, bool SIGMOID>
__global__ __launch_bounds__(256) void choose(ChooseArgs a) {
    constexpr uint32_t G = 256 / L;  // tokens at a time
    constexpr int kPitch = V + 4;
    __shared__ __align__(16) float held[256 * kPitch];  // scores by lane; sums at the end
    __shared__ uint32_t hist[kMaxExperts];
    __shared__ uint32_t live_tokens;
    const uint32_t tid = threadIdx.x, l = tid % L, g = tid / L, e0 = l * V;
    for (uint32_t e = tid; e < a.experts; e += 256) hist[e] = 0;
    if (tid == 0) live_tokens = 0;
    if (blockIdx.x == 0 && tid == 0) *a.arrived = 0;
    __syncthreads();
    float sums[V], bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sums[j] = 0.0f;
        bias[j] = a.bias && e0 + j < a.experts ? a.bias[e0 + j] : 0.0f;
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
        float x[V], s[V], total;
        load_logits<T, V>(static_cast<const T*>(a.logits) + t * a.stride, e0, a.experts, x);
        const float back = scores<V, L, SIGMOID>(x, s, total);
        const float part = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sums[j] += s[j] * part;
            held[tid * kPitch + j] = s[j];
        }
        // what is compared, in 64 bits
        double key[V];
        float top = -kInf;
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
            top = group_max<L>(top);
            double sum = 0.0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                key[j] = SIGMOID ? 1.0 / (1.0 + exp(-(double)x[j])) : exp((double)x[j] - (double)top);
                sum += key[j];
            }
#pragma unroll
            for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d);
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = (SIGMOID ? key[j] : key[j] / sum) + (double)bias[j];
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = (double)x[j];
        }
        uint32_t open = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (x[j] > -kInf && key[j] > -(double)kInf) open |= 1u << j;  // neither closed nor NaN
        wave_sees();
        float mine[64 / L], chosen = 0.0f;
#pragma unroll
        for (int h = 0; h < 64 / L; ++h) {
            mine[h] = 0.0f;
            if (h * L >= (int)a.topk) break;
            int32_t id = -1;
            for (uint32_t r = 0; r < L && h * L + r < a.topk; ++r) {
                double best = 0.0;
                uint32_t at = ~0u;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if ((open >> j & 1) && (at == ~0u || key[j] > best)) {
                        best = key[j];
                        at = e0 + j;
                    }
#pragma unroll
                for (int d = 1; d < L; d <<= 1) {
                    const double other = __shfl_xor(best, d);
                    const uint32_t oat = __shfl_xor(at, d);
                    if (oat != ~0u && (at == ~0u || other > best || (other == best && oat < at))) {
                        best = other;
                        at = oat;
                    }
                }
                if (at - e0 < (uint32_t)V) open &= ~(1u << (at - e0));
                if (r == l) id = (int32_t)at;
            }
            if (h * L + l < a.topk) {
                ids[h * L + l] = id;
                if (id >= 0) {
                    mine[h] = held[((g * L) + id / V) * kPitch + id % V];
                    atomicAdd(&hist[id], 1u);
                }
            }
            chosen += mine[h];
        }
        chosen = group_sum<L>(chosen);
        // a NaN among the token's logits reaches its weights wherever it was chosen
        const float factor = total != total ? total : a.normalize ? (chosen > 0.0f ? a.scale / chosen : chosen == 0.0f ? 0.0f : chosen) : a.scale * back;
#pragma unroll
        for (int h = 0; h < 64 / L; ++h)
            if (h * L + l < a.topk) weights[h * L + l] = mine[h] * factor;
        wave_sees();
    }
    __syncthreads();
    if (live) atomicAdd(&live_tokens, live);
#pragma unroll
    for (int j = 0; j < V; ++j) held[g * (L * V) + e0 + j] = sums[j];
    __syncthreads();
    for (uint32_t e = tid; e < a.experts; e += 256) {
        float s = 0.0f;
        for (uint32_t q = 0; q < G; ++q) s += held[q * (L * V) + e];
        a.part_sums[(uint64_t)blockIdx.x * a.experts + e] = s;
        a.part_counts[(uint64_t)blockIdx.x * a.experts + e] = hist[e];
    }
    if (tid == 0) a.part_live[blockIdx.x] = live_tokens;
}

// Sums of what the workgroups of `choose` left, 16 experts a workgroup, and by
// the last of them the loss.
__global__ __launch_bounds__(256) void finish_choice(ChooseArgs a, uint32_t parts) {
    __shared__ double sum[256];
    __shared__ uint32_t count[256], last;
    const uint32_t c = threadIdx.x & 15, first = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
    double s = 0.0;
    uint32_t n = 0;
    if (e < a.experts)
        for (uint32_t q = first; q < parts; q += 16) {
            s += a.part_sums[(uint64_t)q * a.experts + e];
            n += a.part_counts[(uint64_t)q * a.experts + e];
        }
    sum[threadIdx.x] = s;
    count[threadIdx.x] = n;
    __syncthreads();
    if (threadIdx.x < 16) {
        for (uint32_t q = 1; q < 16; ++q) {
            s += sum[q * 16 + c];
            n += count[q * 16 + c];
        }
        if (e < a.experts) {
            a.sums[e] = (float)s;
            a.counts[e] = (int32_t)n;
        }
        double dot = s * n;
        for (int d = 1; d < 16; d <<= 1) dot += __shfl_xor(dot, d);
        if (threadIdx.x == 0) {
            __hip_atomic_store(&a.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    uint32_t live = 0;
    for (uint32_t q = threadIdx.x; q < parts; q += 256) live += a.part_live[q];
    count[threadIdx.x] = live;
    __syncthreads();
    if (threadIdx.x == 0) {
        double dot = 0.0;
        for (uint32_t q = 0; q < gridDim.x; ++q) dot += __hip_atomic_load(&a.dots[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        live = 0;
        for (uint32_t q = 0; q < 256; ++q) live += count[q];
        *a.counted = (int32_t)live;
        const double t = (double)live;
        *a.loss = live ? (float)((double)a.balance * a.experts * dot / ((double)a.topk * t * t)) : 0.0f;
    }
}

template <typename T, int L, int V, bool SIGMOID>
__global__ __launch_bounds__(256) void choose_backward(ChooseGradArgs a) {
    constexpr uint32_t G = 256 / L;
    constexpr int kPitch = V + 4;
    __shared__ __align__(16) float held[256 * kPitch];
    const uint32_t tid = threadIdx.x, l = tid % L, g = tid / L, e0 = l * V;
    // the loss's gradient for p, the same for every token
    float of_loss[V];
    {
        const double n = (double)*a.counted;
        const double f = n > 0.0 ? (double)a.balance * a.experts * (a.dloss ? (double)*a.dloss : 1.0) / ((double)a.topk * n * n) : 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) of_loss[j] = e0 + j < a.experts ? (float)(f * a.counts[e0 + j]) : 0.0f;
    }
    for (uint32_t t = blockIdx.x * G + g; t < a.tokens; t += gridDim.x * G) {
        T* out = static_cast<T*>(a.dlogits) + t * a.out_stride;
        float d[V];
        if (a.mask && !a.mask[t]) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e0 + j < a.experts) out[e0 + j] = (T)0.0f;
            continue;
        }
        const T* row = static_cast<const T*>(a.logits) + t * a.stride;
        float x[V], s[V], total;
        load_logits<T, V>(row, e0, a.experts, x);
        const float back = scores<V, L, SIGMOID>(x, s, total);
#pragma unroll
        for (int j = 0; j < V; ++j) held[tid * kPitch + j] = s[j];
        wave_sees();
        // the chosen: scores, and the weights' gradient
        float mine[64 / L], dw[64 / L], chosen = 0.0f, both = 0.0f;
        int32_t id[64 / L];
#pragma unroll
        for (int h = 0; h < 64 / L; ++h) {
            const uint32_t k = h * L + l;
            id[h] = a.dweights && k < a.topk ? a.ids[(uint64_t)t * a.topk + k] : -1;
            if ((uint32_t)id[h] >= a.experts) id[h] = -1;
            mine[h] = id[h] >= 0 ? held[((g * L) + id[h] / V) * kPitch + id[h] % V] : 0.0f;
            dw[h] = id[h] >= 0 ? a.dweights[(uint64_t)t * a.topk + k] * a.scale : 0.0f;
            chosen += mine[h];
            both += mine[h] * dw[h];
        }
        wave_sees();
        chosen = group_sum<L>(chosen);
        both = group_sum<L>(both);
#pragma unroll
        for (int j = 0; j < V; ++j) held[tid * kPitch + j] = 0.0f;
        wave_sees();
        // by way of the weights, for s as it is held here
        const float inv = chosen > 0.0f ? 1.0f / chosen : chosen == 0.0f ? 0.0f : chosen;
#pragma unroll
        for (int h = 0; h < 64 / L; ++h)
            if (id[h] >= 0) held[((g * L) + id[h] / V) * kPitch + id[h] % V] = a.normalize ? (dw[h] - both * inv) * inv : dw[h] * back;
        wave_sees();
        const float part = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
        float dot = 0.0f;
        if (SIGMOID) {
#pragma unroll
            for (int j = 0; j < V; ++j) dot += of_loss[j] * s[j];
            dot = group_sum<L>(dot) * part;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float up = held[tid * kPitch + j] + (of_loss[j] - dot) * part;
                d[j] = up * s[j] * (1.0f / (1.0f + expf(x[j])));
            }
        } else {
            // d / d p: what is held is for s = p * total
#pragma unroll
            for (int j = 0; j < V; ++j) {
                d[j] = held[tid * kPitch + j] * total + of_loss[j];
                dot += d[j] * s[j];
            }
            dot = group_sum<L>(dot) * part;
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = (d[j] - dot) * (s[j] * part);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < a.experts) out[e0 + j] = (T)d[j];
        wave_sees();
    }
}

constexpr uint32_t kParts = 512;  // workgroups of a choice, at most

uint32_t tokens_at_a_time(uint32_t experts) { return experts <= 256 ? 16 : experts <= 512 ? 8 : 4; }

// f(T, L, V, SIGMOID) for what a call asks for.
template <typename F>
void with_shape(uint32_t dtype, uint32_t experts, bool sigmoid, F f) {
    auto by_score = [&](auto t, auto l, auto v) {
        if (sigmoid) f(t, l, v, std::true_type{});
        else f(t, l, v, std::false_type{});
    };
    auto by_experts = [&](auto t) {
        if (experts <= 64) by_score(t, std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
        else if (experts <= 128) by_score(t, std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
        else if (experts <= 256) by_score(t, std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
        else if (experts <= 512) by_score(t, std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
        else by_score(t, std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
    };
    if (dtype == ZC_BF16) by_experts((__bf16)0.0f);
    else if (dtype == ZC_FP16) by_experts((_Float16)0.0f);
    else by_experts(0.0f);
}

}  // namespace

uint32_t choose_parts(uint64_t tokens, uint32_t experts) {
    const uint32_t g = tokens_at_a_time(experts);
    const uint64_t n = (tokens + g - 1) / g;
    return n < 1 ? 1 : n > kParts ? kParts : (uint32_t)n;
}

zc_status launch_choose(const ChooseArgs& a, uint32_t dtype, bool sigmoid, hipStream_t stream) {
    const uint32_t parts = choose_parts(a.tokens, a.experts);
    with_shape(dtype, a.experts, sigmoid, [&](auto t, auto l, auto v, auto score) {
        hipLaunchKernelGGL((choose<decltype(t), l.value, v.value, score.value>), dim3(parts), dim3(256), 0, stream, a);
    });
    hipLaunchKernelGGL(finish_choice, dim3((a.experts + 15) / 16), dim3(256), 0, stream, a, parts);
    return ZC_OK;
}

zc_status launch_choose_backward(const ChooseGradArgs& a, uint32_t dtype, bool sigmoid, hipStream_t stream) {
    const uint32_t g = tokens_at_a_time(a.experts), n = (a.tokens + g - 1) / g;
    with_shape(dtype, a.experts, sigmoid, [&](auto t, auto l, auto v, auto score) {
        hipLaunchKernelGGL((choose_backward<decltype(t), l.value, v.value, score.value>), dim3(n < 4096 ? n : 4096), dim3(256), 0,
                           stream, a);
    });
    return ZC_OK;
}

}  // namespace zc
