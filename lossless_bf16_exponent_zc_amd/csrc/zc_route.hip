// zc_route.hip -- slots sorted by expert: a stable counting sort.
//
//   row_i = offset_(id_i) + #{ j < i : id_j = id_i },
//   offset_e = sum over f < e of up(c_f, align).
//
// The rank inside an expert is counted, not sorted: a wave takes 64 slots in
// order, finds the lanes with its own expert by one ballot per bit of the id
// (log2(experts + 1) of them), and keeps a running count per expert in LDS
// that only it advances, so the order of rows does not depend on timing.
//
// Up to kSmall slots one workgroup does everything in one launch; above,
// three launches: counts per tile, a scan of each expert's tiles, ranks.
#include "zc_experts_kernels.h"

namespace zc {

namespace {

constexpr uint32_t kTile = 1024;     // slots per workgroup of the large form
constexpr uint32_t kSmall = 8192;    // slots of the one-launch form

// Lanes whose key equals the caller's.
__device__ __forceinline__ uint64_t same_key(uint32_t key, uint32_t bits) {
    uint64_t m = ~0ull;
    for (uint32_t b = 0; b < bits; ++b) {
        const uint64_t v = __ballot((key >> b) & 1u);
        m &= (key >> b) & 1u ? v : ~v;
    }
    return m;
}

__device__ __forceinline__ uint32_t key_bits(uint32_t experts) { return 32u - __clz(experts); }

// Exclusive sum over the workgroup of one value per thread; `total` gets the
// whole.  part: one word per wave.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* part, uint32_t nwaves, uint32_t& total) {
    const uint32_t lane = __lane_id(), wave = threadIdx.x >> 6;
    uint32_t s = v;
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t t = __shfl_up(s, d);
        if (lane >= d) s += t;
    }
    if (lane == 63) part[wave] = s;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (uint32_t w = 0; w < nwaves; ++w) {
        before += w < wave ? part[w] : 0u;
        all += part[w];
    }
    __syncthreads();
    total = all;
    return before + s - v;
}

// Slots [lo, hi) of one wave, in order: their rows from the wave's running
// counts `next` (the row of each expert's next slot).
__device__ __forceinline__ void place(const RouteArgs& a, uint32_t lo, uint32_t hi, uint32_t* next) {
    const uint32_t lane = __lane_id(), bits = key_bits(a.experts);
    for (uint32_t i0 = lo; i0 < hi; i0 += 64) {
        const uint32_t i = i0 + lane;
        uint32_t key = a.experts;
        if (i < hi) {
            const uint32_t id = (uint32_t)a.ids[i];
            if (id < a.experts) key = id;
        }
        const uint64_t m = same_key(key, bits);
        const uint32_t first = __ffsll((unsigned long long)m) - 1;
        uint32_t base = 0;
        if (lane == first && key < a.experts) base = atomicAdd(&next[key], (uint32_t)__popcll(m));
        base = __shfl(base, first);
        if (i < hi) {
            const uint32_t r = base + __popcll(m & ((1ull << lane) - 1));
            a.row[i] = key < a.experts ? (int32_t)r : -1;
            if (key < a.experts) a.slot[r] = (int32_t)i;
        }
    }
}

__device__ __forceinline__ void count(const RouteArgs& a, uint32_t lo, uint32_t hi, uint32_t* cnt) {
    for (uint32_t i = lo + __lane_id(); i < hi; i += 64) {
        const uint32_t id = (uint32_t)a.ids[i];
        if (id < a.experts) atomicAdd(&cnt[id], 1u);
    }
}

// One workgroup of 1024 threads.  LDS: [waves][experts] counts.
__global__ __launch_bounds__(1024) void route_small(RouteArgs a, uint32_t nwaves) {
    extern __shared__ uint32_t cnt[];
    __shared__ uint32_t part[16];
    const uint32_t tid = threadIdx.x, wave = uniform(tid >> 6);
    for (uint32_t i = tid; i < nwaves * a.experts; i += 1024) cnt[i] = 0;
    __syncthreads();
    const uint32_t each = up_to((a.nslots + nwaves - 1) / nwaves, 64);
    const uint32_t lo = wave * each < a.nslots ? wave * each : a.nslots;
    const uint32_t hi = lo + each < a.nslots ? lo + each : a.nslots;
    uint32_t* mine = cnt + wave * a.experts;
    if (wave < nwaves) count(a, lo, hi, mine);
    __syncthreads();
    uint32_t c = 0;
    if (tid < a.experts)
        for (uint32_t w = 0; w < nwaves; ++w) {
            const uint32_t t = cnt[w * a.experts + tid];
            cnt[w * a.experts + tid] = c;
            c += t;
        }
    const uint32_t padded = up_to(c, a.align);
    uint32_t total;
    const uint32_t off = block_exclusive(tid < a.experts ? padded : 0u, part, 16, total);
    if (tid < a.experts) {
        for (uint32_t w = 0; w < nwaves; ++w) cnt[w * a.experts + tid] += off;
        a.offsets[tid] = (int32_t)off;
        a.counts[tid] = (int32_t)c;
        for (uint32_t r = off + c; r < off + padded; ++r) a.slot[r] = -1;
    }
    if (tid == 0) a.offsets[a.experts] = (int32_t)total;
    for (uint32_t r = total + tid; r < a.capacity; r += 1024) a.slot[r] = -1;
    __syncthreads();
    if (wave < nwaves) place(a, lo, hi, mine);
}

__global__ __launch_bounds__(256) void route_count(RouteArgs a) {
    extern __shared__ uint32_t cnt[];
    for (uint32_t i = threadIdx.x; i < a.experts; i += 256) cnt[i] = 0;
    __syncthreads();
    const uint32_t lo = blockIdx.x * kTile, hi = lo + kTile < a.nslots ? lo + kTile : a.nslots;
    for (uint32_t i = lo + threadIdx.x; i < hi; i += 256) {
        const uint32_t id = (uint32_t)a.ids[i];
        if (id < a.experts) atomicAdd(&cnt[id], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += 256)
        a.ws[(uint64_t)e * a.tiles + blockIdx.x] = cnt[e];
}

// Workgroup e: exclusive sums over the tiles of expert e, and its count.
__global__ __launch_bounds__(256) void route_scan(RouteArgs a) {
    __shared__ uint32_t part[4];
    uint32_t* c = a.ws + (uint64_t)blockIdx.x * a.tiles;
    uint32_t carry = 0;
    for (uint32_t t0 = 0; t0 < a.tiles; t0 += 256) {
        const uint32_t t = t0 + threadIdx.x;
        const uint32_t v = t < a.tiles ? c[t] : 0u;
        uint32_t total;
        const uint32_t before = block_exclusive(v, part, 4, total);
        if (t < a.tiles) c[t] = carry + before;
        carry += total;
    }
    if (threadIdx.x == 0) a.counts[blockIdx.x] = (int32_t)carry;
}

// Workgroup b: offsets (every workgroup for itself), then the rows of its
// tile.  LDS: [4][experts] counts of the waves, which become next rows.
__global__ __launch_bounds__(256) void route_place(RouteArgs a) {
    extern __shared__ uint32_t cnt[];
    __shared__ uint32_t part[4];
    const uint32_t tid = threadIdx.x, wave = uniform(tid >> 6);
    for (uint32_t i = tid; i < 4 * a.experts; i += 256) cnt[i] = 0;
    __syncthreads();
    const uint32_t first = blockIdx.x * kTile;
    const uint32_t lo = first + wave * (kTile / 4) < a.nslots ? first + wave * (kTile / 4) : a.nslots;
    const uint32_t hi = lo + kTile / 4 < a.nslots ? lo + kTile / 4 : a.nslots;
    uint32_t* mine = cnt + wave * a.experts;
    count(a, lo, hi, mine);
    __syncthreads();
    uint32_t carry = 0;
    for (uint32_t e0 = 0; e0 < a.experts; e0 += 256) {
        const uint32_t e = e0 + tid;
        const uint32_t c = e < a.experts ? (uint32_t)a.counts[e] : 0u;
        const uint32_t padded = up_to(c, a.align);
        uint32_t total;
        const uint32_t off = carry + block_exclusive(padded, part, 4, total);
        carry += total;
        if (e < a.experts) {
            uint32_t next = off + a.ws[(uint64_t)e * a.tiles + blockIdx.x];
            for (uint32_t w = 0; w < 4; ++w) {
                const uint32_t t = cnt[w * a.experts + e];
                cnt[w * a.experts + e] = next;
                next += t;
            }
            if (blockIdx.x == e % a.tiles)
                for (uint32_t r = off + c; r < off + padded; ++r) a.slot[r] = -1;
            if (blockIdx.x == 0) a.offsets[e] = (int32_t)off;
        }
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = (int32_t)carry;
    for (uint64_t r = (uint64_t)carry + blockIdx.x * 256u + tid; r < a.capacity; r += (uint64_t)a.tiles * 256u)
        a.slot[r] = -1;
    __syncthreads();
    place(a, lo, hi, mine);
}

}  // namespace

uint64_t route_tiles(uint64_t nslots) { return nslots <= kSmall ? 0 : (nslots + kTile - 1) / kTile; }

zc_status launch_route(const RouteArgs& a, hipStream_t stream) {
    if (a.tiles == 0) {
        uint32_t nwaves = (a.nslots + 63) / 64;
        nwaves = nwaves < 1 ? 1 : nwaves > 16 ? 16 : nwaves;
        hipLaunchKernelGGL(route_small, dim3(1), dim3(1024), nwaves * a.experts * 4u, stream, a, nwaves);
        return ZC_OK;
    }
    hipLaunchKernelGGL(route_count, dim3(a.tiles), dim3(256), a.experts * 4u, stream, a);
    hipLaunchKernelGGL(route_scan, dim3(a.experts), dim3(256), 0, stream, a);
    hipLaunchKernelGGL(route_place, dim3(a.tiles), dim3(256), 4u * a.experts * 4u, stream, a);
    return ZC_OK;  // at most 2^21 tiles
}

}  // namespace zc
