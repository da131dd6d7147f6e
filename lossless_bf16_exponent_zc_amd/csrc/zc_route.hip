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
// Up to kSmall slots one workgroup does everything in one launch.  Above, two:
// counts per tile, then ranks, for which every workgroup adds up the tiles
// before its own; from kMostSummed tiles on a launch between them scans the
// tiles once for all.
//
// Bound by latency: 64 slots on 256 experts 3.7 us, 65,536 slots 8.8 us in a row
// of such calls and 10.6 behind other kernels (4.7 + 5.9; 0.8 MB, 0.2 us at the
// memory's rate), 524,288 slots 15 us.  Tiles of 2048 put 65,536
// slots on 32 CUs and leave few counts to add up (tiles of 1024 in three
// launches: 16.3 us); one launch for 8192 slots took 12.5 us, two take 8.
#include "zc_experts_kernels.h"

namespace zc {

namespace {

constexpr uint32_t kTile = 2048;       // slots per workgroup of the large form
constexpr uint32_t kSmall = 2048;      // slots of the one-launch form
constexpr uint32_t kMostSummed = 128;  // tiles that a workgroup adds up by itself

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

// A wave's slots: 64 * R from `lo` on, below `hi`, R of them per lane (the
// i-th of a lane is lo + 64 i + lane); their ids are read once, at the start.
template <int R>
struct Keys {
    uint32_t key[R];  // expert, or `experts` for none
    __device__ __forceinline__ Keys(const RouteArgs& a, uint32_t lo, uint32_t hi) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const uint32_t i = lo + q * 64 + __lane_id();
            const uint32_t id = i < hi ? (uint32_t)a.ids[i] : ~0u;
            key[q] = id < a.experts ? id : a.experts;
        }
    }
    // adds the slots of each expert to cnt
    __device__ __forceinline__ void count(const RouteArgs& a, uint32_t* cnt) const {
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (key[q] < a.experts) atomicAdd(&cnt[key[q]], 1u);
    }
    // writes rows and slots; next: the row of each expert's next slot, which
    // this wave alone advances
    __device__ __forceinline__ void place(const RouteArgs& a, uint32_t lo, uint32_t hi, uint32_t* next) const {
        const uint32_t lane = __lane_id(), bits = key_bits(a.experts);
        uint32_t first[R], rank[R], base[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const uint64_t m = same_key(key[q], bits);
            first[q] = __ffsll((unsigned long long)m) - 1;
            rank[q] = __popcll(m & ((1ull << lane) - 1));
            base[q] = 0;
            if (lane == first[q] && key[q] < a.experts) base[q] = atomicAdd(&next[key[q]], (uint32_t)__popcll(m));
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const uint32_t i = lo + q * 64 + lane, r = __shfl(base[q], first[q]) + rank[q];
            if (i < hi) {
                a.row[i] = key[q] < a.experts ? (int32_t)r : -1;
                if (key[q] < a.experts) a.slot[r] = (int32_t)i;
            }
        }
    }
};

// The rows from `from` on to no slot, by `groups` workgroups together.  With
// padding that is done for all rows, before those with a slot get it (a thread
// for an expert's padding rows: 100 tokens on 512 experts, align 128, 21.4 us;
// so 6.4); without, for what the packed rows leave.
__device__ __forceinline__ void no_slots(const RouteArgs& a, uint32_t from, uint32_t groups) {
    for (uint64_t r = (uint64_t)from + blockIdx.x * 1024u + threadIdx.x; r < a.capacity; r += groups * 1024ull) a.slot[r] = -1;
}

// One workgroup of 1024 threads.  LDS: [waves][experts] counts.
__global__ __launch_bounds__(1024) void route_small(RouteArgs a, uint32_t nwaves) {
    extern __shared__ uint32_t cnt[];
    __shared__ uint32_t part[16];
    const uint32_t tid = threadIdx.x, wave = uniform(tid >> 6);
    for (uint32_t i = tid; i < nwaves * a.experts; i += 1024) cnt[i] = 0;
    if (a.align > 1) no_slots(a, 0, 1);
    __syncthreads();
    const uint32_t each = up_to((a.nslots + nwaves - 1) / nwaves, 64);
    const uint32_t lo = wave * each < a.nslots ? wave * each : a.nslots;
    const uint32_t hi = lo + each < a.nslots ? lo + each : a.nslots;
    uint32_t* mine = cnt + wave * a.experts;
    const Keys<kSmall / 1024> keys(a, lo, hi);
    if (wave < nwaves) keys.count(a, mine);
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
    }
    if (tid == 0) a.offsets[a.experts] = (int32_t)total;
    if (a.align == 1) no_slots(a, total, 1);
    __syncthreads();
    if (wave < nwaves) keys.place(a, lo, hi, mine);
}

__global__ __launch_bounds__(1024) void route_count(RouteArgs a) {
    extern __shared__ uint32_t cnt[];
    for (uint32_t i = threadIdx.x; i < a.experts; i += 1024) cnt[i] = 0;
    if (a.align > 1) no_slots(a, 0, a.tiles);
    __syncthreads();
    const uint32_t lo = blockIdx.x * kTile;
#pragma unroll
    for (uint32_t q = 0; q < kTile / 1024; ++q) {
        const uint32_t i = lo + q * 1024 + threadIdx.x;
        const uint32_t id = i < a.nslots ? (uint32_t)a.ids[i] : ~0u;
        if (id < a.experts) atomicAdd(&cnt[id], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += 1024) a.ws[(uint64_t)blockIdx.x * a.experts + e] = cnt[e];
}

// For 64 experts a workgroup: sums over the tiles before each, in place, and
// after the last tile's the experts' counts.  16 threads share an expert.
__global__ __launch_bounds__(1024) void route_scan(RouteArgs a) {
    __shared__ uint32_t part[16][64];
    const uint32_t lane = threadIdx.x & 63, seg = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
    const uint32_t each = (a.tiles + 15) / 16, lo = seg * each, hi = lo + each < a.tiles ? lo + each : a.tiles;
    uint32_t sum = 0;
    if (e < a.experts) {
#pragma unroll 8
        for (uint32_t t = lo; t < hi; ++t) sum += a.ws[(uint64_t)t * a.experts + e];
    }
    part[seg][lane] = sum;
    __syncthreads();
    if (e >= a.experts) return;
    uint32_t before = 0, all = 0;
    for (uint32_t s = 0; s < 16; ++s) {
        before += s < seg ? part[s][lane] : 0u;
        all += part[s][lane];
    }
#pragma unroll 8
    for (uint32_t t = lo; t < hi; ++t) {
        const uint32_t v = a.ws[(uint64_t)t * a.experts + e];
        a.ws[(uint64_t)t * a.experts + e] = before;
        before += v;
    }
    if (seg == 0) a.ws[(uint64_t)a.tiles * a.experts + e] = all;
}

// Workgroup b: offsets (every workgroup for itself), then the rows of its
// tile.  LDS: [16][experts] counts of the waves, which become next rows.
__global__ __launch_bounds__(1024) void route_place(RouteArgs a, bool scanned) {
    extern __shared__ uint32_t cnt[];
    __shared__ uint32_t part[16];
    const uint32_t tid = threadIdx.x, wave = uniform(tid >> 6);
    const uint32_t first = blockIdx.x * kTile + wave * (kTile / 16);
    const uint32_t lo = first < a.nslots ? first : a.nslots;
    const uint32_t hi = lo + kTile / 16 < a.nslots ? lo + kTile / 16 : a.nslots;
    const Keys<kTile / 1024> keys(a, lo, hi);
    for (uint32_t i = tid; i < 16 * a.experts; i += 1024) cnt[i] = 0;
    __syncthreads();
    uint32_t* mine = cnt + wave * a.experts;
    keys.count(a, mine);
    uint32_t before = 0, c = 0;  // of expert tid: slots in earlier tiles, and in all
    if (tid < a.experts) {
        if (scanned) {
            before = a.ws[(uint64_t)blockIdx.x * a.experts + tid];
            c = a.ws[(uint64_t)a.tiles * a.experts + tid];
        } else {
#pragma unroll 16
            for (uint32_t t = 0; t < a.tiles; ++t) {
                const uint32_t v = a.ws[(uint64_t)t * a.experts + tid];
                c += v;
                before += t < blockIdx.x ? v : 0u;
            }
        }
    }
    __syncthreads();
    const uint32_t padded = up_to(c, a.align);
    uint32_t total;
    const uint32_t off = block_exclusive(padded, part, 16, total);
    if (tid < a.experts) {
        uint32_t next = off + before;
        uint32_t v[16];
#pragma unroll
        for (uint32_t w = 0; w < 16; ++w) v[w] = cnt[w * a.experts + tid];
#pragma unroll
        for (uint32_t w = 0; w < 16; ++w) {
            cnt[w * a.experts + tid] = next;
            next += v[w];
        }
        if (blockIdx.x == 0) {
            a.offsets[tid] = (int32_t)off;
            a.counts[tid] = (int32_t)c;
        }
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = (int32_t)total;
    if (a.align == 1) no_slots(a, total, a.tiles);
    __syncthreads();
    keys.place(a, lo, hi, mine);
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
    const bool scan = a.tiles >= kMostSummed;
    hipLaunchKernelGGL(route_count, dim3(a.tiles), dim3(1024), a.experts * 4u, stream, a);
    if (scan) hipLaunchKernelGGL(route_scan, dim3((a.experts + 63) / 64), dim3(1024), 0, stream, a);
    hipLaunchKernelGGL(route_place, dim3(a.tiles), dim3(1024), 16u * a.experts * 4u, stream, a, scan);
    return ZC_OK;  // at most 2^20 tiles of 2^10 threads
}

}  // namespace zc
