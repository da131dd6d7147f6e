// zc_product.hip -- the experts' products of 8-bit blocks.
//
//   out[r, j] = sum over b of sA[r,b] sW[j,b] <A[r,b], W[j,b]>
//
// on v_mfma_scale_f32_16x16x128_f8f6f4: one instruction takes 16 rows of each
// side over a whole block of 128 and applies both blocks' scale exponents, so
// the scales cost no arithmetic and the sum over blocks stays in the unit's
// 32-bit accumulators.  The weight side is the instruction's first operand:
// a lane then has four neighbouring columns j of one row r.
//
// Rounding.  Before it adds them, the unit cuts the products of 8 neighbouring
// k to multiples of 2^-13 of the largest one's power of two.  That is a choice
// of this unit, for its rate; of one block of Gaussian values, error of the
// sum in its root mean square, and cycles a wave for 16 x 16 results:
//   this instruction               1.5e-5   32
//   16x16x32 of E4M3, unscaled     1.5e-5   65
//   16x16x32 of the values in bf16 1e-8     65
// Against products in 64 bits, bf16 results are off by 1.661e-3 of their rms
// with 32-bit sums and with these, fp16 results by 2.08e-4 and 2.09e-4: their
// own rounding.  In 32-bit results the cut is all there is (1.5e-5, whatever
// k); a caller who wants those closer multiplies the blocks' values in 32
// bits.
//
// Long sums are bound by the matrix unit and the chip's clock under it (16,384
// rows, n 4096, k 7168: 360 us, 2.7 PFLOP/s, 67% of the unit's cycles; for that
// the tiles are 256 x 256, a byte of operands for every 128 products); few rows
// an expert by the weights (64 rows on 32 experts, n 4096, k 7168: 117 us, 5.8
// TB/s); short sums by the results' stores (64 experts' weight gradients 2048 x
// 4096 over 128 rows each: 271 us, 4.0 TB/s).
#include "zc_experts_kernels.h"

#include <algorithm>
#include <type_traits>

namespace zc {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

[[maybe_unused]] __device__ __forceinline__ i32x8 two(xu32x4 lo, xu32x4 hi) {
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// One tile of a product, whichever product it is: rows of the token side
// against rows of the weight side, over `blocks` blocks.
struct Tile {
    const uint8_t* a;         // first row of the token side, at its first block
    const uint8_t* w;         // first row of the weight side, at its first block
    const uint8_t* as;        // their scales: by row (four blocks to a word), or
    const uint8_t* ws;        // by block (four rows to a word)
    uint32_t a_rows, w_rows;  // rows that exist from there on
    uint32_t a_stride, w_stride;    // bytes between rows
    uint64_t a_block, w_block;      // bytes between blocks
    uint32_t as_stride, ws_stride;  // bytes between scale rows, or scale blocks
    uint32_t blocks;
};

// How segments are cut: into slots of kRows rows; what is left is a slot of its
// own, a short one up to kShort rows.
struct WideCut {
    static constexpr uint32_t kRows = 256, kCols = 256, kShort = 128;
};
struct MidCut {
    static constexpr uint32_t kRows = 128, kCols = 128, kShort = 0;
    static constexpr int kStages = 4;
};
struct PairCut {  // MidCut's tiles, two workgroups on a CU
    static constexpr uint32_t kRows = 128, kCols = 128, kShort = 0;
    static constexpr int kStages = 2;
};
struct SmallCut {
    static constexpr uint32_t kRows = 64, kCols = 64, kShort = 0;
};
struct FewCut {
    static constexpr uint32_t kRows = 64, kCols = 32, kShort = 0;
};

__device__ __forceinline__ uint32_t clamp_to(int32_t v, uint32_t lo, uint32_t hi) {
    return v < (int32_t)lo ? lo : (uint32_t)v > hi ? hi : (uint32_t)v;
}

// The rows of one tile: `count` of expert's segment from `row` on (there may
// be more than a tile's), padding after them up to `end`.
struct Found {
    uint32_t expert, row, count, end, col;
    uint32_t any;
};

// Workgroup -> rows and columns.  Long slots keep the matrix unit busy and
// short ones the memory, so a launch of many tiles gives every XCD both in
// turn (kRuns): its CUs take tiles in runs of 32, 4 slots by 8 columns of one
// kind, so that what they read at one time is 4 + 8 strips shared through the
// XCD's L2, and runs of long and short slots alternate in proportion (65,536
// rows, Zipf counts on 256 experts, n 4096, k 7168: 2.57 ms; kinds as the
// experts come: 2.64).
enum Order { kInOrder, kRuns };

struct Slots {
    uint32_t slot, col;
    bool is_long, any;
};

__device__ __forceinline__ Slots slot_of(uint32_t index, uint32_t cols, uint32_t nlong, uint32_t nshort, Order order) {
    if (order == kInOrder) {
        const uint32_t s = index / cols;
        const bool l = s < nlong;
        return Slots{l ? s : s - nlong, index % cols, l, s < nlong + nshort};
    }
    const uint32_t xcd = index & 7, n = index >> 3, run = n >> 5;
    const uint32_t runs_l = ((nlong + 3) / 4 * cols + 7) / 8, runs_s = ((nshort + 3) / 4 * cols + 7) / 8;
    const uint32_t mine_l = (runs_l + 7 - xcd) / 8, mine_s = (runs_s + 7 - xcd) / 8, mine = mine_l + mine_s;
    if (run >= mine) return Slots{0, 0, false, false};
    // long runs before this one, and with it (a launch has below 2^24
    // workgroups, so an XCD below 2^16 runs and the products below 2^32)
    const uint32_t phase = xcd * mine / 8;
    const uint32_t before = (run * mine_l + phase) / mine, upto = ((run + 1) * mine_l + phase) / mine;
    const bool l = upto > before;
    const uint32_t tile = ((l ? before : run - before) * 8 + xcd) * 32 + (n & 31);
    const uint32_t group = tile / (4 * cols), in = tile % (4 * cols), slot = group * 4 + (in & 3);
    return Slots{slot, in >> 2, l, slot < (l ? nlong : nshort)};
}

// Long and short slots of a segment.
template <typename Cut>
__device__ __forceinline__ void slots_in(uint32_t count, bool padding, uint32_t& nlong, uint32_t& nshort) {
    const uint32_t rest = count % Cut::kRows;
    nlong = count / Cut::kRows + (rest > Cut::kShort ? 1 : 0);
    nshort = rest && rest <= Cut::kShort ? 1 : 0;
    if (!count && padding) nshort = 1;  // a segment of padding only
}

// Every thread looks at four experts; `shared` has room for 16 words.
template <typename Cut>
__device__ __forceinline__ Found find_tile(const ProductArgs& p, uint32_t index, uint32_t cols, Order order,
                                           uint32_t* shared) {
    if (!p.offsets) {
        uint32_t nl, ns;
        slots_in<Cut>(p.rows, false, nl, ns);
        const Slots s = slot_of(index, cols, nl, ns, order);
        const uint32_t row = (s.is_long ? s.slot : nl) * Cut::kRows;
        return Found{0, row, p.rows - row, p.rows, s.col, s.any};
    }
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6);
    uint32_t lo[4], count[4], end[4], nl[4], ns[4], sum_l = 0, sum_s = 0;
    const uint32_t e0 = threadIdx.x * 4;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        lo[q] = count[q] = end[q] = nl[q] = ns[q] = 0;
        if (e0 + q < p.experts) {
            const int32_t o0 = p.offsets[e0 + q], o1 = p.offsets[e0 + q + 1];
            const int32_t c = p.counts ? p.counts[e0 + q] : 0x7FFFFFFF;
            lo[q] = clamp_to(o0, 0, p.rows);
            end[q] = clamp_to(o1, lo[q], p.rows);
            count[q] = clamp_to(c, 0, end[q] - lo[q]);
            slots_in<Cut>(count[q], end[q] > lo[q], nl[q], ns[q]);
        }
        sum_l += nl[q];
        sum_s += ns[q];
    }
    uint32_t run_l = sum_l, run_s = sum_s;
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t tl = __shfl_up(run_l, d), ts = __shfl_up(run_s, d);
        if (lane >= d) {
            run_l += tl;
            run_s += ts;
        }
    }
    if (lane == 63) {
        shared[wave * 2] = run_l;
        shared[wave * 2 + 1] = run_s;
    }
    __syncthreads();
    uint32_t before_l = run_l - sum_l, before_s = run_s - sum_s, all_l = 0, all_s = 0;
#pragma unroll
    for (uint32_t v = 0; v < 4; ++v) {
        if (v < wave) {
            before_l += shared[v * 2];
            before_s += shared[v * 2 + 1];
        }
        all_l += shared[v * 2];
        all_s += shared[v * 2 + 1];
    }
    const Slots s = slot_of(index, cols, uniform(all_l), uniform(all_s), order);
    if (!s.any) return Found{0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t in = s.slot - (s.is_long ? before_l : before_s);
        if (in < (s.is_long ? nl[q] : ns[q])) {  // one thread of the workgroup
            const uint32_t skip = (s.is_long ? in : nl[q]) * Cut::kRows;
            shared[8] = e0 + q;
            shared[9] = lo[q] + skip;
            shared[10] = count[q] - skip;
            shared[11] = end[q];
        }
        before_l += nl[q];
        before_s += ns[q];
    }
    __syncthreads();
    const Found f{uniform(shared[8]), uniform(shared[9]), uniform(shared[10]), uniform(shared[11]), s.col, 1};
    __syncthreads();  // the tile's first loads may write where this was
    return f;
}

// The shape of a tile: 4 waves as WM x WN, each TM x TN instruction tiles of
// 16 x 16; S stages of one block (128 bytes of every row, and the scales) in
// LDS.  BY_BLOCK: scales lie by block, a byte for every row of either side;
// else by row, four blocks' bytes to a word, and 128 rows of the weight side
// share one.
template <int WM_, int TM_, int TN_, int S_, bool BY_BLOCK_>
struct Shape {
    static constexpr int WM = WM_, WN = 4 / WM_, TM = TM_, TN = TN_, S = S_;
    static constexpr bool BY_BLOCK = BY_BLOCK_;
    static constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    static constexpr int kScaleAt = (BM + BN) * 128;
    static constexpr int kStage = kScaleAt + 2048;
    static constexpr int kLoads = (BM + BN) / 32 + 2;  // per wave and stage
    static constexpr int kLds = S * kStage;
};

// Where a tile's results go.
template <typename T>
struct Out {
    T* out;              // row 0, column 0 of the tile
    uint64_t stride;     // elements
    uint32_t rows, cols; // of the tile that exist
};

// From here to the kernels the code uses types and registers that only the
// device has; the host's pass over this file sees the kernels' names alone.
#if defined(__HIP_DEVICE_COMPILE__)

typedef __attribute__((address_space(3))) void lds_void;

template <int N>
__device__ __forceinline__ void wait_loads_and_barrier() {
    // at most N loads to LDS outstanding and no read of LDS, in every wave
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0xFFFFFFFFu, 0x00020000);
}

// Row of the weight side that lane row m (0..15) of instruction tile i holds:
// two neighbouring tiles interleave in fours, so that a lane's results of the
// two are 8 neighbouring columns (one 16-byte store in 16-bit types).
__device__ __forceinline__ constexpr uint32_t weight_row(uint32_t i, uint32_t m) {
    return (i >> 1) * 32 + (m >> 2) * 8 + (i & 1) * 4 + (m & 3);
}

// Piece c (16 bytes) of a row lies at place c ^ turn(row) of its 128 bytes.
// LDS has 16 such places side by side (64 banks), two rows; a 16-byte read
// takes 16 lanes at a time, of which 8 have pieces one further than the other
// 8 (lanes 0-3, 12-15 with 20-27, and so on).  With the row orders in use
// (token rows as they come, weight rows as above) these turns give the 16
// lanes 16 different places, for the pieces g and g + 4 of lane group g.
__device__ __forceinline__ uint32_t turn_a(uint32_t row) { return (row >> 1) & 7; }
__device__ __forceinline__ uint32_t turn_w(uint32_t row) { return ((row >> 1) & 1) + ((row >> 3) & 3) * 2; }

// acc += the product of 16 weight rows and 16 token rows over one block, with
// both scales (low bytes).  The compiler knows the instruction and keeps the
// waits between it and whatever else touches its registers.  The empty asm
// holds it where it stands between loads, reads and barriers (the compiler
// takes it for arithmetic that may move: a wave's weight side then was copied,
// 64 moves a block) and its accumulators in the unit's own registers.
__device__ __forceinline__ void pin(f32x4& acc) { asm volatile("" : "+a"(acc)); }
__device__ __forceinline__ void multiply(f32x4& acc, const i32x8& w, const i32x8& a, uint32_t sw, uint32_t sa) {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc, 0, 0, 0, (int)sw, 0, (int)sa);
    pin(acc);
}

template <typename SH>
__device__ __forceinline__ void tile_product(const Tile& t, uint8_t* lds, f32x4 (&acc)[SH::TM][SH::TN]) {
    constexpr int NA = SH::BM / 32, NW = SH::BN / 32;
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6);
    const uint32_t r = lane & 15, g = lane >> 4;
    // a load moves 8 rows: lane l brings the piece that belongs at l's place
    uint32_t at_a[NA], at_w[NW];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const uint32_t row = (wave * NA + i) * 8 + (lane >> 3);
        at_a[i] = (row < t.a_rows ? row : t.a_rows - 1) * t.a_stride + (((lane & 7) ^ turn_a(row)) << 4);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const uint32_t row = (wave * NW + i) * 8 + (lane >> 3);
        at_w[i] = (row < t.w_rows ? row : t.w_rows - 1) * t.w_stride + (((lane & 7) ^ turn_w(row)) << 4);
    }
    // scales: by row, a lane brings its row's word of four blocks; by block, a
    // lane brings four rows' bytes, and every wave all of them for itself
    const uint32_t srow = SH::BY_BLOCK ? lane * 4 : wave * 64 + lane;
    const uint32_t last_a = t.a_rows < SH::BM ? t.a_rows - 1 : SH::BM - 1;
    const uint32_t last_w = t.w_rows < SH::BN ? t.w_rows - 1 : SH::BN - 1;
    const uint32_t arow = srow < last_a ? srow : last_a, wrow = srow < last_w ? srow : last_w;
    const uint32_t at_as = SH::BY_BLOCK ? arow & ~3u : arow * t.as_stride;
    const uint32_t at_ws = SH::BY_BLOCK ? wrow & ~3u : (wrow >> 7) * t.ws_stride;

    // the n-th of a wave's loads of a block.  PAST_END: blocks past the last are
    // loaded again instead of none, so that the loop is one piece; short sums
    // are faster without (256 experts 128 x 512 of 256 rows 43 -> 32 us), long
    // ones of the widest product's with (8192 rows, n 4096, k 7168 177 -> 170)
    constexpr bool PAST_END = SH::TM == 8 && !SH::BY_BLOCK;
    auto clamped = [&](uint32_t block) { return PAST_END && block >= t.blocks ? t.blocks - 1 : block; };
    auto load_one = [&](int n, uint32_t block, uint8_t* base) {
        const uint64_t sa = SH::BY_BLOCK ? (uint64_t)block * t.as_stride : block & ~3u;
        const uint64_t sw = SH::BY_BLOCK ? (uint64_t)block * t.ws_stride : block & ~3u;
        if (n < NA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(t.a + block * t.a_block),
                                                     (lds_void*)(base + (wave * NA + n) * 1024), 16, at_a[n], 0, 0, 0);
        else if (n < NA + NW)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(t.w + block * t.w_block),
                                                     (lds_void*)(base + SH::BM * 128 + (wave * NW + n - NA) * 1024), 16,
                                                     at_w[n - NA], 0, 0, 0);
        else if (n == NA + NW)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(t.as + sa), (lds_void*)(base + SH::kScaleAt + wave * 256), 4,
                                                     at_as, 0, 0, 0);
        else if (n == NA + NW + 1)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(t.ws + sw), (lds_void*)(base + SH::kScaleAt + 1024 + wave * 256),
                                                     4, at_ws, 0, 0, 0);
    };
    const uint32_t wave_a = (wave / SH::WN) * SH::TM * 16, wave_w = (wave % SH::WN) * SH::TN * 16;
    // where a lane's two pieces of a row lie (pieces g and g + 4)
    const uint32_t a_lo = (wave_a + r) * 128 + ((g ^ turn_a(r)) << 4), a_hi = a_lo ^ 64;
    const uint32_t w_lo = SH::BM * 128 + (wave_w + weight_row(0, r)) * 128 + ((g ^ turn_w(weight_row(0, r))) << 4);
    const uint32_t w_hi = w_lo ^ 64;
    const uint32_t a_scale = SH::kScaleAt + (SH::BY_BLOCK ? wave * 256 + wave_a + r : (wave_a + r) * 4);
    const uint32_t w_scale = SH::kScaleAt + 1024 + (SH::BY_BLOCK ? wave * 256 + wave_w + weight_row(0, r) : wave_w * 4);

    struct Side {     // 16 rows of one block
        i32x8 v;
        uint32_t s;   // the block's scale, or four blocks' scales
    };
    auto read_a = [&](const uint8_t* base, int j) {
        return Side{two(*(const xu32x4*)(base + a_lo + j * 2048), *(const xu32x4*)(base + a_hi + j * 2048)),
                    SH::BY_BLOCK ? base[a_scale + j * 16] : *(const uint32_t*)(base + a_scale + j * 64)};
    };
    auto read_w = [&](const uint8_t* base, int i, Side& x) {
        const uint32_t row = (i >> 1) * 32 + (i & 1) * 4;
        x.v = two(*(const xu32x4*)(base + w_lo + row * 128), *(const xu32x4*)(base + w_hi + row * 128));
        if (SH::BY_BLOCK) x.s = base[w_scale + row];
        else if (i == 0) x.s = *(const uint32_t*)(base + w_scale);
    };

    uint8_t* base = lds;
    for (uint32_t s = 0; s < SH::S && (PAST_END || s < t.blocks); ++s) {
#pragma unroll
        for (int n = 0; n < SH::kLoads; ++n) load_one(n, clamped(s), lds + s * SH::kStage);
    }
    if (PAST_END || t.blocks >= SH::S) wait_loads_and_barrier<(SH::S - 1) * SH::kLoads>();
    else wait_loads_and_barrier<0>();
    Side w[SH::TN], first = read_a(base, 0);
#pragma unroll
    for (int i = 0; i < SH::TN; ++i) read_w(base, i, w[i]);

    // One block a turn.  The weight side and the first token tile are in
    // registers; the other token tiles are read while the unit works on the
    // first HALF of them.  Then, with every wave that far, the stage is free:
    // while the unit works on the rest, the block S later is loaded there, its
    // loads spread evenly over the instructions (in one bunch they hold the
    // wave up: 2280 against 2580 TFLOP/s at 16384 x 4096 x 7168), and during the last
    // two tiles the next block's weight side replaces this one's.
    constexpr int HALF = SH::TM / 4 * 2, kEach = HALF ? (SH::TM - 2 + HALF) / HALF : 0;
    constexpr int kRest = (SH::TM - HALF) * SH::TN;
    // MORE: the block S later exists; without it all loads in flight are waited for.
    auto one_block = [&](auto more, uint32_t b) {
        constexpr bool MORE = decltype(more)::value;
        const uint32_t shift = SH::BY_BLOCK ? 0 : (b & 3) * 8;
        uint32_t sw[SH::TN];
        Side a[SH::TM];
        a[0] = first;
#pragma unroll
        for (int i = 0; i < SH::TN; ++i) sw[i] = SH::BY_BLOCK || i == 0 ? w[i].s >> shift : sw[0];
#pragma unroll
        for (int j = 0; j < HALF; ++j) {
#pragma unroll
            for (int n = 1 + j * kEach; n < 1 + (j + 1) * kEach && n < SH::TM; ++n) a[n] = read_a(base, n);
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t sa = a[j].s >> shift;
#pragma unroll
            for (int i = 0; i < SH::TN; ++i) multiply(acc[j][i], w[i].v, a[j].v, sw[i], sa);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (HALF == 0) a[1] = read_a(base, 1);
        wait_loads_and_barrier<MORE ? (SH::S - 2) * SH::kLoads : 0>();
        __builtin_amdgcn_sched_barrier(0);
        uint8_t* const free = base;
        const uint32_t ahead = clamped(b + SH::S);
        base = base == lds + (SH::S - 1) * SH::kStage ? lds : base + SH::kStage;
        int done = 0;
        auto load_share = [&](int at) {  // the loads due by the at-th instruction
            if (MORE)
#pragma unroll
                for (; done < SH::kLoads && done * kRest < at * SH::kLoads; ++done) load_one(done, ahead, free);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int j = HALF; j < SH::TM - 2; ++j) {
            const uint32_t sa = a[j].s >> shift;
#pragma unroll
            for (int i = 0; i < SH::TN; ++i) {
                multiply(acc[j][i], w[i].v, a[j].v, sw[i], sa);
                load_share((j - HALF) * SH::TN + i + 1);
            }
        }
        constexpr int J = SH::TM - 2;
        const uint32_t sa0 = a[J].s >> shift, sa1 = a[J + 1].s >> shift;
        first = read_a(base, 0);
#pragma unroll
        for (int i = 0; i < SH::TN; ++i) {
            multiply(acc[J][i], w[i].v, a[J].v, sw[i], sa0);
            multiply(acc[J + 1][i], w[i].v, a[J + 1].v, sw[i], sa1);
            read_w(base, i, w[i]);
            load_share(kRest - 2 * (SH::TN - 1 - i));
        }
    };
    // without this the first sums are known to be 0 + x, and the steady loop of
    // the smaller tiles moves its accumulators around (64 moves a block)
#pragma unroll
    for (int j = 0; j < SH::TM; ++j)
#pragma unroll
        for (int i = 0; i < SH::TN; ++i) pin(acc[j][i]);
    uint32_t b = 0;
    for (; b + (PAST_END ? 0 : SH::S) < t.blocks; ++b) one_block(std::true_type{}, b);
    if (!PAST_END)
        for (; b < t.blocks; ++b) one_block(std::false_type{}, b);
    // no load may still write LDS when another workgroup has it
    if (PAST_END) wait_loads_and_barrier<0>();
}

// An accumulator read where it is written down and no earlier: read ahead of
// the branches below, all of them would not fit the general registers.
__device__ __forceinline__ f32x4 late(f32x4 v) {
    pin(v);
    return v;
}

// 8 neighbouring results of a lane, as they lie in memory.
template <typename T>
struct Eight {
    xu32x4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Eight<T> eight(const f32x4& lo, const f32x4& hi) {
    if constexpr (sizeof(T) == 4) {
        return Eight<T>{{__builtin_bit_cast(xu32x4, lo), __builtin_bit_cast(xu32x4, hi)}};
    } else {
        typedef T Pair __attribute__((ext_vector_type(2)));
        auto pair = [](float x, float y) { return __builtin_bit_cast(uint32_t, Pair{(T)x, (T)y}); };
        return Eight<T>{{xu32x4{pair(lo[0], lo[1]), pair(lo[2], lo[3]), pair(hi[0], hi[1]), pair(hi[2], hi[3])}}};
    }
}

// The first `left` (1..7) of them, as 4 + 2 + 1.
template <typename T>
__device__ __forceinline__ void store_some(T* p, const Eight<T>& v, uint32_t left) {
    typedef xu32x4 __attribute__((aligned(2))) Four;
    typedef xu32x2 __attribute__((aligned(2))) Two;
    typedef uint32_t __attribute__((aligned(2))) One;
    const bool past = left & 4;
    if constexpr (sizeof(T) == 4) {
        const xu32x4 a = v.w[0], b = v.w[1];
        if (past) *reinterpret_cast<Four*>(p) = a;
        const uint32_t x = past ? b[0] : a[0], y = past ? b[1] : a[1], z = past ? b[2] : a[2];
        if (left & 2) *reinterpret_cast<Two*>(p + (left & 4)) = xu32x2{x, y};
        if (left & 1) *reinterpret_cast<One*>(p + (left & 6)) = left & 2 ? z : x;
    } else {
        const xu32x4 a = v.w[0];
        if (past) *reinterpret_cast<Two*>(p) = xu32x2{a[0], a[1]};
        const uint32_t x = past ? a[2] : a[0], y = past ? a[3] : a[1];
        if (left & 2) *reinterpret_cast<One*>(p + (left & 4)) = x;
        if (left & 1) *reinterpret_cast<uint16_t*>(p + (left & 6)) = (uint16_t)(left & 2 ? y : x);
    }
}

// A tile leaves from the registers, 8 neighbouring columns per lane, in
// 16-byte words.  Words that begin between multiples of 4 bytes cost twice
// (weight gradient, 64 experts 2048 x 4096, 4097 wide: 295, 632 us; with all
// words at multiples of 4: 373).  EDGES: the tile's columns end early,
// or its rows are of 16-bit values and some begin there; words of such a row
// begin one column before, with the column that the lane before holds.
template <typename T, typename SH, bool EDGES>
__device__ __forceinline__ void store_tile(const Out<T>& o, const f32x4 (&acc)[SH::TM][SH::TN]) {
    typedef xu32x4 __attribute__((aligned(2))) Word;
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t m0 = (wave / SH::WN) * SH::TM * 16, n0 = (wave % SH::WN) * SH::TN * 16 + g * 8;
    T* p = o.out + (m0 + r) * o.stride + n0;
    const uint32_t odd = EDGES && sizeof(T) == 2 ? ((uint32_t)(uintptr_t)p >> 1) & 1 : 0;  // in 16 rows the same again
#pragma unroll
    for (int j = 0; j < SH::TM; ++j) {
        if (m0 + j * 16 + r < o.rows) {
            uint32_t carry = 0;
#pragma unroll
            for (int i = 0; i < SH::TN; i += 2) {
                const f32x4 lo = late(acc[j][i]), hi = late(acc[j][i + 1]);
                Eight<T> v = eight<T>(lo, hi);
                T* to = p + i * 16;
                if constexpr (!EDGES) {
#pragma unroll
                    for (int q = 0; q < (int)sizeof(T) / 2; ++q) reinterpret_cast<Word*>(to)[q] = v.w[q];
                } else {
                    const uint32_t at = n0 + i * 16;
                    if constexpr (sizeof(T) == 2) {
                        const xu32x4 w = v.w[0];
                        const uint32_t behind = __shfl(w[3], (lane + 48) & 63), before = g ? behind : carry;
                        carry = behind;
                        if (odd) {
                            v.w[0] = xu32x4{w[0] << 16 | before >> 16, w[1] << 16 | w[0] >> 16, w[2] << 16 | w[1] >> 16,
                                            w[3] << 16 | w[2] >> 16};
                            uint16_t* edge = reinterpret_cast<uint16_t*>(to);
                            if (i == SH::TN - 2 && g == 3 && at + 7 < o.cols) edge[7] = (uint16_t)(w[3] >> 16);
                            if (i == 0 && g == 0) {
                                if (at < o.cols) edge[0] = (uint16_t)w[0];
                                if (at + 1 < o.cols)
                                    store_some(to + 1, Eight<T>{{xu32x4{v.w[0][1], v.w[0][2], v.w[0][3], 0}}},
                                               o.cols - at < 7 ? o.cols - at - 1 : 6);
                                continue;
                            }
                        }
                    }
                    if (at - odd + 8 <= o.cols) {
#pragma unroll
                        for (int q = 0; q < (int)sizeof(T) / 2; ++q) reinterpret_cast<Word*>(to - odd)[q] = v.w[q];
                    } else if (at - odd < o.cols) {
                        store_some(to - odd, v, o.cols - at + odd);
                    }
                }
            }
        }
        p += 16 * o.stride;
    }
}

#endif  // __HIP_DEVICE_COMPILE__

// start: what the sums begin with.
template <typename SH, typename T>
__device__ __forceinline__ void run_tile(const Tile& t, const Out<T>& o, uint8_t* lds, float start = 0.0f) {
#if defined(__HIP_DEVICE_COMPILE__)
    f32x4 acc[SH::TM][SH::TN];
#pragma unroll
    for (int j = 0; j < SH::TM; ++j)
#pragma unroll
        for (int i = 0; i < SH::TN; ++i) acc[j][i] = f32x4{start, start, start, start};
    if (t.blocks) tile_product<SH>(t, lds, acc);
    const bool odd = sizeof(T) == 2 && (((uintptr_t)o.out >> 1 | o.stride) & 1);
    if (o.cols >= (uint32_t)SH::BN && !odd) store_tile<T, SH, false>(o, acc);
    else store_tile<T, SH, true>(o, acc);
#endif
}

// Padding rows after the segment's last slot; cols of them from o.
template <typename T>
__device__ __forceinline__ void zero_padding(const Out<T>& o, const Found& f, uint32_t rows, uint32_t cols) {
    const uint32_t c = threadIdx.x % cols;
    if (f.count <= rows && c < o.cols)
        for (uint32_t q = f.count + threadIdx.x / cols; q < f.end - f.row; q += 256 / cols)
            o.out[q * o.stride + c] = (T)0.0f;
}

// One kernel for every length of a segment: a tile takes the shape of the rows
// it has, so that short segments do not pay for a whole slot and run beside
// long ones.
template <typename T, typename Cut>
__global__ __launch_bounds__(256, 1) void product(ProductArgs p, uint32_t col_tiles, Order order) {
    extern __shared__ __align__(16) uint8_t lds[];
    const Found f = find_tile<Cut>(p, blockIdx.x, col_tiles, order, reinterpret_cast<uint32_t*>(lds));
    if (!f.any) return;
    const uint32_t n0 = f.col * Cut::kCols;
    const uint32_t wrows = (p.n + 127) / 128;
    const Out<T> o{static_cast<T*>(p.out) + (uint64_t)f.row * p.out_stride + n0, p.out_stride, f.count, p.n - n0};
    if (f.count) {
        const Tile t{p.a + (uint64_t)f.row * p.k,
                     p.w + ((uint64_t)f.expert * p.n + n0) * p.k,
                     p.a_scale + (uint64_t)f.row * p.a_scale_stride,
                     p.w_scale + ((uint64_t)f.expert * wrows + n0 / 128) * p.w_scale_stride,
                     f.count, p.n - n0, p.k, p.k, 128, 128, p.a_scale_stride, p.w_scale_stride, p.k / 128};
        if constexpr (Cut::kRows == 256) {
            if (f.count > 128) run_tile<Shape<2, 8, 8, 2, false>>(t, o, lds);
            else if (f.count > 64) run_tile<Shape<2, 4, 8, 3, false>>(t, o, lds);
            else if (f.count > 32) run_tile<Shape<1, 4, 4, 3, false>>(t, o, lds);
            else run_tile<Shape<1, 2, 4, 4, false>>(t, o, lds);
        } else if constexpr (Cut::kRows == 64) {
            run_tile<Shape<2, 2, 2, 8, false>>(t, o, lds);
        } else {
            if (f.count > 64) run_tile<Shape<2, 4, 4, Cut::kStages, false>>(t, o, lds);
            else run_tile<Shape<1, 4, 2, Cut::kStages, false>>(t, o, lds);
        }
    }
    zero_padding(o, f, Cut::kRows, Cut::kCols);
}

// Few rows, or few tiles: 32 columns of up to 16 * TM rows per workgroup, the
// four waves taking every fourth block, straight from memory to the unit, and
// adding up in LDS in their order.  Nothing here is used twice but the rows,
// so staging would only hold loads back; narrow tiles put the weights of a few
// experts on all CUs (one CU draws about 50 GB/s from memory so, each wave
// with one block's loads in flight).
template <typename T, int TM>
__device__ __forceinline__ void few_tile(const ProductArgs& p, const Found& f, uint32_t n0, const Out<T>& o, float* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t left = p.n - n0, blocks = p.k / 128;
    const uint8_t* w[2];
    const uint8_t* a[TM];
    const uint8_t* as[TM];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t row = weight_row(i, r);
        w[i] = p.w + ((uint64_t)f.expert * p.n + n0 + (row < left ? row : left - 1)) * p.k + wave * 128 + g * 16;
    }
    const uint8_t* ws = p.w_scale + ((uint64_t)f.expert * ((p.n + 127) / 128) + n0 / 128) * p.w_scale_stride + wave;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const uint32_t row = j * 16 + r;
        const uint64_t at = f.row + (row < f.count ? row : f.count - 1);
        a[j] = p.a + at * p.k + wave * 128 + g * 16;
        as[j] = p.a_scale + at * p.a_scale_stride + wave;
    }
    f32x4 acc[TM][2];
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[j][0] = acc[j][1] = f32x4{0, 0, 0, 0};
    auto piece = [](const uint8_t* q) { return two(*(const xu32x4*)q, *(const xu32x4*)(q + 64)); };
    for (uint32_t b = wave; b < blocks; b += 4) {
        const uint32_t at = (b >> 2) * 512, sat = b & ~3u;
        const i32x8 w0 = piece(w[0] + at), w1 = piece(w[1] + at);
        const int sw = ws[sat];
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const i32x8 v = piece(a[j] + at);
            const int sa = as[j][sat];
            acc[j][0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w0, v, acc[j][0], 0, 0, 0, sw, 0, sa);
            acc[j][1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w1, v, acc[j][1], 0, 0, 0, sw, 0, sa);
        }
    }
    constexpr uint32_t kPitch = 36;
    float* mine = lds + wave * TM * 16 * kPitch;
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<f32x4*>(mine + (j * 16 + r) * kPitch + g * 8 + i * 4) = acc[j][i];
    __syncthreads();
    const uint32_t c = (threadIdx.x & 15) * 2;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const uint32_t row = j * 16 + (threadIdx.x >> 4);
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[h] += lds[(q * TM * 16 + row) * kPitch + c + h];
        if (row < f.count) {
            T* out = o.out + row * o.stride + c;
            struct Two {  // at any element's address
                T v[2];
            };
            if (c + 1 < o.cols) *reinterpret_cast<Two*>(out) = Two{{(T)v[0], (T)v[1]}};
            else if (c < o.cols) *out = (T)v[0];
        }
    }
#endif
}

template <typename T>
__global__ __launch_bounds__(256, 2) void product_few(ProductArgs p, uint32_t col_tiles) {
    __shared__ __align__(16) float lds[4 * 64 * 36];
    const Found f = find_tile<FewCut>(p, blockIdx.x, col_tiles, kInOrder, reinterpret_cast<uint32_t*>(lds));
    if (!f.any) return;
    const uint32_t n0 = f.col * FewCut::kCols;
    const Out<T> o{static_cast<T*>(p.out) + (uint64_t)f.row * p.out_stride + n0, p.out_stride, f.count, p.n - n0};
    if (f.count > 32) few_tile<T, 4>(p, f, n0, o, lds);
    else if (f.count > 16) few_tile<T, 2>(p, f, n0, o, lds);
    else if (f.count) few_tile<T, 1>(p, f, n0, o, lds);
    zero_padding(o, f, FewCut::kRows, FewCut::kCols);
}

// Workgroup -> (slot of rows of Y, tile of columns) in runs of 32 tiles, 4 slots
// by 8 columns, that the eight XCDs take in turn, so that what an XCD's 32 CUs
// read at one time is 4 + 8 strips, shared through its L2.
struct Place {
    uint32_t slot, col;
};
__device__ __forceinline__ Place place_of(uint32_t index, uint32_t cols) {
    const uint32_t xcd = index & 7, n = index >> 3;
    const uint32_t tile = ((n >> 5) * 8 + xcd) * 32 + (n & 31);
    const uint32_t group = tile / (4 * cols), in = tile % (4 * cols);
    return Place{group * 4 + (in & 3), in >> 2};
}

// Blocks of an expert's segment.  False, and no blocks, where it shares one
// with another segment: their rows cannot be told apart.
__device__ __forceinline__ bool segment_blocks(const WeightGradArgs& p, uint32_t e, uint32_t& b0, uint32_t& n) {
    b0 = 0;
    n = p.rows / 128;
    if (!p.offsets) return true;
    const int32_t begin = p.offsets[e], end = p.offsets[e + 1];
    const uint32_t lo = clamp_to(begin, 0, p.rows), hi = clamp_to(end, lo, p.rows);
    bool alone = (lo == hi) | ((lo | hi) % 128 == 0);
    // the last segment may end anywhere; its end is read only then (241 experts
    // 44 x 1986 of 128 rows, the shortest tiles: 85.4 us without a check, 87.5
    // so, 88.5 where every tile reads it; 37 experts 1000 x 1401 36.5 each way)
    if (!alone && lo % 128 == 0) alone = clamp_to(p.offsets[p.experts], hi, p.rows) == hi;
    b0 = lo / 128;
    n = lo < hi && alone ? (hi + 127) / 128 - b0 : 0;
    return alone;
}

// In how many parts a segment of n blocks is summed, of at most `parts`.
__device__ __forceinline__ uint32_t parts_of(uint32_t n, uint32_t parts) { return n < parts ? (n ? n : 1) : parts; }

// One tile of one expert's gradient, or (parts > 1) of its sum over one part
// of the segment, which goes to the part's own array of all gradients.
template <typename T, typename SH>
__global__ __launch_bounds__(256, 1) void weight_grad(WeightGradArgs p, T* out, uint32_t row_tiles, uint32_t col_tiles,
                                                      Order order, uint32_t per_part, uint32_t parts) {
    extern __shared__ __align__(16) uint8_t lds[];
    const uint32_t index = blockIdx.x % per_part, part = blockIdx.x / per_part;
    Place where;
    uint32_t e, i0;
    if (order == kRuns) {
        const uint32_t padded = (row_tiles + 3) / 4 * 4;  // an expert's slots, in whole runs
        where = place_of(index, col_tiles);
        e = where.slot / padded;
        i0 = where.slot % padded * SH::BM;
        if (e >= p.experts || i0 >= p.n) return;
    } else {
        where.col = index % col_tiles;
        where.slot = index / col_tiles;
        e = where.slot / row_tiles;
        i0 = where.slot % row_tiles * SH::BM;
    }
    const uint32_t j0 = where.col * SH::BN;
    uint32_t b0, n;
    const float start = segment_blocks(p, e, b0, n) ? 0.0f : __builtin_nanf("");
    if (parts > 1) {
        const uint32_t mine = parts_of(n, parts);
        if (part >= mine) return;
        const uint32_t lo = (uint32_t)((uint64_t)n * part / mine), hi = (uint32_t)((uint64_t)n * (part + 1) / mine);
        b0 += lo;
        n = hi - lo;
        out += (uint64_t)part * p.experts * p.n * p.k;
    }
    // block b of Y: [n][128] bytes, and n scale bytes
    const Tile t{p.y + ((uint64_t)b0 * p.n + i0) * 128,
                 p.x + ((uint64_t)b0 * p.k + j0) * 128,
                 p.y_scale + (uint64_t)b0 * p.y_scale_stride + i0,
                 p.x_scale + (uint64_t)b0 * p.x_scale_stride + j0,
                 p.n - i0, p.k - j0, 128, 128, (uint64_t)p.n * 128, (uint64_t)p.k * 128,
                 p.y_scale_stride, p.x_scale_stride, n};
    const Out<T> o{out + ((uint64_t)e * p.n + i0) * p.k + j0, p.k, p.n - i0, p.k - j0};
    run_tile<SH>(t, o, lds, start);
}

// The sum of an expert's parts, in their order.  grid: (pieces, experts).
template <typename T>
__global__ __launch_bounds__(256) void join_parts(WeightGradArgs p, const float* part, T* out, uint32_t parts) {
    const uint32_t e = blockIdx.y;
    uint32_t b0, n;
    segment_blocks(p, e, b0, n);
    const uint32_t mine = parts_of(n, parts);
    const uint64_t size = (uint64_t)p.n * p.k, all = size * p.experts;
    for (uint64_t i = (blockIdx.x * 256u + threadIdx.x) * 4ull; i < size; i += (uint64_t)gridDim.x * 1024) {
        const float* src = part + e * size + i;
        T* dst = out + e * size + i;
        if (i + 4 <= size) {
            typedef f32x4 __attribute__((aligned(4))) Word;
            f32x4 v = *reinterpret_cast<const Word*>(src);
            for (uint32_t q = 1; q < mine; ++q) v += *reinterpret_cast<const Word*>(src + q * all);
            struct Four {
                T v[4];
            };
            *reinterpret_cast<Four*>(dst) = Four{{(T)v[0], (T)v[1], (T)v[2], (T)v[3]}};
        } else {
            for (uint32_t j = 0; i + j < size; ++j) {
                float v = src[j];
                for (uint32_t q = 1; q < mine; ++q) v += src[q * all + j];
                dst[j] = (T)v;
            }
        }
    }
}

typedef Shape<2, 8, 8, 2, true> GradWide;
typedef Shape<2, 4, 4, 4, true> GradMid;
typedef Shape<2, 4, 4, 2, true> GradMidPair;  // two workgroups on a CU
typedef Shape<2, 2, 2, 4, true> GradSmall;
typedef Shape<2, 2, 2, 2, true> GradSmallMany;  // four workgroups on a CU

constexpr int kLdsProduct = Shape<1, 2, 4, 4, false>::kLds > Shape<2, 4, 8, 3, false>::kLds ? Shape<1, 2, 4, 4, false>::kLds
                                                                                           : Shape<2, 4, 8, 3, false>::kLds;
static_assert(kLdsProduct <= 160 * 1024 && Shape<2, 8, 8, 2, false>::kLds <= kLdsProduct &&
                  Shape<1, 4, 4, 3, false>::kLds <= kLdsProduct,
              "one LDS allocation serves every shape");
constexpr int kLdsMid = Shape<2, 4, 4, 4, false>::kLds;
static_assert(Shape<1, 4, 2, 4, false>::kLds <= kLdsMid, "one LDS allocation serves every shape");
constexpr int kLdsPair = Shape<2, 4, 4, 2, false>::kLds;
static_assert(Shape<1, 4, 2, 2, false>::kLds <= kLdsPair && 2 * kLdsPair <= 160 * 1024, "two workgroups on a CU");
constexpr int kLdsSmall = Shape<2, 2, 2, 8, false>::kLds;

// More LDS than the default limit has to be asked for.  Every launch does (a
// call of 3.5 us of host time, 3.4 without), so nothing has to be kept of
// which GPU has been asked.
template <typename K>
zc_status allow_lds(K kernel, int bytes) {
    const auto f = reinterpret_cast<const void*>(kernel);
    if (hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess) return ZC_OK;
    (void)hipGetLastError();  // reported here, not by the next launch
    return ZC_ERR_HIP;
}

}  // namespace

namespace {

// Which cut, from what the host knows: rows, experts, n (not the counts).
// Measured, in us, at n 4096, k 7168 where not said (wide / mid / pair):
//   few    up to 4 rows an expert and 32 more, against mid / small: 16 rows, 1
//          expert 13/24/20; 64 rows, 8 experts, n 14336, k 4096 95/110/117; 128
//          rows, 32 experts 164/163/181, but 512 rows there 217/174/201
//   wide   where its tiles fill most CUs, and an expert's rows most of a tile:
//          4096 rows, 1 expert 92/149/127, but 2048 rows 79/76/62; 16384 rows,
//          16 experts, n 512, k 1024 23/32/28; 2048 rows, 32 experts 254/206/211
//   small  where mid has at most 64 tiles: 128 rows, 1 expert 22 (mid 33); 256
//          rows 24 (33), but 512 rows 44 (34)
//   pair   where mid has more tiles than CUs, so that one's stores run beside
//          the other's loads, but not for many blocks of few rows, whose loads
//          need mid's depth: 5947 rows, 201 experts, n 849, k 113 34/31/20; 8423
//          rows, 1 expert, n 543, k 4297 51/49/41; but 1024 rows, 32 experts
//          245/180/199, and 1024 rows, 1 expert (256 tiles) 72/39/47
//   mid    else
template <typename T>
zc_status product_as(const ProductArgs& a, hipStream_t stream) {
    const uint64_t segments = a.offsets ? a.experts : 1;
    const uint64_t used = a.experts < a.rows ? a.experts : a.rows;  // segments that can have rows
    auto cols = [&](uint32_t c) { return (a.n + c - 1) / c; };
    auto in_order = [&](auto kernel, auto cut, int lds) {
        typedef decltype(cut) Cut;
        const uint64_t grid = (a.rows / Cut::kRows + segments) * cols(Cut::kCols);
        if (!fits(grid)) return ZC_ERR_UNSUPPORTED;
        if (zc_status e = allow_lds(kernel, lds)) return e;
        hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(256), lds, stream, a, cols(Cut::kCols), kInOrder);
        return ZC_OK;
    };
    if (a.rows <= 4 * a.experts + 32) {
        const uint64_t grid = (a.rows / FewCut::kRows + segments) * cols(FewCut::kCols);
        if (!fits(grid)) return ZC_ERR_UNSUPPORTED;
        hipLaunchKernelGGL((product_few<T>), dim3((uint32_t)grid), dim3(256), 0, stream, a, cols(FewCut::kCols));
        return ZC_OK;
    }
    const uint64_t whole = a.rows / WideCut::kRows, ends = std::min(used / 2, whole / 4);
    if ((whole + ends) * cols(WideCut::kCols) >= 144 && a.rows >= 128 * used) {
        const uint64_t s = a.rows / WideCut::kRows + segments, c = cols(WideCut::kCols);
        if (s * c <= 512) return in_order(product<T, WideCut>, WideCut{}, kLdsProduct);
        // runs: each kind's slots rounded up to 4, its tiles to runs of 32, its
        // runs to the 8 XCDs
        const uint64_t grid = (((s + 6) / 4 * c + 14) / 8 + 14) / 8 * 256;
        if (!fits(grid)) return ZC_ERR_UNSUPPORTED;
        if (zc_status e = allow_lds(product<T, WideCut>, kLdsProduct)) return e;
        hipLaunchKernelGGL((product<T, WideCut>), dim3((uint32_t)grid), dim3(256), kLdsProduct, stream, a, (uint32_t)c, kRuns);
        return ZC_OK;
    }
    const uint64_t rest = a.experts > 1 ? used : a.rows % MidCut::kRows ? 1 : 0;
    const uint64_t tiles = (a.rows / MidCut::kRows + rest) * cols(MidCut::kCols);
    if (tiles <= 64) return in_order(product<T, SmallCut>, SmallCut{}, kLdsSmall);
    if (tiles > 256 && (a.k <= 2048 || a.rows >= 64 * a.experts)) return in_order(product<T, PairCut>, PairCut{}, kLdsPair);
    return in_order(product<T, MidCut>, MidCut{}, kLdsMid);
}

}  // namespace

zc_status launch_product(const ProductArgs& a, hipStream_t stream) {
    if (a.out_dtype == ZC_BF16) return product_as<__bf16>(a, stream);
    if (a.out_dtype == ZC_FP16) return product_as<_Float16>(a, stream);
    return product_as<float>(a, stream);
}

namespace {

template <typename T, typename SH>
zc_status weight_grad_in(const WeightGradArgs& a, T* out, uint32_t parts, hipStream_t stream) {
    const uint32_t rows = (a.n + SH::BM - 1) / SH::BM, cols = (a.k + SH::BN - 1) / SH::BN;
    const uint64_t tiles = (uint64_t)a.experts * rows * cols;
    const Order order = tiles > 512 ? kRuns : kInOrder;
    const uint64_t each = order == kRuns ? ((uint64_t)a.experts * ((rows + 3) / 4 * 4) * cols + 255) / 256 * 256 : tiles;
    if (!fits(each * parts)) return ZC_ERR_UNSUPPORTED;
    if (zc_status e = allow_lds(weight_grad<T, SH>, SH::kLds)) return e;
    hipLaunchKernelGGL((weight_grad<T, SH>), dim3((uint32_t)(each * parts)), dim3(256), SH::kLds, stream, a, out, rows, cols,
                       order, (uint32_t)each, parts);
    return ZC_OK;
}

template <typename T>
zc_status weight_grad_shaped(const WeightGradArgs& a, T* out, const WeightGradPlan& plan, hipStream_t stream) {
    if (plan.side == 256) return weight_grad_in<T, GradWide>(a, out, plan.parts, stream);
    // with more tiles than CUs, a tile's stores beside the next one's loads are
    // worth more than loads further ahead: 32 experts 2048 x 7168 of 128 rows
    // 444 us one to a CU, 316 in pairs
    const uint64_t tiles = (uint64_t)a.experts * ((a.n + 127) / 128) * ((a.k + 127) / 128) * plan.parts;
    if (plan.side == 128 && tiles > 256) return weight_grad_in<T, GradMidPair>(a, out, plan.parts, stream);
    if (plan.side == 128) return weight_grad_in<T, GradMid>(a, out, plan.parts, stream);
    // likewise, where they outnumber what the CUs hold: 62 experts 62 x 526 of
    // 896 rows 35 (one to a CU, 7 blocks ahead) / 22 (two, 4) / 18 (four, 2); but 1
    // expert 1024 x 1024, 4096 rows 12.8 / 12.7 / 19.1
    const uint64_t small = (uint64_t)a.experts * ((a.n + 63) / 64) * ((a.k + 63) / 64) * plan.parts;
    if (small > 512) return weight_grad_in<T, GradSmallMany>(a, out, plan.parts, stream);
    return weight_grad_in<T, GradSmall>(a, out, plan.parts, stream);
}

template <typename T>
zc_status weight_grad_as(const WeightGradArgs& a, const WeightGradPlan& plan, float* ws, hipStream_t stream) {
    T* out = static_cast<T*>(a.dw);
    if (plan.parts == 1) return weight_grad_shaped<T>(a, out, plan, stream);
    if (zc_status e = weight_grad_shaped<float>(a, ws, plan, stream)) return e;
    const uint64_t pieces = ((uint64_t)a.n * a.k + 1023) / 1024, most = 4096 / a.experts + 1;
    hipLaunchKernelGGL(join_parts<T>, dim3((uint32_t)(pieces < most ? pieces : most), a.experts), dim3(256), 0, stream, a, ws,
                       out, plan.parts);
    return ZC_OK;
}

}  // namespace

WeightGradPlan plan_weight_grad(uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, bool split) {
    auto tiles = [&](uint32_t side) { return (uint64_t)experts * ((n + side - 1) / side) * ((k + side - 1) / side); };
    // The widest tiles that still give most CUs one; in us, 256 / 128 / 64 wide:
    //   448, 1792, 7168 tiles (1 expert 4096 x 7168, 4096 rows) 99/134/326
    //   192, 704, 2816 (8 experts 1000 x 1401, 32768 rows)      137/87/153
    //   128, 512, 2048 (16 experts 512 x 1024, 32768 rows)      109/60/67
    //   16, 64, 256 (1 expert 1024 x 1024, 4096 rows)           42/20/15
    // and do not go past n and k by more than two fifths; in us, 128 / 64 wide:
    //   241 experts 44 x 1986, 128 rows each    89/70    50 experts 88 x 8791, 128 rows  117/79
    //   but 100 experts 300 x 1000, 256 rows    30/39 (31% past)
    auto snug = [&](uint32_t side) { return tiles(side) * side * side * 5 <= (uint64_t)experts * n * k * 7; };
    const uint32_t blocks = rows / 128 / experts;
    // Short segments leave most of the time to the stores, which a pair on a CU
    // hides; 256 wide / pairs of 128, by blocks of 128 rows an expert:
    //   37 experts 1000 x 1401  1: 44/39  4: 58/55      16 experts 1408 x 2048  2: 38/27  8: 73/70
    //   8 experts 4096 x 4096   1: 63/62  3: 94/103     128 experts 1024 x 1024  2: 90/111
    const bool loose = tiles(256) * 65536 * 20 > (uint64_t)experts * n * k * 21;
    const bool pairs = tiles(128) >= 512 && (blocks <= 1 || (loose && blocks <= 8));
    if (tiles(256) >= 256 && snug(256) && !pairs) return WeightGradPlan{256, 1};
    // Few tiles and long segments: a CU draws some 50 GB/s past its L2, so the
    // segments go to more CUs, at the price of the join; whole / in parts:
    //   1 expert 1024 x 1024, 32768 rows  87 (64 wide) / 53 (128 wide, 4 parts)
    //   1 expert 60 x 300, 32768 rows     77 / 16 (64 wide, 16 parts)
    //   but at 32 blocks of 128 rows an expert, 1024 x 1024   15 / 20
    if (split && blocks >= 64 && tiles(128) <= 128) {
        const uint32_t side = tiles(64) <= 32 ? 64 : 128;
        const uint64_t most = 256 / tiles(side);
        return WeightGradPlan{side, most > 16 ? 16u : (uint32_t)most};
    }
    if (tiles(128) >= 192 && snug(128)) return WeightGradPlan{128, 1};
    return WeightGradPlan{64, 1};
}

zc_status launch_weight_grad(const WeightGradArgs& a, const WeightGradPlan& plan, void* ws, hipStream_t stream) {
    if (a.out_dtype == ZC_BF16) return weight_grad_as<__bf16>(a, plan, static_cast<float*>(ws), stream);
    if (a.out_dtype == ZC_FP16) return weight_grad_as<_Float16>(a, plan, static_cast<float*>(ws), stream);
    return weight_grad_as<float>(a, plan, static_cast<float*>(ws), stream);
}

}  // namespace zc
