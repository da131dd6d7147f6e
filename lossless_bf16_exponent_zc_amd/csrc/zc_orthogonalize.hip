// zc_orthogonalize.hip -- updates made orthogonal by Newton-Schulz products.
//
// Of a matrix, Y is the orientation with at least as many rows as columns (x or
// its transpose), length x side:
//   Y <- Y / (|Y| + eps);   steps times:  A = Y^T Y,  P = b A + c A^2,
//                                         Y <- a Y + Y P
// which is X <- a X + (b A + c A^2) X, A = X X^T, turned over where x has fewer
// rows.  Y is held in both orientations, as rows of `side` and as rows of
// `length`, so that every product sums along rows of both its factors and
// nothing is transposed between memory and the matrix unit.
//
// Numbers.  The products run on v_mfma_f32_16x16x32_f16.  Their factors are
// fp16, 11 bits at bf16's rate: with bf16 factors results are off by 1e-2 of
// their rms and more.  Y itself is kept as a pair of fp16, hi and 2^11 times what
// hi was rounded by, within 2^-23 of itself; the products read hi.  A step
// multiplies a small singular value by up to a, five of them by 485, and with
// them what Y was rounded by, while errors of the products' factors stay where A
// is large.  Near the end A and P are nearly diagonal, and what their diagonals
// were rounded by is kept in 32 bits and put back where P and the new Y are made,
// as is the diagonal's product with lo in the last two steps.  (Off from 64 bits
// by, in the root mean square, steps one by one: Gaussian 512 x 1792 6e-4,
// spectrum 1/i^2 and rank one in bf16 2e-4; without lo 1.4e-3, 2e-2, 1e-1.  Rank one 512 x 512 after 8, 10
// and 12 steps 2e-3, 2e-2 and 0.3, with all in 32 bits 5e-3, 6e-2 and 0.7.  The
// result's own rounding to bf16 is 1.7e-3.)
// Y is held times 2^shift, about the square root of its length, so that its
// elements lie in fp16's normal range.
#include "zc_experts_kernels.h"

#include <type_traits>
#include <utility>

namespace zc {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Of matrices of side x side: A = Y^T Y (kGram), gamma M^2 + alpha M (kSquare),
// gamma M N + alpha M + beta N (kMix).  Of Y: factor Y + Y M, in the making
// (kApply) or as the result (kLast).
enum Product { kGram, kSquare, kMix, kApply, kLast };

// Tiles of kSide x kSide by four waves, 2 x 2, each T x T instruction tiles of
// 16 x 16; S stages in LDS, each of 64 of the summed dimension.
template <int T_, int S_>
struct Shape {
    static constexpr int T = T_, S = S_;
    static constexpr int kSide = 32 * T;
    static constexpr int kOperand = kSide * 128;  // bytes of one operand's stage
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kEach = kSide / 32;      // loads per wave, operand and stage
    static constexpr int kLoads = 2 * kEach;
    static constexpr int kLds = S * kStage;
    static constexpr int kOnCu = 2 * kLds <= 160 * 1024 ? 2 : 1;
};

// One operand of a product, result[i][j] = sum over c of left[i][c] right[j][c].
struct Operand {
    const uint8_t* p;  // first row of the tile
    uint32_t stride;   // bytes between rows
    uint32_t rows;     // that exist from there on
};

// lo is what hi was rounded by, times kLow: at most as large as hi, so that it is
// not subnormal before hi is, and 11 bits more of Y are kept whatever its size.
constexpr float kLow = 2048.0f;
template <typename H, typename F>
__device__ __forceinline__ H remainder(const F& v, const H& hi) {
    return __builtin_convertvector((v - __builtin_convertvector(hi, F)) * kLow, H);
}

// New Y: product + factor (hi + lo) + low lo.
template <typename F, typename H>
__device__ __forceinline__ F stepped(const F& product, const F& factor, const F& low, const H& hi, const H& lo) {
    const F h = __builtin_convertvector(hi, F), l = __builtin_convertvector(lo, F);
    const F whole = __builtin_elementwise_fma(l, F(1.0f / kLow), h);
    return __builtin_elementwise_fma(factor, whole, __builtin_elementwise_fma(low, l, product));
}

// The products read hi alone.  Where P is nearly diagonal, as it is in the end,
// what lo is missed by most is the diagonal's product with it, which Y + Y P
// adds by itself: the products of the last two steps, `done` of all being done
// then.  Not before: where singular values are next to nothing it would be noise
// in their directions (the rest of P takes it away again), and what grows by a in
// every step after.  Off by, after five steps, without / in the last / in the
// last two / in all: Gaussian 512 x 512 1.2e-3 / 1.0e-3 / 0.8e-3 / 0.7e-3, 512 x
// 1024 1.6e-3 / 1.5e-3 / 0.5e-3 / 0.5e-3, rank one 64 x 64 7e-4 / 7e-4 / 7e-4 /
// 6e-3.
__host__ __device__ constexpr float low_of(uint32_t done, uint32_t steps) { return done + 1 >= steps ? 1.0f / kLow : 0.0f; }

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

// The empty asm holds the accumulators in the unit's own registers, and the
// instructions where they stand between loads, reads and barriers.
__device__ __forceinline__ void pin(f32x4& acc) { asm volatile("" : "+a"(acc)); }

struct Part {  // 16 rows of an operand, 64 of c: c = 8 g + 0..7 and 32 more, lane group g
    f16x8 v[2];
};

__device__ __forceinline__ void multiply(f32x4& acc, const Part& right, const Part& left) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(right.v[0], left.v[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(right.v[1], left.v[1], acc, 0, 0, 0);
    pin(acc);
}

// Row that lane row m (0..15) of part t holds: two neighbouring parts interleave
// in fours, so that a lane's results of two by two parts are 8 neighbouring
// columns of two rows, and 8 neighbouring rows where they leave turned over:
// 16-byte words either way.
__device__ __forceinline__ constexpr uint32_t part_row(uint32_t t, uint32_t m) {
    return (t >> 1) * 32 + (m >> 2) * 8 + (t & 1) * 4 + (m & 3);
}

// Piece c (16 bytes) of a row lies at place c ^ turn(row) of its 128 bytes.  LDS
// has 16 places side by side, two rows, and a 16-byte read takes 16 lanes at a
// time, of which 8 have pieces one further than the other 8 (lanes 0-3, 12-15
// with 20-27, and so on); with the rows in the order above these turns give
// them 16 different places.
__device__ __forceinline__ uint32_t turn(uint32_t row) { return ((row >> 1) & 1) + ((row >> 3) & 3) * 2; }

// acc[ti][tj] += the products of a tile, over `blocks` blocks of 64.  A lane
// then has, of part (ti, tj), row part_row(ti, lane & 15) and the four columns
// from part_row(tj, (lane >> 4) * 4) on.
template <typename SH>
__device__ __forceinline__ void tile_product(const Operand& left, const Operand& right, uint32_t blocks, uint8_t* lds,
                                             f32x4 (&acc)[SH::T][SH::T]) {
    constexpr int T = SH::T, E = SH::kEach;
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    // a load moves 8 rows: lane l brings the piece that belongs at l's place
    uint32_t at_l[E], at_r[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const uint32_t row = (wave * E + i) * 8 + (lane >> 3), piece = ((lane & 7) ^ turn(row)) << 4;
        at_l[i] = (row < left.rows ? row : left.rows - 1) * left.stride + piece;
        at_r[i] = (row < right.rows ? row : right.rows - 1) * right.stride + piece;
    }
    auto load_one = [&](int n, uint32_t block, uint8_t* stage) {
        if (n < E)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(left.p + block * 128ull), (lds_void*)(stage + (wave * E + n) * 1024),
                                                     16, at_l[n], 0, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(right.p + block * 128ull),
                                                     (lds_void*)(stage + SH::kOperand + (wave * E + n - E) * 1024), 16,
                                                     at_r[n - E], 0, 0, 0);
    };
    // where a lane's two pieces of a row lie (pieces g and g + 4)
    const uint32_t first = part_row(0, r), in = first * 128 + ((g ^ turn(first)) << 4);
    const uint32_t lo_l = (wave >> 1) * T * 2048 + in, lo_r = SH::kOperand + (wave & 1) * T * 2048 + in;
    auto read = [&](const uint8_t* stage, uint32_t lo, int t) {
        const uint8_t* p = stage + part_row(t, 0) * 128;
        return Part{{*reinterpret_cast<const f16x8*>(p + lo), *reinterpret_cast<const f16x8*>(p + (lo ^ 64))}};
    };

    for (uint32_t s = 0; s < SH::S && s < blocks; ++s) {
#pragma unroll
        for (int n = 0; n < SH::kLoads; ++n) load_one(n, s, lds + s * SH::kStage);
    }
    if (blocks >= SH::S) wait_loads_and_barrier<(SH::S - 1) * SH::kLoads>();
    else wait_loads_and_barrier<0>();
    uint8_t* stage = lds;
    Part right_part[T], next = read(stage, lo_l, 0);
#pragma unroll
    for (int j = 0; j < T; ++j) right_part[j] = read(stage, lo_r, j);

    // One block a turn.  The right side and the left's first part are in
    // registers; the other left parts are read while the unit works on the first
    // HALF of them.  Then, with every wave that far, the stage is free: while the
    // unit works on the rest, the block S later is loaded there, its loads spread
    // over the instructions, and during the last two parts the next block's right
    // side replaces this one's.
    constexpr int HALF = T / 4 * 2, kAhead = HALF ? (T - 2 + HALF) / HALF : 0;
    constexpr int kRest = (T - HALF) * T;
    auto one_block = [&](auto more, uint32_t b) {
        constexpr bool MORE = decltype(more)::value;  // the block S later exists
        Part l[T];
        l[0] = next;
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
#pragma unroll
            for (int n = 1 + i * kAhead; n < 1 + (i + 1) * kAhead && n < T; ++n) l[n] = read(stage, lo_l, n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < T; ++j) multiply(acc[i][j], right_part[j], l[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (HALF == 0) l[1] = read(stage, lo_l, 1);
        wait_loads_and_barrier<MORE ? (SH::S - 2) * SH::kLoads : 0>();
        __builtin_amdgcn_sched_barrier(0);
        uint8_t* const free = stage;
        stage = stage == lds + (SH::S - 1) * SH::kStage ? lds : stage + SH::kStage;
        int done = 0;
        auto load_share = [&](int at) {  // the loads due by the at-th instruction
            if (MORE)
#pragma unroll
                for (; done < SH::kLoads && done * kRest < at * SH::kLoads; ++done) load_one(done, b + SH::S, free);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int i = HALF; i < T - 2; ++i) {
#pragma unroll
            for (int j = 0; j < T; ++j) {
                multiply(acc[i][j], right_part[j], l[i]);
                load_share((i - HALF) * T + j + 1);
            }
        }
        next = read(stage, lo_l, 0);
#pragma unroll
        for (int j = 0; j < T; ++j) {
            multiply(acc[T - 2][j], right_part[j], l[T - 2]);
            multiply(acc[T - 1][j], right_part[j], l[T - 1]);
            right_part[j] = read(stage, lo_r, j);
            load_share(kRest - 2 * (T - 1 - j));
        }
    };
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) pin(acc[i][j]);
    uint32_t b = 0;
    for (; b + SH::S < blocks; ++b) one_block(std::true_type{}, b);
    for (; b < blocks; ++b) one_block(std::false_type{}, b);
}

// An accumulator read where it is written down and no earlier.
__device__ __forceinline__ f32x4 late(f32x4 v) {
    pin(v);
    return v;
}

// The transpose of 4 x 4 values that a quad of lanes holds, one row each.
__device__ __forceinline__ f16x4 turned_over(f16x4 v) {
    const uint32_t lane = __lane_id();
    const xu32x2 w = __builtin_bit_cast(xu32x2, v);
    auto from = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xF, 0xF, true);
    };
    typedef std::integral_constant<int, 0x4E> Two;  // lanes 2, 3, 0, 1
    typedef std::integral_constant<int, 0xB1> One;  // lanes 1, 0, 3, 2
    const uint32_t got = from(lane & 2 ? w[0] : w[1], Two{});
    // rows of lanes 0, 1 and of lanes 2, 3 (their values 0, 1, or 2, 3)
    const uint32_t a = lane & 2 ? got : w[0], b = lane & 2 ? w[1] : got;
    const uint32_t oa = from(a, One{}), ob = from(b, One{});
    // v_perm picks bytes 0-3 of the second and 4-7 of the first operand
    const uint32_t pick = lane & 1 ? 0x07060302u : 0x01000504u;
    return __builtin_bit_cast(f16x4, xu32x2{__builtin_amdgcn_perm(a, oa, pick), __builtin_amdgcn_perm(b, ob, pick)});
}

// A block's two rows of 8 columns as two columns' 8 rows: o[w] is column 4 w +
// (lane & 3) of the lane group's 8, and the 8 rows from the quad's first on.
__device__ __forceinline__ void over_rows(f16x8 (&o)[2]) {
    auto half = [](f16x8 v, auto w) {
        constexpr int W = decltype(w)::value;
        return turned_over(__builtin_shufflevector(v, v, W, W + 1, W + 2, W + 3));
    };
    typedef std::integral_constant<int, 0> First;
    typedef std::integral_constant<int, 4> Second;
    const f16x8 a = __builtin_shufflevector(half(o[0], First{}), half(o[1], First{}), 0, 1, 2, 3, 4, 5, 6, 7);
    const f16x8 b = __builtin_shufflevector(half(o[0], Second{}), half(o[1], Second{}), 0, 1, 2, 3, 4, 5, 6, 7);
    o[0] = a;
    o[1] = b;
}
__device__ __forceinline__ void store_over(_Float16* m, uint32_t stride, uint32_t i, uint32_t j, f16x8 (&o)[2]) {
    const uint32_t q = __lane_id() & 3;
    over_rows(o);
    *reinterpret_cast<f16x8*>(m + (uint64_t)(j + q) * stride + (i - q)) = o[0];
    *reinterpret_cast<f16x8*>(m + (uint64_t)(j + 4 + q) * stride + (i - q)) = o[1];
}

// The first `left` of 8 values of 16 bits, at any element's address.
__device__ __forceinline__ void store_some(__bf16* p, f16x8 o, int32_t left) {
    typedef xu32x4 __attribute__((aligned(2))) Word;
    const xu32x4 w = __builtin_bit_cast(xu32x4, o);
    if (left >= 8) {
        *reinterpret_cast<Word*>(p) = w;
        return;
    }
    uint16_t* to = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int q = 0; q < 7; ++q)
        if (q < left) to[q] = (uint16_t)(w[q / 2] >> (q & 1) * 16);
}

// Workgroup -> tile.  Workgroups go to the eight XCDs in turn, and an XCD takes
// one run of neighbouring tiles, so that what its CUs read at one time is a few
// strips, shared through its L2.
__device__ __forceinline__ uint32_t of_run(uint32_t index, uint32_t per_xcd) { return (index & 7) * per_xcd + (index >> 3); }

struct Place {
    uint32_t i, j;
};
// Tile `index` of the lower triangle, row by row.
__device__ __forceinline__ Place lower(uint32_t index) {
    uint32_t i = (uint32_t)((sqrtf(8.0f * (float)index + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > index) --i;
    while ((i + 1) * (i + 2) / 2 <= index) ++i;
    return Place{i, index - i * (i + 1) / 2};
}
// Tile `index` of `rows` x `cols`, in bands of four rows, column by column.
__device__ __forceinline__ Place banded(uint32_t index, uint32_t rows, uint32_t cols) {
    const uint32_t band = index / (4 * cols), in = index % (4 * cols), left = rows - 4 * band, high = left < 4 ? left : 4;
    return Place{4 * band + in % high, in / high};
}

#endif  // __HIP_DEVICE_COMPILE__

// One product of a step, one tile a workgroup.  Long sums are bound by the matrix
// unit (Y P of 1 x 14336 x 4096 500 us, 0.96 PFLOP/s); short ones by what a tile
// reads and writes beside its sum, which nothing overlaps on a CU that holds one
// tile: Y P of 32 x 7168 x 2048 2.42 ms, 0.80 PFLOP/s and 3.4 TB/s, as the result
// (bf16 alone) 1.92.  OVER: the result leaves turned over (kLast).
template <typename SH, int KIND, bool OVER>
__global__ __launch_bounds__(256, SH::kOnCu) void step_product(OrthArgs p, uint32_t tiles, uint32_t side_tiles) {
    extern __shared__ __align__(16) uint8_t lds[];
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr bool SYMMETRIC = KIND <= kMix;
    constexpr int T = SH::T;
    const uint32_t place = of_run(blockIdx.x, gridDim.x >> 3), matrix = place / tiles, index = place % tiles;
    if (matrix >= p.batch) return;
    const Place at = SYMMETRIC ? lower(index) : banded(index, tiles / side_tiles, side_tiles);
    const uint32_t i0 = at.i * SH::kSide, j0 = at.j * SH::kSide;
    const uint64_t y_at = (uint64_t)matrix * p.length * p.side, s_at = (uint64_t)matrix * p.side * p.side;
    const _Float16 *hi = p.hi + y_at, *across = p.across + y_at, *M = p.matrix + s_at, *N = p.other + s_at;
    f32x4 acc[T][T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    // addresses in scalar registers, where the loads to LDS want them
    auto rows_of = [](const _Float16* m, uint32_t from, uint32_t rows, uint32_t stride) {
        const uint64_t p = (uint64_t)(m + (uint64_t)from * stride);
        const uint64_t scalar = (uint64_t)uniform((uint32_t)(p >> 32)) << 32 | uniform((uint32_t)p);
        return Operand{reinterpret_cast<const uint8_t*>(scalar), stride * 2, rows - from};
    };
    if constexpr (KIND == kGram)
        tile_product<SH>(rows_of(across, i0, p.side, p.length), rows_of(across, j0, p.side, p.length), p.length / 64, lds, acc);
    else if constexpr (SYMMETRIC)
        tile_product<SH>(rows_of(M, i0, p.side, p.side), rows_of(N, j0, p.side, p.side), p.side / 64, lds, acc);
    else
        tile_product<SH>(rows_of(hi, i0, p.length, p.side), rows_of(M, j0, p.side, p.side), p.side / 64, lds, acc);

    // Results leave in blocks of two by two parts: of a block, a lane has 8
    // neighbouring columns of two rows, four apart.
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t wi = i0 + (wave >> 1) * T * 16, wj = j0 + (wave & 1) * T * 16, ri = wi + part_row(0, r), rj = wj + g * 8;
    const uint32_t end_i = SYMMETRIC ? p.side : p.length;
    auto results = [&](int b, int h) {
        const int ti = b / (T / 2) * 2 + h, tj = b % (T / 2) * 2;
        return __builtin_shufflevector(late(acc[ti][tj]), late(acc[ti][tj + 1]), 0, 1, 2, 3, 4, 5, 6, 7);
    };
    constexpr int kBlocks = T * T / 4, kAhead = kBlocks < 2 ? kBlocks : 2;  // loads run ahead by so many
    // side and length are multiples of 64: a block is there or not as a whole
    auto there = [&](int b) { return wi + b / (T / 2) * 32 < end_i && wj + b % (T / 2) * 32 < p.side; };
    const float *rest_m = p.rest_m + (uint64_t)matrix * 2 * p.side, *rest_n = p.rest_n + (uint64_t)matrix * 2 * p.side;
    if constexpr (SYMMETRIC) {
        _Float16* out = p.made + s_at;
        float* left_over = p.rest_made + (uint64_t)matrix * 2 * p.side;
        struct Was {
            f16x8 m[2], n[2];
        };
        auto fetch = [&](int b) {
            const uint32_t i = ri + b / (T / 2) * 32, j = rj + b % (T / 2) * 32;
            Was w;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t e = (uint64_t)(i + 4 * h) * p.side + j;
                w.m[h] = *reinterpret_cast<const f16x8*>(M + e);
                w.n[h] = KIND == kMix ? *reinterpret_cast<const f16x8*>(N + e) : w.m[h];
            }
            return w;
        };
        auto value = [&](int b, int h, const Was& was) __attribute__((always_inline)) {
            f32x8 v = results(b, h);
            if constexpr (KIND == kGram) {
                v *= p.inverse_square;
            } else {
                // with what the diagonals of M and N were rounded by, to the first order
                const uint32_t row = ri + b / (T / 2) * 32 + 4 * h, j = rj + b % (T / 2) * 32;
                const f32x8 m = __builtin_convertvector(was.m[h], f32x8), n = __builtin_convertvector(was.n[h], f32x8);
                v = p.gamma * (v + m * *reinterpret_cast<const f32x8*>(rest_n + j) + rest_m[row] * n) + p.alpha * m + p.beta * n;
            }
            return v;
        };
        auto leave = [&](int b, const Was& was) __attribute__((always_inline)) {
            const uint32_t i = ri + b / (T / 2) * 32, j = rj + b % (T / 2) * 32;
            f16x8 o[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                o[h] = __builtin_convertvector(value(b, h, was), f16x8);
                *reinterpret_cast<f16x8*>(out + (uint64_t)(i + 4 * h) * p.side + j) = o[h];
            }
            store_over(out, p.side, i, j, o);
        };
        // What is left of the diagonal leaves turned over too, as what is right of
        // it: the two halves of M N are only equal up to rounding, and which tile
        // an element is in must not change it.
        if (wi > wj && i0 + SH::kSide <= p.side) {
            Was was[kAhead];
            if (KIND != kGram)
#pragma unroll
                for (int b = 0; b < kAhead; ++b) was[b] = fetch(b);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const Was now = was[b % kAhead];
                if (KIND != kGram && b + kAhead < kBlocks) was[b % kAhead] = fetch(b + kAhead);
                leave(b, now);
            }
        } else if (wi >= wj) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                if ((wi > wj || b / (T / 2) > b % (T / 2)) && there(b)) leave(b, KIND == kGram ? Was{} : fetch(b));
        }
        if (wi == wj) {
#pragma unroll
            for (int d = 0; d < T / 2; ++d) {
                const int b = d * (T / 2) + d;
                if (!there(b)) continue;
                const uint32_t j = rj + d * 32;
                const Was was = KIND == kGram ? Was{} : fetch(b);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t row = ri + d * 32 + 4 * h;
                    const f32x8 v = value(b, h, was);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float e = v[q];
                        if (KIND != kGram && j + q == row) e += p.alpha * rest_m[row] + p.beta * rest_n[row];
                        const _Float16 o = (_Float16)e;
                        if (j + q <= row) out[(uint64_t)row * p.side + j + q] = o;
                        if (j + q < row) out[(uint64_t)(j + q) * p.side + row] = o;
                        if (j + q == row) {
                            left_over[row] = e - (float)o;
                            left_over[p.side + row] = (float)o;
                        }
                    }
                }
            }
        }
    } else {
        struct Was {
            f16x8 hi[2], lo[2];
            f32x8 rest, diagonal;
        };
        auto fetch = [&](int b) {
            const uint32_t i = ri + b / (T / 2) * 32, j = rj + b % (T / 2) * 32;
            Was w;
            w.rest = *reinterpret_cast<const f32x8*>(rest_m + j);
            w.diagonal = *reinterpret_cast<const f32x8*>(rest_m + p.side + j);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t e = y_at + (uint64_t)(i + 4 * h) * p.side + j;
                w.hi[h] = *reinterpret_cast<const f16x8*>(p.hi + e);
                w.lo[h] = *reinterpret_cast<const f16x8*>(p.lo + e);
            }
            return w;
        };
        auto leave = [&](auto whole) __attribute__((always_inline)) {
            constexpr bool WHOLE = decltype(whole)::value;
            Was was[kAhead];
#pragma unroll
            for (int b = 0; b < kAhead; ++b)
                if (WHOLE || there(b)) was[b] = fetch(b);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const Was now = was[b % kAhead];
                if (b + kAhead < kBlocks && (WHOLE || there(b + kAhead))) was[b % kAhead] = fetch(b + kAhead);
                if (!WHOLE && !there(b)) continue;
                const uint32_t i = ri + b / (T / 2) * 32, j = rj + b % (T / 2) * 32;
                const f32x8 factor = p.factor + now.rest, low = p.low * now.diagonal;
                f16x8 o[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x8 v = stepped(results(b, h), factor, low, now.hi[h], now.lo[h]);
                    if constexpr (KIND == kApply) {
                        const uint64_t e = y_at + (uint64_t)(i + 4 * h) * p.side + j;
                        o[h] = __builtin_convertvector(v, f16x8);
                        *reinterpret_cast<f16x8*>(p.next + e) = o[h];
                        *reinterpret_cast<f16x8*>(p.lo + e) = remainder<f16x8>(v, o[h]);
                    } else {
                        o[h] = __builtin_bit_cast(f16x8, __builtin_convertvector(v * p.inverse, bf16x8));
                    }
                }
                if constexpr (KIND == kApply) {
                    store_over(p.across + y_at, p.length, i, j, o);
                } else {
                    __bf16* out = p.out + (uint64_t)matrix * p.n * p.k;
                    if (OVER) over_rows(o);
                    const uint32_t row = OVER ? j + (r & 3) : i, col = OVER ? i - (r & 3) : j;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (row + 4 * h < p.n) store_some(out + (uint64_t)(row + 4 * h) * p.k + col, o[h], (int32_t)(p.k - col));
                }
            }
        };
        if (i0 + SH::kSide <= p.length && j0 + SH::kSide <= p.side) leave(std::true_type{});
        else leave(std::false_type{});
    }
#endif
}

// Sums of squares of x, p.parts of them a matrix.  In 64 bits: neither values
// near 1e38 nor near 1e-38 leave their range.
template <typename T>
__global__ __launch_bounds__(256) void squares(OrthArgs p) {
    __shared__ double sum[4];
    constexpr uint32_t kEach = 16 / sizeof(T);
    const uint64_t size = (uint64_t)p.n * p.k, words = (size + kEach - 1) / kEach;
    const uint32_t matrix = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    const T* x = static_cast<const T*>(p.x) + matrix * size;
    double s = 0.0;
    for (uint64_t w = (uint64_t)part * 256 + threadIdx.x; w < words; w += p.parts * 256ull) {
        const uint64_t at = w * kEach, left = size - at;
        const xu32x4 word = load_word(x + at, left < kEach ? (int32_t)left : (int32_t)kEach);
        T v[kEach];
        __builtin_memcpy(v, &word, 16);
#pragma unroll
        for (uint32_t q = 0; q < kEach; ++q) {
            const double d = (double)to_float(v[q]);
            s = fma(d, d, s);
        }
    }
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) p.part[blockIdx.x] = sum[0] + sum[1] + sum[2] + sum[3];
}

// Y = x / (|x| + eps) times 2^shift, with zeros up to multiples of 64 rows and
// columns: hi and lo as rows of side, hi alone as rows of length.  OVER: Y is x
// turned over.  One tile of 64 x 64 a workgroup, by way of LDS.
template <typename T, bool OVER>
__global__ __launch_bounds__(256) void normalize(OrthArgs p, uint32_t col_tiles) {
    __shared__ double sum[4];
    __shared__ float tile[64][65];
    const uint32_t matrix = blockIdx.y, i0 = blockIdx.x / col_tiles * 64, j0 = blockIdx.x % col_tiles * 64;
    double s = 0.0;
    for (uint32_t q = threadIdx.x; q < p.parts; q += 256) s += p.part[(uint64_t)matrix * p.parts + q];
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = s;
    __syncthreads();
    const double size = sqrt(sum[0] + sum[1] + sum[2] + sum[3]) + (double)p.eps;
    const double f = size == 0.0 ? 0.0 : (double)p.scale / size;
    const T* x = static_cast<const T*>(p.x) + (uint64_t)matrix * p.n * p.k;
    constexpr uint32_t kEach = 16 / sizeof(T), kWords = 64 / kEach;
#pragma unroll
    for (uint32_t w = threadIdx.x; w < 64 * kWords; w += 256) {
        const uint32_t r = w / kWords, c = w % kWords * kEach, i = i0 + r, j = j0 + c;
        xu32x4 word = {0, 0, 0, 0};
        if (i < p.n && j < p.k) word = load_word(x + (uint64_t)i * p.k + j, p.k - j < kEach ? (int32_t)(p.k - j) : (int32_t)kEach);
        T v[kEach];
        __builtin_memcpy(v, &word, 16);
#pragma unroll
        for (uint32_t q = 0; q < kEach; ++q) tile[r][c + q] = (float)((double)to_float(v[q]) * f);
    }
    __syncthreads();
    const uint64_t y_at = (uint64_t)matrix * p.length * p.side;
    const uint32_t along = OVER ? p.length : p.side, down = OVER ? p.side : p.length;  // of x's rows, of its columns
#pragma unroll
    for (uint32_t w = threadIdx.x; w < 512; w += 256) {
        const uint32_t a = w >> 3, b = w & 7;
        f16x8 straight, straight_lo, over, over_lo;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float v = tile[a][b * 8 + q], t = tile[b * 8 + q][a];
            straight[q] = (_Float16)v;
            straight_lo[q] = (_Float16)((v - (float)straight[q]) * kLow);
            over[q] = (_Float16)t;
            over_lo[q] = (_Float16)((t - (float)over[q]) * kLow);
        }
        const uint64_t at_s = y_at + (uint64_t)(i0 + a) * along + j0 + b * 8, at_o = y_at + (uint64_t)(j0 + a) * down + i0 + b * 8;
        *reinterpret_cast<f16x8*>((OVER ? p.across : p.next) + at_s) = straight;
        *reinterpret_cast<f16x8*>((OVER ? p.next : p.across) + at_o) = over;
        if (OVER) *reinterpret_cast<f16x8*>(p.lo + at_o) = over_lo;
        else *reinterpret_cast<f16x8*>(p.lo + at_s) = straight_lo;
    }
}

// A whole update of a matrix of side up to 64 and length up to 512 in one
// workgroup, with Y (hi, lo), A and P in LDS: the steps of such a matrix take
// less than the launches that go between them (1 x 64 x 256: 71 us in 17
// launches).  Sums, factors and roundings are those of the tiled products.
constexpr uint32_t kSmallLength = 512;
constexpr uint32_t small_lds(uint32_t length) { return 2 * length * 128 + 2 * 8192 + 3 * 256; }

template <typename T, bool OVER>
__global__ __launch_bounds__(512) void update_small(OrthArgs p, uint32_t steps) {
    extern __shared__ __align__(16) uint8_t lds[];
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ double sum[8];
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    const uint32_t tid = threadIdx.x, lane = __lane_id(), wave = uniform(tid >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t L = p.length;
    uint8_t *const hi = lds, *const lo = lds + L * 128, *const A = lds + 2 * L * 128, *const P = A + 8192;
    float *const rest_a = reinterpret_cast<float*>(P + 8192), *const rest_p = rest_a + 64, *const diagonal = rest_p + 64;
    // rows of 64 fp16, their 16-byte pieces turned: Y's in pairs, so that reads
    // along rows and across them find different banks
    auto y_at = [](uint32_t row, uint32_t col) {
        return row * 128 + (((col >> 3) ^ ((row & 2) | ((row >> 1) & 4))) << 4) + (col & 7) * 2;
    };
    auto m_at = [](uint32_t row, uint32_t col) { return row * 128 + (((col >> 3) ^ ((row >> 1) & 7)) << 4) + (col & 7) * 2; };
    // f(row, col, value) of every value of x, in little code: with one workgroup,
    // instructions come from memory once and are waited for
    const uint32_t size = p.n * p.k, down = 512 / p.k, right_by = 512 % p.k;
    const T* x = static_cast<const T*>(p.x) + (uint64_t)blockIdx.x * size;
    auto each = [&](auto f) {
        uint32_t row = tid / p.k, col = tid % p.k;
#pragma unroll 4
        for (uint32_t e = tid; e < size; e += 512) {
            f(row, col, to_float(x[e]));
            row += down;
            col += right_by;
            if (col >= p.k) {
                col -= p.k;
                ++row;
            }
        }
    };
    for (uint32_t at = tid * 16; at < 2 * L * 128; at += 512 * 16) *reinterpret_cast<xu32x4*>(lds + at) = xu32x4{0, 0, 0, 0};
    double s = 0.0;
    each([&](uint32_t, uint32_t, float v) { s = fma((double)v, (double)v, s); });
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) sum[wave] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < 8; ++w) s += sum[w];
    const double whole = sqrt(s) + (double)p.eps, f = whole == 0.0 ? 0.0 : (double)p.scale / whole;
    each([&](uint32_t row, uint32_t col, float v) {
        const float y = (float)((double)v * f);
        const _Float16 h = (_Float16)y;
        const uint32_t at = OVER ? y_at(col, row) : y_at(row, col);
        *reinterpret_cast<_Float16*>(hi + at) = h;
        *reinterpret_cast<_Float16*>(lo + at) = (_Float16)((y - (float)h) * kLow);
    });
    __syncthreads();

    // 16 rows, or columns, of an operand: c = 8 g to 8 g + 7 of the 32 from c0 on
    auto along = [&](const uint8_t* m, uint32_t at) { return *reinterpret_cast<const f16x8*>(m + at); };
    auto across = [&](uint32_t t, uint32_t c0) {
        i16x4 q[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)  // lane 4 a + b of a group brings columns 4 b to 4 b + 3 of row a, and gets column 4 a + b
            q[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(hi + y_at(c0 + 8 * g + 4 * u + (r >> 2), t * 16 + (r & 3) * 4)));
        return __builtin_bit_cast(f16x8, __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    // of the matrices 64 x 64 a wave has two of the 16 parts: rows i, columns j to j + 3
    const uint32_t ti = wave & 3, tj0 = wave >> 2 << 1, i = ti * 16 + r;
    for (uint32_t step = 0; step < steps; ++step) {
        f32x4 acc[4] = {};
        for (uint32_t c = 0; c < L; c += 64) {
            f16x8 part[2][3];  // asked for at once
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                part[h][0] = across(ti, c + 32 * h);
                part[h][1] = across(tj0, c + 32 * h);
                part[h][2] = across(tj0 + 1, c + 32 * h);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < 2; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(part[h][1 + t], part[h][0], acc[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t j = (tj0 + t) * 16 + g * 4;
            const f32x4 v = acc[t] * p.inverse_square;
            const f16x4 h = __builtin_convertvector(v, f16x4);
            *reinterpret_cast<f16x4*>(A + m_at(i, j)) = h;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i == j + q) rest_a[i] = v[q] - (float)h[q];
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (uint32_t c0 = 0; c0 < 64; c0 += 32) {
            const f16x8 left = along(A, m_at(i, c0 + 8 * g));
#pragma unroll
            for (int t = 0; t < 2; ++t)
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(along(A, m_at((tj0 + t) * 16 + r, c0 + 8 * g)), left, acc[t], 0, 0, 0);
        }
        const float rest_i = rest_a[i], low = low_of(step + 1, steps);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t j = (tj0 + t) * 16 + g * 4;
            const f32x4 m = __builtin_convertvector(*reinterpret_cast<const f16x4*>(A + m_at(i, j)), f32x4);
            f32x4 v = p.c * (acc[t] + m * *reinterpret_cast<const f32x4*>(rest_a + j) + rest_i * m) + p.b * m;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i == j + q) v[q] += p.b * rest_i;
            const f16x4 h = __builtin_convertvector(v, f16x4);
            *reinterpret_cast<f16x4*>(P + m_at(i, j)) = h;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i == j + q) {
                    rest_p[i] = v[q] - (float)h[q];
                    diagonal[i] = low * (float)h[q];
                }
        }
        __syncthreads();
        const bool last = step + 1 == steps;
        f16x8 right[4][2];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) right[t][h] = along(P, m_at(t * 16 + r, h * 32 + 8 * g));
        // every wave its own rows of Y, which no other one reads here
        for (uint32_t part = wave; part < L / 16; part += 8) {
            const uint32_t row = part * 16 + r;
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f16x8 left = along(hi, y_at(row, h * 32 + 8 * g));
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(right[t][h], left, acc[t], 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t j = t * 16 + g * 4, at = y_at(row, j);
                const f32x4 v = stepped(acc[t], p.a + *reinterpret_cast<const f32x4*>(rest_p + j), *reinterpret_cast<const f32x4*>(diagonal + j),
                                        *reinterpret_cast<const f16x4*>(hi + at), *reinterpret_cast<const f16x4*>(lo + at));
                if (!last) {
                    const f16x4 h = __builtin_convertvector(v, f16x4);
                    *reinterpret_cast<f16x4*>(hi + at) = h;
                    *reinterpret_cast<f16x4*>(lo + at) = remainder<f16x4>(v, h);
                } else {
                    __bf16* out = p.out + (uint64_t)blockIdx.x * size;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t a = OVER ? j + q : row, b = OVER ? row : j + q;
                        if (a < p.n && b < p.k) out[a * p.k + b] = (__bf16)(v[q] * p.inverse);
                    }
                }
            }
        }
        __syncthreads();
    }
#endif
}

template <typename T, bool OVER>
zc_status launch_small(const OrthArgs& a, uint32_t steps, hipStream_t stream) {
    const uint32_t bytes = small_lds(a.length);
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(update_small<T, OVER>), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)bytes) != hipSuccess) {
        (void)hipGetLastError();  // reported here, not by the next launch
        return ZC_ERR_HIP;
    }
    hipLaunchKernelGGL((update_small<T, OVER>), dim3(a.batch), dim3(512), bytes, stream, a, steps);
    return ZC_OK;
}
static_assert(small_lds(kSmallLength) + 64 <= 160 * 1024, "Y, A and P in one CU's LDS");

uint64_t tiles_of(const OrthArgs& a, int kind, uint32_t t) {
    const uint64_t side = (a.side + t - 1) / t, length = (a.length + t - 1) / t;
    return kind <= kMix ? side * (side + 1) / 2 : side * length;
}

// Which tiles.  Wide ones read least from LDS but are one to a CU, so that their
// stores stand beside no other tile's products, and their rounds end late where
// they hardly fill the CUs.  A round of tiles takes about per_sum hundredths of
// the summed length and a fixed part, in units of what 256 x 256 tiles take for
// one of it.  Measured, in us, at 256 / 128 / 64 wide:
//   A^2   of 32 x 2048 384/394/541, 1 x 4096 93/105/160, 37 x 1024 89/64/77, 4 x 1408 48/26/25,
//         1 x 1024 42/18/10, 128 x 128 23/12/8
//   Y^T Y of 32 x 7168 x 2048 914/1043/2053, 37 x 1408 x 1024 85/85/110, 8 x 5056 x 640 92/49/28
//   Y P   of 32 x 7168 x 2048 2668/2796/3550, 1 x 14336 x 4096 502/528/734, 37 x 1408 x 1024
//         239/227/278, 8 x 5056 x 640 104/89/94, 1 x 2048 x 2048 56/30/31
uint32_t tile_side(const OrthArgs& a, int kind) {
    const bool symmetric = kind <= kMix;
    const uint64_t sum = kind == kGram ? a.length : a.side;
    auto cost = [&](uint32_t t, uint32_t on_cu, uint64_t per_sum, uint64_t fixed) {
        const uint64_t tiles = a.batch * tiles_of(a, kind, t), at_once = 256 * on_cu;
        return (tiles + at_once - 1) / at_once * (per_sum * sum / 100 + fixed);
    };
    const bool alone = a.batch * tiles_of(a, kind, 128) <= 256;
    const uint64_t wide = cost(256, 1, 100, symmetric ? 400 : 1000), mid = cost(128, 2, alone ? 53 : 62, symmetric ? 150 : 450),
                   small = cost(64, 2, 29, symmetric ? 100 : 200);
    return wide <= mid && wide <= small ? 256 : mid <= small ? 128 : 64;
}

template <typename SH, int KIND, bool OVER>
zc_status enqueue_product(const OrthArgs& a, hipStream_t stream) {
    const auto kernel = step_product<SH, KIND, OVER>;
    const uint64_t tiles = tiles_of(a, KIND, SH::kSide), side = (a.side + SH::kSide - 1) / SH::kSide;
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, SH::kLds) != hipSuccess) {
        (void)hipGetLastError();  // reported here, not by the next launch
        return ZC_ERR_HIP;
    }
    const uint64_t grid = (tiles * a.batch + 7) / 8 * 8;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(256), SH::kLds, stream, a, (uint32_t)tiles, (uint32_t)side);
    return ZC_OK;
}

template <int KIND, bool OVER = false>
zc_status product_of(const OrthArgs& a, hipStream_t stream) {
    const uint32_t side = tile_side(a, KIND);
    if (side == 256) return enqueue_product<Shape<8, 2>, KIND, OVER>(a, stream);
    if (side == 128) return enqueue_product<Shape<4, 2>, KIND, OVER>(a, stream);  // two workgroups on a CU
    return enqueue_product<Shape<2, 4>, KIND, OVER>(a, stream);
}

template <typename T>
void prepare(const OrthArgs& a, bool over, hipStream_t stream) {
    hipLaunchKernelGGL(squares<T>, dim3(a.parts * a.batch), dim3(256), 0, stream, a);
    const uint32_t cols = (a.k + 63) / 64, tiles = (a.n + 63) / 64 * cols;
    if (over) hipLaunchKernelGGL((normalize<T, true>), dim3(tiles, a.batch), dim3(256), 0, stream, a, cols);
    else hipLaunchKernelGGL((normalize<T, false>), dim3(tiles, a.batch), dim3(256), 0, stream, a, cols);
}

// Whether two steps are taken at once where another one follows: from this side
// on (below it their roundings average out less), and where Y is long enough
// that the three products of side x side more cost less than one Y^T Y and one
// Y P.  One step twice against both at once, us: 37 x 1408 x 1024 778/653, 32 x 7168
// x 2048 7930/5650; but 4 x 2048 x 1408 212/210, 1 x 4096 x 4096 604/690.
bool in_pairs(const OrthArgs& a) { return a.side >= 512 && 8ull * a.length >= 11ull * a.side; }

// Makes gamma M N + alpha M + beta N of the matrices m and n as the matrix `to`.
zc_status mix(OrthArgs& a, int m, int n, int to, float gamma, float alpha, float beta, hipStream_t stream) {
    a.matrix = a.square[m];
    a.other = a.square[n];
    a.made = a.square[to];
    a.rest_m = a.rest[m];
    a.rest_n = a.rest[n];
    a.rest_made = a.rest[to];
    a.gamma = gamma;
    a.alpha = alpha;
    a.beta = beta;
    return m == n ? product_of<kSquare>(a, stream) : product_of<kMix>(a, stream);
}

// The matrix by which one step, or two, go from Y to factor Y + Y M.  Of two:
//   B = b A + c A^2, T = a A + B A, A' = a T + T B  (that is (a + B) A (a + B), the
//   A of the step between), B' = b A' + c A'^2,
//   (a + B) (a + B') = a^2 + M, M = B' B + a B' + a B,
// so that Y is read and written once for both.  All of these are polynomials of
// A, which commute and are symmetric.
zc_status step_matrix(OrthArgs& a, bool two, int& m, hipStream_t stream) {
    a.matrix = a.other = nullptr;
    a.made = a.square[0];
    a.rest_made = a.rest[0];
    if (zc_status e = product_of<kGram>(a, stream)) return e;
    a.factor = a.a;
    m = 1;
    if (zc_status e = mix(a, 0, 0, 1, a.c, a.b, 0, stream)) return e;         // B
    if (!two) return ZC_OK;
    a.factor = a.a * a.a;
    m = 0;
    if (zc_status e = mix(a, 1, 0, 2, 1, 0, a.a, stream)) return e;           // T
    if (zc_status e = mix(a, 2, 1, 0, 1, a.a, 0, stream)) return e;           // A'
    if (zc_status e = mix(a, 0, 0, 2, a.c, a.b, 0, stream)) return e;         // B'
    return mix(a, 2, 1, 0, 1, a.a, a.a, stream);                              // M
}

}  // namespace

zc_status launch_orthogonalize(OrthArgs a, uint32_t dtype, uint32_t steps, hipStream_t stream) {
    // more workgroups than a launch may have, with the smallest tiles, in eights
    if (!fits(((uint64_t)a.batch * (a.length / 64) * (a.side / 64) + 7) / 8 * 8)) return ZC_ERR_UNSUPPORTED;
    const bool over = a.n < a.k;
    if (a.side == 64 && a.length <= kSmallLength) {
        auto small = [&](auto t) {
            typedef decltype(t) T;
            return over ? launch_small<T, true>(a, steps, stream) : launch_small<T, false>(a, steps, stream);
        };
        return dtype == ZC_BF16 ? small((__bf16)0.0f) : dtype == ZC_FP16 ? small((_Float16)0.0f) : small(0.0f);
    }
    _Float16 *from = a.hi_a, *to = a.hi_b;
    a.next = from;
    if (dtype == ZC_BF16) prepare<__bf16>(a, over, stream);
    else if (dtype == ZC_FP16) prepare<_Float16>(a, over, stream);
    else prepare<float>(a, over, stream);
    for (uint32_t s = 0; s < steps;) {
        const bool two = in_pairs(a) && s + 2 < steps;
        int m;
        a.hi = from;
        a.next = to;
        if (zc_status e = step_matrix(a, two, m, stream)) return e;
        a.matrix = a.square[m];
        a.rest_m = a.rest[m];
        s += two ? 2 : 1;
        a.low = low_of(s, steps);
        if (s == steps) return over ? product_of<kLast, true>(a, stream) : product_of<kLast>(a, stream);
        if (zc_status e = product_of<kApply>(a, stream)) return e;
        std::swap(from, to);
    }
    return ZC_OK;
}

}  // namespace zc
