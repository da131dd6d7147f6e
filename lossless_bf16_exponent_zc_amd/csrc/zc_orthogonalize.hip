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
// their rms and more.  Y itself is kept as a pair hi + lo of fp16 (22 bits), of
// which the products read hi: a step multiplies a small singular value by up to
// a, five of them by 485, and with them what Y was rounded by, while errors of
// the products' factors stay where A is large.  (Off from 64 bits by, in the
// root mean square: Gaussian 512 x 1792 1.1e-3, spectrum 1/i^2 2e-4, rank one
// and rounding noise 2e-4; without lo 1.5e-3, 2e-2, 1e-1.  The result's own
// rounding to bf16 is 1.7e-3.)  Near the end A and P are nearly diagonal, and
// what their diagonals were rounded by is the largest error left; it is kept
// in 32 bits and put back where P and the new Y are made.
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

enum Product { kGram, kSquare, kApply, kLast };

// Tiles of kSide x kSide by four waves, 2 x 2, each T x T instruction tiles of
// 16 x 16; S stages of 64 of the summed dimension in LDS.
template <int T_, int S_>
struct Shape {
    static constexpr int T = T_, S = S_;
    static constexpr int kSide = 32 * T;
    static constexpr int kOperand = kSide * 128;   // bytes of one operand's stage
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kEach = kSide / 32;       // loads per wave, operand and stage
    static constexpr int kLoads = 2 * kEach;
    static constexpr int kLds = S * kStage;
};

// One operand of a product, result[i][j] = sum over c of left[i][c] right[j][c].
struct Operand {
    const uint8_t* p;  // first row of the tile
    uint32_t stride;   // bytes between rows
    uint32_t rows;     // that exist from there on
};

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

// Piece c (16 bytes) of a row lies at place c ^ turn(row) of its 128 bytes, so
// that the 16 lanes that a 16-byte read takes at a time find 16 places of the
// 64 banks.
__device__ __forceinline__ uint32_t turn(uint32_t row) { return (row >> 1) & 7; }

// acc[ti][tj] += the products of a tile, over `blocks` blocks of 64.  A lane
// then has, of part (ti, tj), row ti * 16 + (lane & 15) and the four columns
// from tj * 16 + (lane >> 4) * 4 on.
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
    const uint32_t lo_l = ((wave >> 1) * T * 16 + r) * 128 + ((g ^ turn(r)) << 4);
    const uint32_t lo_r = SH::kOperand + ((wave & 1) * T * 16 + r) * 128 + ((g ^ turn(r)) << 4);
    auto read = [&](const uint8_t* stage, uint32_t lo, int t) {
        return Part{{*reinterpret_cast<const f16x8*>(stage + lo + t * 2048), *reinterpret_cast<const f16x8*>(stage + (lo ^ 64) + t * 2048)}};
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

// OVER: the result leaves turned over (kLast).
template <typename SH, int KIND, bool OVER>
__global__ __launch_bounds__(256, SH::T == 8 ? 1 : 2) void step_product(OrthArgs p, uint32_t tiles, uint32_t side_tiles) {
    extern __shared__ __align__(16) uint8_t lds[];
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr bool SYMMETRIC = KIND == kGram || KIND == kSquare;
    constexpr int T = SH::T;
    const uint32_t place = of_run(blockIdx.x, gridDim.x >> 3), matrix = place / tiles, index = place % tiles;
    if (matrix >= p.batch) return;
    const Place at = SYMMETRIC ? lower(index) : banded(index, tiles / side_tiles, side_tiles);
    const uint32_t i0 = at.i * SH::kSide, j0 = at.j * SH::kSide;
    const uint64_t y_at = (uint64_t)matrix * p.length * p.side, s_at = (uint64_t)matrix * p.side * p.side;
    const _Float16 *hi = p.hi + y_at, *across = p.across + y_at, *A = p.gram + s_at, *P = p.poly + s_at;
    f32x4 acc[T][T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    auto rows_of = [](const _Float16* m, uint32_t from, uint32_t rows, uint32_t stride) {
        return Operand{reinterpret_cast<const uint8_t*>(m + (uint64_t)from * stride), stride * 2, rows - from};
    };
    if constexpr (KIND == kGram)
        tile_product<SH>(rows_of(across, i0, p.side, p.length), rows_of(across, j0, p.side, p.length), p.length / 64, lds, acc);
    else if constexpr (KIND == kSquare)
        tile_product<SH>(rows_of(A, i0, p.side, p.side), rows_of(A, j0, p.side, p.side), p.side / 64, lds, acc);
    else
        tile_product<SH>(rows_of(hi, i0, p.length, p.side), rows_of(P, j0, p.side, p.side), p.side / 64, lds, acc);

    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4, q4 = r & 3;
    const uint32_t ri = i0 + (wave >> 1) * T * 16 + r, rj = j0 + (wave & 1) * T * 16 + g * 4;
    const uint32_t end_i = SYMMETRIC ? p.side : p.length;
    const float* rest = (KIND == kSquare ? p.gram_rest : p.poly_rest) + (uint64_t)matrix * p.side;
#pragma unroll
    for (int ti = 0; ti < T; ++ti) {
        const uint32_t i = ri + ti * 16;
        if (i - r >= end_i) break;  // whole parts: side and length are multiples of 64
        const float rest_i = KIND == kSquare ? rest[i] : 0.0f;
#pragma unroll
        for (int tj = 0; tj < T; ++tj) {
            const uint32_t j = rj + tj * 16;
            if (j - g * 4 >= p.side) break;
            f32x4 v = late(acc[ti][tj]);
            if constexpr (SYMMETRIC) {
                if constexpr (KIND == kGram) {
                    v *= p.inverse_square;
                } else {
                    const f16x4 was = *reinterpret_cast<const f16x4*>(A + (uint64_t)i * p.side + j);
                    const f32x4 rest_j = *reinterpret_cast<const f32x4*>(rest + j);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[q] = (float)was[q] * (p.b + p.c * (rest_i + rest_j[q])) + p.c * v[q];
                        if (i == j + q) v[q] += p.b * rest_i;
                    }
                }
                _Float16* out = (KIND == kGram ? p.gram : p.poly) + s_at;
                const f16x4 h = __builtin_convertvector(v, f16x4);
                *reinterpret_cast<f16x4*>(out + (uint64_t)i * p.side + j) = h;
                if (at.i != at.j) {
                    *reinterpret_cast<f16x4*>(out + (uint64_t)(j + q4) * p.side + (i - q4)) = turned_over(h);
                } else if (i - j < 4) {
                    float* left_over = (KIND == kGram ? p.gram_rest : p.poly_rest) + (uint64_t)matrix * p.side;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (i == j + q) left_over[i] = v[q] - (float)h[q];
                }
            } else {
                const uint64_t e = y_at + (uint64_t)i * p.side + j;
                const f16x4 h = *reinterpret_cast<const f16x4*>(p.hi + e), l = *reinterpret_cast<const f16x4*>(p.lo + e);
                const f32x4 factor = p.a + *reinterpret_cast<const f32x4*>(rest + j);
                v += factor * (__builtin_convertvector(h, f32x4) + __builtin_convertvector(l, f32x4));
                if constexpr (KIND == kApply) {
                    const f16x4 nh = __builtin_convertvector(v, f16x4);
                    *reinterpret_cast<f16x4*>(p.next + e) = nh;
                    *reinterpret_cast<f16x4*>(p.lo + e) = __builtin_convertvector(v - __builtin_convertvector(nh, f32x4), f16x4);
                    *reinterpret_cast<f16x4*>(p.across + y_at + (uint64_t)(j + q4) * p.length + (i - q4)) = turned_over(nh);
                } else {
                    v *= p.inverse;
                    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                    bf16x4 o = __builtin_convertvector(v, bf16x4);
                    uint32_t row = i, col = j;
                    if (OVER) {
                        o = __builtin_bit_cast(bf16x4, turned_over(__builtin_bit_cast(f16x4, o)));
                        row = j + q4;
                        col = i - q4;
                    }
                    if (row < p.n) {
                        __bf16* out = p.out + ((uint64_t)matrix * p.n + row) * p.k + col;
                        struct Four {
                            __bf16 v[4];
                        };
                        if (col + 4 <= p.k) {
                            *reinterpret_cast<Four*>(out) = Four{{o[0], o[1], o[2], o[3]}};
                        } else {
#pragma unroll
                            for (int q = 0; q < 3; ++q)
                                if (col + q < p.k) out[q] = o[q];
                        }
                    }
                }
            }
        }
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
            straight_lo[q] = (_Float16)(v - (float)straight[q]);
            over[q] = (_Float16)t;
            over_lo[q] = (_Float16)(t - (float)over[q]);
        }
        const uint64_t at_s = y_at + (uint64_t)(i0 + a) * along + j0 + b * 8, at_o = y_at + (uint64_t)(j0 + a) * down + i0 + b * 8;
        *reinterpret_cast<f16x8*>((OVER ? p.across : p.next) + at_s) = straight;
        *reinterpret_cast<f16x8*>((OVER ? p.next : p.across) + at_o) = over;
        if (OVER) *reinterpret_cast<f16x8*>(p.lo + at_o) = over_lo;
        else *reinterpret_cast<f16x8*>(p.lo + at_s) = straight_lo;
    }
}

uint64_t tiles_of(const OrthArgs& a, int kind, uint32_t t) {
    const uint64_t side = (a.side + t - 1) / t, length = (a.length + t - 1) / t;
    return kind == kGram || kind == kSquare ? side * (side + 1) / 2 : side * length;
}

uint32_t tile_side(const OrthArgs& a, int kind) {
    if (a.batch * tiles_of(a, kind, 256) >= 256) return 256;
    if (a.batch * tiles_of(a, kind, 128) >= 256) return 128;
    return 64;
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

}  // namespace

zc_status launch_orthogonalize(OrthArgs a, uint32_t dtype, uint32_t steps, hipStream_t stream) {
    // more workgroups than a launch may have, with the smallest tiles
    if (!fits((uint64_t)a.batch * (a.length / 64) * (a.side / 64))) return ZC_ERR_UNSUPPORTED;
    const bool over = a.n < a.k;
    _Float16 *from = a.hi_a, *to = a.hi_b;
    a.next = from;
    if (dtype == ZC_BF16) prepare<__bf16>(a, over, stream);
    else if (dtype == ZC_FP16) prepare<_Float16>(a, over, stream);
    else prepare<float>(a, over, stream);
    for (uint32_t s = 0; s < steps; ++s) {
        a.hi = from;
        a.next = to;
        if (zc_status e = product_of<kGram>(a, stream)) return e;
        if (zc_status e = product_of<kSquare>(a, stream)) return e;
        if (s + 1 == steps) return over ? product_of<kLast, true>(a, stream) : product_of<kLast>(a, stream);
        if (zc_status e = product_of<kApply>(a, stream)) return e;
        std::swap(from, to);
    }
    return ZC_OK;
}

}  // namespace zc
