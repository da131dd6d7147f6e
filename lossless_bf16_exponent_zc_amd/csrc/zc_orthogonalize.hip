// zc_orthogonalize.hip -- updates made orthogonal by Newton-Schulz products.
//
//   X <- x / (|x| + eps);   steps times:  A = X X^T,  P = b A + c A^2,
//                                         X <- a X + P X
// with X of more rows than columns: A = X^T X and X <- a X + X P, so that A and
// P are of the shorter side and no matrix is ever transposed in memory.
//
// Numbers.  The products run on v_mfma_f32_16x16x32_f16.  Their factors are
// fp16, 11 bits at bf16's rate: with bf16 factors results are off by 1e-2 of
// their rms and more.  X itself is kept as a pair hi + lo of fp16 (22 bits), of
// which the products read hi: a step multiplies a small singular value by up to
// a, five of them by 485, and with them what X was rounded by, while errors of
// the products' factors stay where A is large.  (Off from 64 bits by, in the
// root mean square: Gaussian 512 x 1792 1.1e-3, spectrum 1/i^2 2e-4, rank one
// and rounding noise 2e-4; without lo 1.5e-3, 2e-2, 1e-1.  The result's own
// rounding to bf16 is 1.7e-3.)  Near the end A and P are nearly diagonal, and
// what their diagonals were rounded by is the largest error left; it is kept
// in 32 bits and put back where P and the new X are made.
// X is held times 2^shift, about the square root of its longer side, so that
// its elements lie in fp16's normal range.
#include "zc_experts_kernels.h"

#include <type_traits>

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

// One operand of a product, result[i][j] = sum over c of left[i,c] right[j,c]:
// rows of fp16 with c along them, or (ACROSS) with c from row to row and i or j
// along them.
struct Operand {
    const uint8_t* p;  // its first element of the tile
    uint32_t stride;   // bytes between rows
    uint32_t count;    // of i or j that exist from there on, a multiple of 64
};

#if defined(__HIP_DEVICE_COMPILE__)

typedef __attribute__((address_space(3))) void lds_void;
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

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

// How an operand's stage lies in LDS.  Along: 128 bytes a row, piece c (16
// bytes) at place c ^ (row / 2 % 8), so that the 16 lanes that a 16-byte read
// takes at a time find 16 places of the 64 banks.  Across: kSide values a row
// of c, 64 rows; pairs of pieces (32 bytes) turned by the row, so that the
// eight rows that half a wave reads 32 bytes of lie in all banks.
template <typename SH, bool ACROSS>
struct Layout {
    static constexpr uint32_t kRow = ACROSS ? SH::kSide * 2 : 128;  // bytes
    static __device__ __forceinline__ uint32_t turn(uint32_t row) {
        if (!ACROSS) return (row >> 1) & 7;
        return SH::kSide == 64 ? (((row >> 1) & 1) | ((row >> 2) & 2)) * 2 : ((row & 3) | ((row >> 1) & 4)) * 2;
    }
    // what lane `lane` of load `index` of the stage brings: the offset from the
    // operand's first element
    static __device__ __forceinline__ uint32_t source(uint32_t index, uint32_t lane, const Operand& o) {
        const uint32_t at = index * 1024 + lane * 16, row = at / kRow, piece = (at % kRow / 16) ^ turn(row);
        if (ACROSS) return row * o.stride + (piece * 8 < o.count ? piece : o.count / 8 - 1) * 16;
        return (row < o.count ? row : o.count - 1) * o.stride + piece * 16;
    }
};

// Reads part t (16 of i or j from `first` + 16 t on) of a stage.
template <typename SH, bool ACROSS>
struct Reader {
    typedef Layout<SH, ACROSS> L;
    uint32_t at, turned, first;
    __device__ __forceinline__ Reader(uint32_t operand, uint32_t first_) : first(first_) {
        const uint32_t lane = __lane_id(), r = lane & 15, g = lane >> 4;
        if (ACROSS) {
            // lane 4 q + p of a group reads columns 4 p to 4 p + 3 of row q; the
            // instruction turns the group's 4 x 16 values over
            const uint32_t row = 8 * g + (r >> 2);
            at = operand + row * L::kRow + (r & 3) * 8;
            turned = L::turn(row) << 4;
        } else {
            at = operand + (first + r) * 128 + ((g ^ L::turn(r)) << 4);
            turned = 0;
        }
    }
    __device__ __forceinline__ Part read(const uint8_t* stage, int t) const {
        Part x;
        if (ACROSS) {
            const uint8_t* p = stage + at + ((first * 2 + t * 32) ^ turned);
            i16x4 q[4];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                q[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + ((h >> 1) * 32 + (h & 1) * 4) * L::kRow));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x.v[h] = __builtin_bit_cast(f16x8, __builtin_shufflevector(q[2 * h], q[2 * h + 1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            x.v[0] = *reinterpret_cast<const f16x8*>(stage + at + t * 2048);
            x.v[1] = *reinterpret_cast<const f16x8*>(stage + (at ^ 64) + t * 2048);
        }
        return x;
    }
};

// acc[ti][tj] += the products of a tile, over `blocks` blocks of 64.  A lane
// then has, of part (ti, tj), row ti * 16 + (lane & 15) and the four columns
// from tj * 16 + (lane >> 4) * 4 on.
template <typename SH, bool LEFT_ACROSS, bool RIGHT_ACROSS>
__device__ __forceinline__ void tile_product(const Operand& left, const Operand& right, uint32_t blocks, uint8_t* lds,
                                             f32x4 (&acc)[SH::T][SH::T]) {
    constexpr int T = SH::T, E = SH::kEach;
    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6);
    uint32_t at_l[E], at_r[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        at_l[i] = Layout<SH, LEFT_ACROSS>::source(wave * E + i, lane, left);
        at_r[i] = Layout<SH, RIGHT_ACROSS>::source(wave * E + i, lane, right);
    }
    const uint64_t step_l = LEFT_ACROSS ? 64ull * left.stride : 128, step_r = RIGHT_ACROSS ? 64ull * right.stride : 128;
    auto load_one = [&](int n, uint32_t block, uint8_t* stage) {
        if (n < E)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(left.p + block * step_l), (lds_void*)(stage + (wave * E + n) * 1024),
                                                     16, at_l[n], 0, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(right.p + block * step_r),
                                                     (lds_void*)(stage + SH::kOperand + (wave * E + n - E) * 1024), 16,
                                                     at_r[n - E], 0, 0, 0);
    };
    const Reader<SH, LEFT_ACROSS> rl(0, (wave >> 1) * T * 16);
    const Reader<SH, RIGHT_ACROSS> rr(SH::kOperand, (wave & 1) * T * 16);

    for (uint32_t s = 0; s < SH::S && s < blocks; ++s) {
#pragma unroll
        for (int n = 0; n < SH::kLoads; ++n) load_one(n, s, lds + s * SH::kStage);
    }
    if (blocks >= SH::S) wait_loads_and_barrier<(SH::S - 1) * SH::kLoads>();
    else wait_loads_and_barrier<0>();
    uint8_t* stage = lds;
    Part right_part[T], next = rl.read(stage, 0);
#pragma unroll
    for (int j = 0; j < T; ++j) right_part[j] = rr.read(stage, j);

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
            for (int n = 1 + i * kAhead; n < 1 + (i + 1) * kAhead && n < T; ++n) l[n] = rl.read(stage, n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < T; ++j) multiply(acc[i][j], right_part[j], l[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (HALF == 0) l[1] = rl.read(stage, 1);
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
        next = rl.read(stage, 0);
#pragma unroll
        for (int j = 0; j < T; ++j) {
            multiply(acc[T - 2][j], right_part[j], l[T - 2]);
            multiply(acc[T - 1][j], right_part[j], l[T - 1]);
            right_part[j] = rr.read(stage, j);
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

// Tile `index` of the lower triangle, row by row.
struct Place {
    uint32_t i, j;
};
__device__ __forceinline__ Place lower(uint32_t index) {
    uint32_t i = (uint32_t)((sqrtf(8.0f * (float)index + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > index) --i;
    while ((i + 1) * (i + 2) / 2 <= index) ++i;
    return Place{i, index - i * (i + 1) / 2};
}

#endif  // __HIP_DEVICE_COMPILE__

template <typename SH, int KIND, bool TALL>
__global__ __launch_bounds__(256, SH::T == 8 ? 1 : 2) void step_product(OrthArgs p, uint32_t tiles, uint32_t col_tiles) {
    extern __shared__ __align__(16) uint8_t lds[];
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr bool SYMMETRIC = KIND == kGram || KIND == kSquare;
    constexpr int T = SH::T;
    const uint32_t matrix = blockIdx.x / tiles, index = blockIdx.x % tiles;
    const Place at = SYMMETRIC ? lower(index) : Place{index / col_tiles, index % col_tiles};
    const uint32_t i0 = at.i * SH::kSide, j0 = at.j * SH::kSide;
    const uint64_t x_at = (uint64_t)matrix * p.rows * p.cols, s_at = (uint64_t)matrix * p.side * p.side;
    const _Float16 *hi = p.hi + x_at, *A = p.gram + s_at, *P = p.poly + s_at;
    f32x4 acc[T][T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    auto rows_of = [](const _Float16* m, uint32_t from, uint32_t rows, uint32_t stride) {
        return Operand{reinterpret_cast<const uint8_t*>(m + (uint64_t)from * stride), stride * 2, rows - from};
    };
    auto cols_of = [](const _Float16* m, uint32_t from, uint32_t cols) {
        return Operand{reinterpret_cast<const uint8_t*>(m + from), cols * 2, cols - from};
    };
    if constexpr (KIND == kGram && TALL)
        tile_product<SH, true, true>(cols_of(hi, i0, p.cols), cols_of(hi, j0, p.cols), p.rows / 64, lds, acc);
    else if constexpr (KIND == kGram)
        tile_product<SH, false, false>(rows_of(hi, i0, p.rows, p.cols), rows_of(hi, j0, p.rows, p.cols), p.cols / 64, lds, acc);
    else if constexpr (KIND == kSquare)
        tile_product<SH, false, false>(rows_of(A, i0, p.side, p.side), rows_of(A, j0, p.side, p.side), p.side / 64, lds, acc);
    else if constexpr (TALL)
        tile_product<SH, false, false>(rows_of(hi, i0, p.rows, p.cols), rows_of(P, j0, p.side, p.side), p.side / 64, lds, acc);
    else
        tile_product<SH, false, true>(rows_of(P, i0, p.side, p.side), cols_of(hi, j0, p.cols), p.side / 64, lds, acc);

    const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t ri = i0 + (wave >> 1) * T * 16 + r, rj = j0 + (wave & 1) * T * 16 + g * 4;
    const uint32_t end_i = SYMMETRIC ? p.side : p.rows, end_j = SYMMETRIC ? p.side : p.cols;
    if constexpr (SYMMETRIC) {
        _Float16* out = (KIND == kGram ? p.gram : p.poly) + s_at;
        float* left_over = (KIND == kGram ? p.gram_rest : p.poly_rest) + (uint64_t)matrix * p.side;
        const float* rest = p.gram_rest + (uint64_t)matrix * p.side;
#pragma unroll
        for (int ti = 0; ti < T; ++ti) {
            const uint32_t i = ri + ti * 16;
            if (i - r >= end_i) break;  // whole parts: sides are multiples of 64
            const float rest_i = KIND == kSquare ? rest[i] : 0.0f;
#pragma unroll
            for (int tj = 0; tj < T; ++tj) {
                const uint32_t j = rj + tj * 16;
                if (j - g * 4 >= end_j) break;
                f32x4 v = late(acc[ti][tj]);
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
                const f16x4 h = __builtin_convertvector(v, f16x4);
                *reinterpret_cast<f16x4*>(out + (uint64_t)i * p.side + j) = h;
                if (at.i != at.j) {
                    const f16x4 o = turned_over(h);
                    *reinterpret_cast<f16x4*>(out + (uint64_t)(j + (r & 3)) * p.side + (i - (r & 3))) = o;
                } else if (i - j < 4) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (i == j + q) left_over[i] = v[q] - (float)h[q];
                }
            }
        }
    } else {
        const float* rest = p.poly_rest + (uint64_t)matrix * p.side;
#pragma unroll
        for (int ti = 0; ti < T; ++ti) {
            const uint32_t i = ri + ti * 16;
            if (i - r >= end_i) break;
            const float factor_i = p.a + (TALL ? 0.0f : rest[i]);
#pragma unroll
            for (int tj = 0; tj < T; ++tj) {
                const uint32_t j = rj + tj * 16;
                if (j - g * 4 >= end_j) break;
                const uint64_t e = (uint64_t)i * p.cols + j;
                const f16x4 h = *reinterpret_cast<const f16x4*>(hi + e), l = *reinterpret_cast<const f16x4*>(p.lo + x_at + e);
                f32x4 factor = {factor_i, factor_i, factor_i, factor_i};
                if (TALL) factor += *reinterpret_cast<const f32x4*>(rest + j);
                const f32x4 was = __builtin_convertvector(h, f32x4) + __builtin_convertvector(l, f32x4);
                const f32x4 v = factor * was + late(acc[ti][tj]);
                if constexpr (KIND == kApply) {
                    const f16x4 nh = __builtin_convertvector(v, f16x4);
                    *reinterpret_cast<f16x4*>(p.next + x_at + e) = nh;
                    *reinterpret_cast<f16x4*>(p.lo + x_at + e) = __builtin_convertvector(v - __builtin_convertvector(nh, f32x4), f16x4);
                } else if (i < p.n) {
                    __bf16* out = p.out + ((uint64_t)matrix * p.n + i) * p.k + j;
                    struct Four {
                        __bf16 v[4];
                    };
                    const Four o{{(__bf16)(v[0] * p.inverse), (__bf16)(v[1] * p.inverse), (__bf16)(v[2] * p.inverse),
                                  (__bf16)(v[3] * p.inverse)}};
                    if (j + 4 <= p.k) {
                        *reinterpret_cast<Four*>(out) = o;
                    } else {
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            if (j + q < p.k) out[q] = o.v[q];
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

// X = x / (|x| + eps) times 2^shift, as hi and lo, with zeros up to multiples
// of 64 rows and columns.  grid: (pieces of 8 values, matrices).
template <typename T>
__global__ __launch_bounds__(256) void normalize(OrthArgs p) {
    __shared__ double factor;
    const uint32_t matrix = blockIdx.y;
    if (threadIdx.x < 64) {
        double s = threadIdx.x < p.parts ? p.part[matrix * p.parts + threadIdx.x] : 0.0;
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        const double size = sqrt(s) + (double)p.eps;
        if (threadIdx.x == 0) factor = size == 0.0 ? 0.0 : (double)p.scale / size;
    }
    __syncthreads();
    const double f = factor;
    const T* x = static_cast<const T*>(p.x) + (uint64_t)matrix * p.n * p.k;
    const uint32_t each = p.cols / 8;
    const uint64_t pieces = (uint64_t)p.rows * each, x_at = (uint64_t)matrix * p.rows * p.cols;
    for (uint64_t w = blockIdx.x * 256ull + threadIdx.x; w < pieces; w += gridDim.x * 256ull) {
        const uint32_t i = (uint32_t)(w / each), j = (uint32_t)(w % each) * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.0f;
        if (i < p.n && j < p.k) {
            const int32_t left = (int32_t)(p.k - j);
            constexpr int kEach = 16 / sizeof(T);
            T t[8];
#pragma unroll
            for (int q = 0; q < 8; q += kEach) {
                const xu32x4 word = load_word(x + (uint64_t)i * p.k + j + q, left - q < kEach ? left - q : kEach);
                __builtin_memcpy(t + q, &word, 16);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = (float)((double)to_float(t[q]) * f);
        }
        f16x8 hi, lo;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            hi[q] = (_Float16)v[q];
            lo[q] = (_Float16)(v[q] - (float)hi[q]);
        }
        *reinterpret_cast<f16x8*>(p.next + x_at + w * 8) = hi;
        *reinterpret_cast<f16x8*>(p.lo + x_at + w * 8) = lo;
    }
}

template <typename SH, int KIND, bool TALL>
zc_status enqueue_product(const OrthArgs& a, hipStream_t stream) {
    const auto kernel = step_product<SH, KIND, TALL>;
    const bool symmetric = KIND == kGram || KIND == kSquare;
    const uint64_t rows = ((symmetric ? a.side : a.rows) + SH::kSide - 1) / SH::kSide;
    const uint64_t cols = ((symmetric ? a.side : a.cols) + SH::kSide - 1) / SH::kSide;
    const uint64_t tiles = symmetric ? rows * (rows + 1) / 2 : rows * cols;
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, SH::kLds) != hipSuccess) {
        (void)hipGetLastError();  // reported here, not by the next launch
        return ZC_ERR_HIP;
    }
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(tiles * a.batch)), dim3(256), SH::kLds, stream, a, (uint32_t)tiles, (uint32_t)cols);
    return ZC_OK;
}

template <int KIND>
zc_status product_of(const OrthArgs& a, bool tall, hipStream_t stream) {
    typedef Shape<4, 2> Mid;
    return tall ? enqueue_product<Mid, KIND, true>(a, stream) : enqueue_product<Mid, KIND, false>(a, stream);
}

template <typename T>
void prepare(const OrthArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(squares<T>, dim3(a.parts * a.batch), dim3(256), 0, stream, a);
    const uint64_t pieces = (uint64_t)a.rows * a.cols / 8, groups = (pieces + 255) / 256, most = 4096 / a.batch + 1;
    hipLaunchKernelGGL(normalize<T>, dim3((uint32_t)(groups < most ? groups : most), a.batch), dim3(256), 0, stream, a);
}

}  // namespace

zc_status launch_orthogonalize(OrthArgs a, uint32_t dtype, uint32_t steps, hipStream_t stream) {
    // more workgroups than a launch may have, with the smallest tiles
    if (!fits((uint64_t)a.batch * ((a.rows + 63) / 64) * ((a.cols + 63) / 64))) return ZC_ERR_UNSUPPORTED;
    const bool tall = a.n > a.k;
    _Float16 *from = a.hi_a, *to = a.hi_b;
    a.next = from;
    if (dtype == ZC_BF16) prepare<__bf16>(a, stream);
    else if (dtype == ZC_FP16) prepare<_Float16>(a, stream);
    else prepare<float>(a, stream);
    for (uint32_t s = 0; s < steps; ++s) {
        a.hi = from;
        a.next = to;
        if (zc_status e = product_of<kGram>(a, tall, stream)) return e;
        if (zc_status e = product_of<kSquare>(a, tall, stream)) return e;
        if (s + 1 == steps) return product_of<kLast>(a, tall, stream);
        if (zc_status e = product_of<kApply>(a, tall, stream)) return e;
        from = a.next;
        to = const_cast<_Float16*>(a.hi);
    }
    return ZC_OK;
}

}  // namespace zc
