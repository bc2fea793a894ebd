// The product of two matrices of block-scaled e4m3 (dopt_fp8_gemm): out[m][n] (+)= sum over k of
// a[m][k] b[n][k].
//
// Four kernels, by plan_of: up to 16 rows of a (k_gemm_few), bound by the one reading of b; 128 x 128
// tiles (k_gemm_tile), bound by latency where tiles are few; 256 x 256 tiles (k_gemm_wide for sums in
// fp32, k_gemm_big for coarse ones), bound by the matrix cores, whose clock falls from 2.4 to 2.05 GHz, and by a tile's first
// loads and its stores, during which they wait.  Time per call of calls in a row on MI355X, where a library's bf16 product of
// these large sizes reaches 1.33 to 1.56 PFLOP/s, an e4m3 one without scales of blocks 2.5 to 3.1, and a copy 5.1 TB/s; ranges are over
// machines; in brackets dopt_fp8_gemm_coarse:
//   1 x 14336 x 4096              13.1 us, 4.5 TB/s                                   k_gemm_few
//   1024 x 2304 x 768             8.7 us (7.7)                                        k_gemm_tile, 3 stages
//   1024 x 4096 x 4096            32 to 36 us (20 to 22)                              k_gemm_tile, 3 stages
//   8192 x 14336 x 4096           649 to 687 us, 1.40 to 1.48 PFLOP/s (374 to 395)    k_gemm_wide (k_gemm_big)
//   8192 x 4096 x 14336           612 to 656 us, 1.47 to 1.57 PFLOP/s (347 to 361)    k_gemm_wide (k_gemm_big)
//   777 x 50257 x 768, fp32 out   94 to 95 us                                         k_gemm_tile, 2 stages: 40 us of them are the stores
//   4096 x 4096 x 8192, fp32 +=   201 to 213 us, 1.29 to 1.37 PFLOP/s                 k_gemm_wide
#include <algorithm>
#include <string>
#include <type_traits>

#include "fp8.h"

namespace dopt {

using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;

constexpr int kStep = DOPT_FP8_BLOCK;  // bytes of a row, and elements of k, per step

struct GemmArgs {
    const uint8_t *a, *b, *as, *bs;
    void *out;
    float *part;  // splits > 1: fp32 sums, [splits][m][part_ld]
    int64_t as_ld, bs_ld, out_ld, part_ld;
    int32_t a_ld, b_ld;
    int32_t m, n, steps;  // steps of 128 along k
    int32_t tiles_m, tiles_n, splits, split_steps;
    int32_t dtype, accumulate;
};

// ---- output -----------------------------------------------------------------------

template <int T>
__device__ __forceinline__ void put4_as(void *out, int64_t e, int n, f32x4 x, bool add) {
    if constexpr (T == DOPT_F32) {
        float *p = static_cast<float *>(out) + e;
        if (n >= 4) {
            Float4 *w = reinterpret_cast<Float4 *>(p);
            if (add) x += w->v;
            w->v = x;
        } else {
            for (int i = 0; i < n; ++i) p[i] = add ? p[i] + x[i] : x[i];
        }
    } else {
        uint16_t *p = static_cast<uint16_t *>(out) + e;
        if (n >= 4) {
            Bytes8 *w = reinterpret_cast<Bytes8 *>(p);
            if (add) {
                const u32x2 o = w->v;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] += to_float<T>(i % 2 ? o[i / 2] >> 16 : o[i / 2] & 0xffffu);
            }
            u32x2 r;
#pragma unroll
            for (int i = 0; i < 2; ++i) r[i] = from_float<T>(x[2 * i]) | from_float<T>(x[2 * i + 1]) << 16;
            w->v = r;
        } else {
            for (int i = 0; i < n; ++i) p[i] = static_cast<uint16_t>(from_float<T>(add ? to_float<T>(p[i]) + x[i] : x[i]));
        }
    }
}

// Elements [col, col + 4) of out's row, as far as they exist.
__device__ __forceinline__ void put4(const GemmArgs &A, int row, int col, f32x4 x) {
    if (row >= A.m || col >= A.n) return;
    const int64_t e = static_cast<int64_t>(row) * A.out_ld + col;
    const int n = A.n - col;
    if (A.dtype == DOPT_F32) put4_as<DOPT_F32>(A.out, e, n, x, A.accumulate);
    else if (A.dtype == DOPT_BF16) put4_as<DOPT_BF16>(A.out, e, n, x, A.accumulate);
    else put4_as<DOPT_F16>(A.out, e, n, x, A.accumulate);
}

// A wave's results, FI x FJ instructions of 16 x 16 from (m0, n0) on: in groups of 4, of
// which instruction i and j hold every fourth row and column from i and j on. Register
// v of a lane is row 4 * (lane / 16) + v of its 16, and column lane % 16. Four neighbours of a
// row are stored at once. Where they are added to out, 16 reads are under way at a time. The type
// and the bounds are told apart once for a tile: what it fetches is straight code for its own.
enum { kWholeTile, kWholeColumns, kRagged };

template <int T, bool ADD, int BOUNDS, int FI, int FJ>
__device__ __forceinline__ void store_as(const GemmArgs &A, int m0, int n0, const f32x4 (&acc)[FI][FJ]) {
    constexpr int ES = T == DOPT_F32 ? 4 : 2, H = FJ / 4, I = FI < 4 / H ? FI : 4 / H;
    const int lane = threadIdx.x % 64;
    const int row0 = m0 + 16 * (lane / 16), col0 = n0 + 4 * (lane % 16);
    const uint32_t of_lane = static_cast<uint32_t>(16 * (lane / 16)) * static_cast<uint32_t>(A.out_ld * ES) + 4u * ES * (lane % 16);
    char *out = static_cast<char *>(A.out) + (static_cast<int64_t>(m0) * A.out_ld + n0) * ES;
    using Four = std::conditional_t<T == DOPT_F32, Float4, Bytes8>;
    const auto delta = [](int i, int v) { return i / 4 * 64 + 4 * v + i % 4; };
    const auto place = [&](int i, int v, int h) { return out + delta(i, v) * A.out_ld * ES + 64 * h * ES + of_lane; };
    const auto row_in = [&](int i, int v) { return BOUNDS == kWholeTile || row0 + delta(i, v) < A.m; };
    const auto all_in = [&](int h) { return BOUNDS != kRagged || col0 + 64 * h + 4 <= A.n; };
#pragma unroll
    for (int i0 = 0; i0 < FI; i0 += I) {
        Four old[I][4][H];
        if constexpr (ADD) {
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        if (row_in(i0 + i, v) && all_in(h)) old[i][v][h] = *reinterpret_cast<const Four *>(place(i0 + i, v, h));
        }
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    if (!row_in(i0 + i, v)) continue;
                    const auto &c = acc[i0 + i];
                    f32x4 x = {c[4 * h][v], c[4 * h + 1][v], c[4 * h + 2][v], c[4 * h + 3][v]};
                    char *p = place(i0 + i, v, h);
                    if (!all_in(h)) {  // the last one to three columns, by one lane
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (col0 + 64 * h + e < A.n) {
                                if constexpr (T == DOPT_F32) {
                                    float *f = reinterpret_cast<float *>(p) + e;
                                    *f = ADD ? *f + x[e] : x[e];
                                } else {
                                    uint16_t *f = reinterpret_cast<uint16_t *>(p) + e;
                                    *f = static_cast<uint16_t>(from_float<T>(ADD ? to_float<T>(*f) + x[e] : x[e]));
                                }
                            }
                    } else if constexpr (T == DOPT_F32) {
                        if (ADD) x += old[i][v][h].v;
                        reinterpret_cast<Float4 *>(p)->v = x;
                    } else {
                        u32x2 r;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if constexpr (ADD) {
                                x[2 * e] += to_float<T>(old[i][v][h].v[e] & 0xffffu);
                                x[2 * e + 1] += to_float<T>(old[i][v][h].v[e] >> 16);
                            }
                            r[e] = from_float<T>(x[2 * e]) | from_float<T>(x[2 * e + 1]) << 16;
                        }
                        reinterpret_cast<Bytes8 *>(p)->v = r;
                    }
                }
    }
}

template <int T, bool ADD, int FI, int FJ>
__device__ __forceinline__ void store_bounded(const GemmArgs &A, int m0, int n0, const f32x4 (&acc)[FI][FJ]) {
    if (n0 + 16 * FJ > A.n) store_as<T, ADD, kRagged>(A, m0, n0, acc);
    else if (m0 + 16 * FI > A.m) store_as<T, ADD, kWholeColumns>(A, m0, n0, acc);
    else store_as<T, ADD, kWholeTile>(A, m0, n0, acc);
}

template <int T, int FI, int FJ>
__device__ __forceinline__ void store_typed(const GemmArgs &A, int m0, int n0, const f32x4 (&acc)[FI][FJ]) {
    if (A.accumulate) store_bounded<T, true>(A, m0, n0, acc);
    else store_bounded<T, false>(A, m0, n0, acc);
}

template <bool EXACT, int FI, int FJ>
__device__ __forceinline__ void store_tile(const GemmArgs &A, int m0, int n0, const f32x4 (&acc)[FI][FJ]) {
    if (EXACT && A.dtype == DOPT_F32) store_typed<DOPT_F32>(A, m0, n0, acc);
    else if (A.dtype == DOPT_BF16) store_typed<DOPT_BF16>(A, m0, n0, acc);
    else store_typed<DOPT_F16>(A, m0, n0, acc);
}

// A split's sums; rows of part are padded to 4.
__device__ __forceinline__ void put4_part(const GemmArgs &A, int split, int row, int col, f32x4 x) {
    if (row >= A.m || col >= A.n) return;
    *reinterpret_cast<f32x4 *>(A.part + (static_cast<int64_t>(split) * A.m + row) * A.part_ld + col) = x;
}

__global__ __launch_bounds__(256) void k_gemm_join(GemmArgs A) {
    const int per_row = static_cast<int>(A.part_ld / 4);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<int64_t>(A.m) * per_row) return;
    const int row = static_cast<int>(i / per_row), col = static_cast<int>(i % per_row) * 4;
    f32x4 x = {0, 0, 0, 0};
    for (int s = 0; s < A.splits; ++s)
        x += *reinterpret_cast<const f32x4 *>(A.part + (static_cast<int64_t>(s) * A.m + row) * A.part_ld + col);
    put4(A, row, col, x);
}

// ---- one step's products ------------------------------------------------------------

// Two ways to multiply, chosen by the caller.
//
// dopt_fp8_gemm (EXACT): the codes become bf16 with their scale applied (exact: 4
// bits of mantissa, and the scale is a power of two) in registers, and the bf16
// instruction multiplies, whose products and sums are fp32's (1e-7 of the result),
// at half the codes' rate.
//
// dopt_fp8_gemm_coarse: the matrix instruction that takes e4m3 codes and applies the
// scales itself.  It adds 8 neighbouring products of k with 14 bits below the
// largest of them, and such sums to one another and to the accumulator in
// fp32 (measured: a product 2^-14 of the largest in its 8 is lost, one 2^-23 of it in
// another 8 is kept).  On random operands a result is thereby off by 3 to 5e-5 of
// the output's root mean square, which moves one of 50 bf16 and one of 10 fp16 outputs by a
// step; where large products cancel, all that is left of the small ones next to them may be lost.  No other
// instruction takes e4m3 and adds more precisely: the one without scales, at half the rate, cuts the same.
//
// A lane holds 32 codes of row (lane % 16) of either operand; which of a step's 128
// does not matter as long as both take the same.
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The scale in byte I of a dword.
template <int I>
__device__ __forceinline__ float scale_of(int bytes) {
    return __uint_as_float((static_cast<uint32_t>(bytes) >> (8 * I) & 0xffu) << 23);
}

// c += a x b over 128 of k; a's and b's scales are byte I and J of a dword per lane.
template <int I, int J>
__device__ __forceinline__ f32x4 mfma(i32x8 a, i32x8 b, f32x4 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, I, sa, J, sb);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join(i32x4 lo, i32x4 hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

// f(0) to f(3) with numbers that the compiler knows, as the byte selectors have to be.
template <class F>
__device__ __forceinline__ void each4(const F &f) {
    f(std::integral_constant<int, 0>{});
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 3>{});
}

// ---- tiles ------------------------------------------------------------------------

__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)p));
}

// 16 (or 4) bytes per lane from base + offset to shared memory at `to` + 16 (4) * lane, past
// the registers.  The compiler does not know of the load: the kernel waits for it.  `base` comes
// from scalar arithmetic; written by a vector instruction it would need 5 cycles before the load.
__device__ __forceinline__ void load_lds16(uint32_t to, uint32_t offset, const uint8_t *base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds4(uint32_t to, uint32_t offset, const uint8_t *base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}

// Where workgroup blockIdx.x's tile lies.  Each XCD takes neighbouring tiles, in
// bands of 8 tile rows, so that its L2 serves them all.
__device__ __forceinline__ void place_tile(const GemmArgs &A, int rows, int cols, int &m0, int &n0) {
    constexpr int kBand = 8;
    const int total = A.tiles_m * A.tiles_n, q = total / 8, rem = total % 8;
    const int x = blockIdx.x % 8, i = blockIdx.x / 8;
    const int tile = x * q + min(x, rem) + i;
    const int band = tile / (kBand * A.tiles_n), in_band = tile % (kBand * A.tiles_n);
    const int height = min(kBand, A.tiles_m - band * kBand);
    m0 = (band * kBand + in_band % height) * rows;
    n0 = in_band / height * cols;
}

// A wave's load l brings 8 slots of a tile to shared memory: where in the operand,
// which has `rows` rows from the tile's first, a lane's 16 bytes lie.  Rows past the
// last are read as the last: their results are not stored.
__device__ __forceinline__ uint32_t slot_offset(int l, int lane, int rows, int ld) {
    const int slot = 8 * l + lane / 8, r = slot % 16;
    const int row = min(slot / 64 * 64 + 4 * r + slot % 64 / 16, rows - 1);
    return static_cast<uint32_t>(row) * static_cast<uint32_t>(ld) + 16u * ((lane % 8) ^ (r / 2));
}

// Waits for a wave's own loads to shared memory and reads of it, then for the other waves.
__device__ __forceinline__ void settle() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Keeps the instructions before and after apart, so that reads stay between the products.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// A step's part of a workgroup's shared memory: SIDE rows of either operand and 256
// bytes for the scales of each.
template <int SIDE>
struct StepMem {
    static constexpr int kB = SIDE * kStep, kScalesA = 2 * SIDE * kStep, kScalesB = kScalesA + 256, kBytes = kScalesA + 512;
};

// A wave's share of a step's loads: SIDE / 8 / WAVES of 1 KB for each operand, numbered from
// 0, the scales with the last.  Then it goes on to the next step, or after the last
// step to that one again: the loops below have no branches, since the compiler
// would gather all products behind the last of them.  Even waves bring the
// same scales of a, odd ones of b (TILE: of a again).
template <int SIDE, int WAVES, bool BROW>
struct Loads {
    static constexpr int kEach = SIDE / 8 / WAVES, kAll = 2 * kEach;
    uint32_t off_a[kEach], off_b[kEach], off_s, to_s, to;
    const uint8_t *pa, *pb, *ps;
    int64_t s_ld;
    int left;

    __device__ __forceinline__ Loads(const GemmArgs &A, const uint8_t *mem, int m0, int n0, int first, int steps, int lane, int wave) {
        pa = A.a + static_cast<int64_t>(m0) * A.a_ld + static_cast<int64_t>(first) * kStep;
        pb = A.b + static_cast<int64_t>(n0) * A.b_ld + static_cast<int64_t>(first) * kStep;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            off_a[i] = slot_offset(kEach * wave + i, lane, A.m - m0, A.a_ld);
            off_b[i] = slot_offset(kEach * wave + i, lane, A.n - n0, A.b_ld);
        }
        const bool of_b = BROW && wave % 2;
        s_ld = of_b ? A.bs_ld : A.as_ld;
        ps = (of_b ? A.bs : A.as) + first * s_ld;
        off_s = of_b ? min(n0 + 4 * lane, (A.n + 3) / 4 * 4 - 4) : min(m0 + 4 * lane, (A.m + 3) / 4 * 4 - 4);
        const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_address(mem));
        to = lds + 1024 * kEach * wave;
        to_s = lds + (of_b ? StepMem<SIDE>::kScalesB : StepMem<SIDE>::kScalesA);
        left = steps;
    }

    __device__ __forceinline__ void start(int buffer, int i) {
        if (i < kEach) load_lds16(to + buffer + 1024 * i, off_a[i % kEach], pa);
        else load_lds16(to + buffer + StepMem<SIDE>::kB + 1024 * (i - kEach), off_b[i % kEach], pb);
        if (i == kAll - 1) {
            load_lds4(to_s + buffer, off_s, ps);
            const bool more = --left > 0;
            pa += more ? kStep : 0;
            pb += more ? kStep : 0;
            ps += more ? s_ld : 0;
        }
    }
};

// A TILE operand's scales of a wave's columns: lane l holds that of step 64 c + l, and
// in `next` that of step 64 (c + 1) + l.
struct TileScales {
    const uint8_t *p;
    int64_t ld;
    int steps, now, next;

    __device__ __forceinline__ int load(int k, int lane) const {
        int x = p[static_cast<int64_t>(min(k + lane, steps - 1)) * ld];
        asm volatile("" : "+v"(x));  // waited for here, with no other loads under way
        return x;
    }
    __device__ __forceinline__ int of(int k, int chunk_end) const {
        const int x = __builtin_amdgcn_readlane(now, k % 64), y = __builtin_amdgcn_readlane(next, 0);
        return (k == chunk_end ? y : x) * 0x01010101;
    }
};

// 128 x 128 of the output by 4 waves of 64 x 64.  A step's operands come to shared memory
// STAGES steps ahead and to registers one ahead, so a step's one barrier stands
// between two steps' products.  In shared memory a group of 64 rows lies in the order 0, 4,
// 8, .. 60, 1, 5, ..: slot 16 i + r holds row 4 r + i.  The matrix instruction that takes slots 16 i
// to 16 i + 15 thereby finds its rows' scales in byte i of the dword of row
// 4 r, one dword for four instructions, and a lane's four results along
// a row of the output are neighbours, which are stored at once.  Within a slot's
// 128 bytes the 16-byte chunk c lies at c ^ (r / 2), which spreads the
// 16 rows that a quarter of a wave reads over all banks (no conflict is counted).
// Two stages let two workgroups share a CU, three are for one (plan_of has the figures).
constexpr int kSmall = 128;

template <int STAGES, bool BROW, bool EXACT>
__global__ __launch_bounds__(256, STAGES > 2 ? 1 : 2) void k_gemm_tile(GemmArgs A) {
    using Mem = StepMem<kSmall>;
    __shared__ __align__(16) uint8_t s_mem[STAGES * Mem::kBytes];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / 2, wn = wave % 2;
    int m0, n0;
    place_tile(A, kSmall, kSmall, m0, n0);
    const int split = blockIdx.y, first = split * A.split_steps, steps = min(A.split_steps, A.steps - first);
    Loads<kSmall, 4, BROW> loads(A, s_mem, m0, n0, first, steps, lane, wave);
    TileScales ts{A.bs + first * A.bs_ld + n0 / DOPT_FP8_BLOCK, A.bs_ld, steps, 0, 0};

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    const int r = lane % 16, quarter = lane / 16;
    const uint32_t low = r * kStep + 16 * (quarter ^ (r / 2)), high = r * kStep + 16 * ((quarter + 4) ^ (r / 2));
    const uint8_t *ma = s_mem + wm * 64 * kStep, *mb = s_mem + Mem::kB + wn * 64 * kStep, *ms = s_mem + 4 * r;
    struct Step {
        i32x8 a[4], b[4];
        int sa, sb;
    } x, y;
    const auto read = [&](i32x8 &v, const uint8_t *mem, int at) {  // the 16 rows from slot `at`
        v = join(*reinterpret_cast<const i32x4 *>(mem + at * kStep + low), *reinterpret_cast<const i32x4 *>(mem + at * kStep + high));
    };
    const auto read_scales = [&](Step &v, int buffer, int k, int chunk_end) {
        v.sa = *reinterpret_cast<const int *>(ms + buffer + Mem::kScalesA + wm * 64);
        if (BROW) v.sb = *reinterpret_cast<const int *>(ms + buffer + Mem::kScalesB + wn * 64);
        else v.sb = ts.of(k, chunk_end);
    };
    // multiplies v; in between next(i) for i in 0 to 3
    const auto multiply = [&](const Step &v, const auto &next) {
        if constexpr (!EXACT) {
            each4([&](auto I) {
                constexpr int i = decltype(I)::value;
                next(i);
                each4([&](auto J) {
                    constexpr int j = decltype(J)::value;
                    acc[i][j] = mfma<i, j>(v.a[i], v.b[j], acc[i][j], v.sa, v.sb);
                });
                in_order();
            });
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int h = 4 * half;
                bf16x8 b[4][2];
                each4([&](auto J) {
                    constexpr int j = decltype(J)::value;
                    const float scale = scale_of<j>(v.sb);
                    b[j][0] = widen8(v.b[j][h], v.b[j][h + 1], scale);
                    b[j][1] = widen8(v.b[j][h + 2], v.b[j][h + 3], scale);
                });
                each4([&](auto I) {
                    constexpr int i = decltype(I)::value;
                    if (i % 2 == 0) next(2 * half + i / 2);
                    const float scale = scale_of<i>(v.sa);
                    const bf16x8 a0 = widen8(v.a[i][h], v.a[i][h + 1], scale), a1 = widen8(v.a[i][h + 2], v.a[i][h + 3], scale);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma(a0, b[j][0], acc[i][j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma(a1, b[j][1], acc[i][j]);
                });
            }
        }
    };
    int at = 0;  // the buffer of the step that is multiplied
    const auto after = [](int buffer) { return buffer == (STAGES - 1) * Mem::kBytes ? 0 : buffer + Mem::kBytes; };
    // multiplies v, a step that all waves have read when the barrier is passed, starts loads into its buffer and
    // reads the step after it, k, which has landed when at most STAGES - 2 steps' loads of the wave are under way
    const auto turn = [&](Step &v, Step &w, int k, int chunk_end) {
        if constexpr (STAGES == 2) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * (Loads<kSmall, 4, BROW>::kAll + 1)) : "memory");
        in_order();
        const int nxt = after(at);
        read_scales(w, nxt, k, chunk_end);
        multiply(v, [&](int i) {
            read(w.b[i], mb + nxt, 16 * i);
            read(w.a[i], ma + nxt, 16 * i);
            loads.start(at, 2 * i);
            loads.start(at, 2 * i + 1);
        });
        in_order();
        at = nxt;
    };

    if (steps > 0) {
        if (!BROW) ts.now = ts.load(0, lane);
#pragma unroll
        for (int g = 0; g < STAGES; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) loads.start(g * Mem::kBytes, i);
        // the first step has landed when at most STAGES - 1 are under way
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((STAGES - 1) * (Loads<kSmall, 4, BROW>::kAll + 1)) : "memory");
        read_scales(x, 0, 0, 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            read(x.b[i], mb, 16 * i);
            read(x.a[i], ma, 16 * i);
        }
    }
    for (int chunk_at = 0; chunk_at < steps; chunk_at += 64) {
        const int chunk_end = min(chunk_at + 64, steps);
        if (!BROW && chunk_at > 0) ts.now = ts.next;
        if (!BROW && chunk_end < steps) ts.next = ts.load(chunk_end, lane);
        int k = chunk_at;
        for (; k + 1 < chunk_end; k += 2) {
            turn(x, y, k + 1, chunk_end);
            turn(y, x, k + 2, chunk_end);
        }
        if (k < chunk_end) turn(x, y, k + 1, chunk_end);  // the last step of an odd number
    }
    settle();  // the loads past the last step land in this workgroup's shared memory, so it stays until they have

    const int row0 = m0 + wm * 64, col0 = n0 + wn * 64;
    if (A.splits == 1) {
        store_tile<EXACT>(A, row0, col0, acc);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            put4_part(A, split, row0 + 4 * (4 * quarter + v) + i, col0 + 4 * r,
                      f32x4{acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]});
}

// ---- large tiles --------------------------------------------------------------------

constexpr int kBig = 256;  // rows and columns of a tile
constexpr int kBigOperand = StepMem<kBig>::kB, kBigBuffer = StepMem<kBig>::kBytes;

// 256 x 256 of the output by 4 waves, one to a SIMD with all of its registers, each
// 128 x 128.  As k_gemm_tile, but a step has two phases with its one barrier
// between them, so that the matrix cores have work on both sides of it:
//   phase 0 multiplies the first 64 rows of a, and reads the others;
//   barrier all have read this step, whose buffer is free, and the next step's loads are done;
//   phase 1 multiplies the other rows, starts the loads of the step after the next into the
//           free buffer, and reads the next step's first 64 rows of a and all of b, each
//           register once its last product is under way.
// 8192 x 14336 x 4096: 374 to 395 us; the matrix cores are busy 60% of the cycles.  With 8 waves of 128 x 64 and
// the same order of work 397 to 415 us (more reads of shared memory, and both waves of a SIMD
// wait at the same time), with reads and products of a step between two barriers 408; by instructions of 32 x 32 390 to
// 401; with all 16 loads at the start of phase 1 401 to 412, since they fill the path to the
// L1 and the products behind them wait; stores told apart by type for every four elements cost 20 to 120 us more.
template <bool BROW>
__global__ __launch_bounds__(256, 1) void k_gemm_big(GemmArgs A) {
    __shared__ __align__(16) uint8_t s_mem[2 * kBigBuffer];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / 2, wn = wave % 2;
    int m0, n0;
    place_tile(A, kBig, kBig, m0, n0);
    Loads<kBig, 4, BROW> loads(A, s_mem, m0, n0, 0, A.steps, lane, wave);
    TileScales ts{A.bs + min(n0 + wn * 128, A.n - 1) / DOPT_FP8_BLOCK, A.bs_ld, A.steps, 0, 0};

    f32x4 acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    const int r = lane % 16, quarter = lane / 16;
    const uint32_t low = r * kStep + 16 * (quarter ^ (r / 2)), high = r * kStep + 16 * ((quarter + 4) ^ (r / 2));
    const uint8_t *ma = s_mem + wm * 128 * kStep, *mb = s_mem + kBigOperand + wn * 128 * kStep;
    const uint8_t *ms = s_mem + 2 * kBigOperand + 4 * r;
    const auto read = [&](i32x8 &x, const uint8_t *mem, int at) {  // the 16 rows from slot `at`
        x = join(*reinterpret_cast<const i32x4 *>(mem + at * kStep + low), *reinterpret_cast<const i32x4 *>(mem + at * kStep + high));
    };
    const auto scales_a = [&](int buffer, int g) { return *reinterpret_cast<const int *>(ms + buffer + wm * 128 + 64 * g); };
    const auto scales_b = [&](int buffer, int g, int k, int chunk_end) {
        if (BROW) return *reinterpret_cast<const int *>(ms + buffer + 256 + wn * 128 + 64 * g);
        return ts.of(k, chunk_end);
    };

    if (A.steps > 0) {
        if (!BROW) ts.now = ts.load(0, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) loads.start(0, i);
#pragma unroll
        for (int i = 0; i < 16; ++i) loads.start(kBigBuffer, i);
    }
    settle();
    i32x8 a[8], b[8];
    int sa[2] = {scales_a(0, 0), scales_a(0, 1)}, sb[2] = {scales_b(0, 0, 0, 64), scales_b(0, 1, 0, 64)};
#pragma unroll
    for (int j = 0; j < 8; ++j) read(b[j], mb, 16 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i) read(a[i], ma, 16 * i);
    __builtin_amdgcn_s_waitcnt(0);  // so that in the loop only the loop's own reads are waited for
    for (int chunk_at = 0; chunk_at < A.steps; chunk_at += 64) {
        const int chunk_end = min(chunk_at + 64, A.steps);
        if (!BROW && chunk_at > 0) ts.now = ts.next;
        if (!BROW) ts.next = ts.load(chunk_end, lane);
        for (int k = chunk_at; k < chunk_end; ++k) {
            const int cur = (k & 1) * kBigBuffer, nxt = kBigBuffer - cur;
            each4([&](auto I) {
                constexpr int i = decltype(I)::value;
                read(a[4 + i], ma + cur, 16 * (4 + i));
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    each4([&](auto J) {
                        constexpr int j = decltype(J)::value;
                        acc[i][4 * g + j] = mfma<i, j>(a[i], b[4 * g + j], acc[i][4 * g + j], sa[0], sb[g]);
                    });
                in_order();
            });
            settle();
            in_order();
            const int next_sa0 = scales_a(nxt, 0), next_sa1 = scales_a(nxt, 1);
            const int next_sb0 = scales_b(nxt, 0, k + 1, chunk_end), next_sb1 = scales_b(nxt, 1, k + 1, chunk_end);
#pragma unroll
            for (int g = 0; g < 2; ++g)
                each4([&](auto J) {
                    constexpr int j = decltype(J)::value;
                    loads.start(cur, 2 * (4 * g + j));
                    loads.start(cur, 2 * (4 * g + j) + 1);
                    if (g == 0) read(a[j], ma + nxt, 16 * j);
                    each4([&](auto I) {
                        constexpr int i = decltype(I)::value;
                        acc[4 + i][4 * g + j] = mfma<i, j>(a[4 + i], b[4 * g + j], acc[4 + i][4 * g + j], sa[1], sb[g]);
                    });
                    in_order();
                    read(b[4 * g + j], mb + nxt, 16 * (4 * g + j));
                    in_order();
                });
            sa[0] = next_sa0;
            sa[1] = next_sa1;
            sb[0] = next_sb0;
            sb[1] = next_sb1;
        }
    }
    settle();  // the loads past the last step land in this workgroup's shared memory, so it stays until they have
    store_tile<false>(A, m0 + wm * 128, n0 + wn * 128, acc);
}

// The same tile with widened codes, by 8 waves of 128 x 64 each.  A step has 16
// turns, one for each half of its k and 16 rows of a, of 8 products.  A turn
// multiplies what the one before has widened, widens the next one's rows and reads those of
// the one after that; the columns of b are widened anew for each half, each right after
// its last product.  The barrier stands before the last turn, when all of the step has been
// read: the next step's loads, started in the first 8 turns, have landed by then.
// 4096 x 4096 x 8192, added to fp32: 202 us, 230 with reads and products of a step between two
// barriers.  As 4 waves of 128 x 128, which would widen a third fewer codes, it spends 350 of each step's
// instructions on moving accumulators about: 239 us.
template <bool BROW>
__global__ __launch_bounds__(512, 2) void k_gemm_wide(GemmArgs A) {
    __shared__ __align__(16) uint8_t s_mem[2 * kBigBuffer];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / 4, wn = wave % 4;
    int m0, n0;
    place_tile(A, kBig, kBig, m0, n0);
    Loads<kBig, 8, BROW> loads(A, s_mem, m0, n0, 0, A.steps, lane, wave);
    TileScales ts{A.bs + min(n0 + wn * 64, A.n - 1) / DOPT_FP8_BLOCK, A.bs_ld, A.steps, 0, 0};

    f32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    const int r = lane % 16, quarter = lane / 16;
    const uint32_t low = r * kStep + 16 * (quarter ^ (r / 2)), high = r * kStep + 16 * ((quarter + 4) ^ (r / 2));
    const uint8_t *ma = s_mem + wm * 128 * kStep, *mb = s_mem + kBigOperand + wn * 64 * kStep;
    const uint8_t *ms = s_mem + 2 * kBigOperand + 4 * r;
    const auto chunk = [&](const uint8_t *mem, int at, uint32_t half) {  // of the 16 rows from slot `at`
        return *reinterpret_cast<const i32x4 *>(mem + at * kStep + half);
    };
    const auto scales_a = [&](int buffer, int g) { return *reinterpret_cast<const int *>(ms + buffer + wm * 128 + 64 * g); };
    const auto scales_b = [&](int buffer, int k, int chunk_end) {
        if (BROW) return *reinterpret_cast<const int *>(ms + buffer + 256 + wn * 64);
        return ts.of(k, chunk_end);
    };

    if (A.steps > 0) {
        if (!BROW) ts.now = ts.load(0, lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) loads.start(0, i);
    }
    settle();
    bf16x8 wb[4][2], wa[2];
    i32x4 ra[2], rb[4];
    const auto widen_b = [&](int scales, auto J) {
        constexpr int j = decltype(J)::value;
        const float scale = scale_of<j>(scales);
        wb[j][0] = widen8(rb[j][0], rb[j][1], scale);
        wb[j][1] = widen8(rb[j][2], rb[j][3], scale);
    };
    int sa[2] = {scales_a(0, 0), scales_a(0, 1)}, sb = scales_b(0, 0, 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) rb[j] = chunk(mb, 16 * j, low);
    ra[0] = chunk(ma, 0, low);
    ra[1] = chunk(ma, 16, low);
    each4([&](auto J) { widen_b(sb, J); });
    wa[0] = widen8(ra[0][0], ra[0][1], scale_of<0>(sa[0]));
    wa[1] = widen8(ra[0][2], ra[0][3], scale_of<0>(sa[0]));
    __builtin_amdgcn_s_waitcnt(0);
    for (int chunk_at = 0; chunk_at < A.steps; chunk_at += 64) {
        const int chunk_end = min(chunk_at + 64, A.steps);
        if (!BROW && chunk_at > 0) ts.now = ts.next;
        if (!BROW) ts.next = ts.load(chunk_end, lane);
        for (int k = chunk_at; k < chunk_end; ++k) {
            const int cur = (k & 1) * kBigBuffer, nxt = kBigBuffer - cur;
            const auto turn = [&](auto T) {
                constexpr int t = decltype(T)::value, i = t % 8, n = (t + 1) % 8;
                if constexpr (t < 8) loads.start(nxt, t);
                if constexpr (t == 15) {
                    settle();
                    in_order();
                    sa[0] = scales_a(nxt, 0);
                    sb = scales_b(nxt, k + 1, chunk_end);
#pragma unroll
                    for (int j = 0; j < 4; ++j) rb[j] = chunk(mb + nxt, 16 * j, low);
                    ra[0] = chunk(ma + nxt, 0, low);
                    ra[1] = chunk(ma + nxt, 16, low);
                    sa[1] = scales_a(nxt, 1);
                } else if constexpr (t < 14) {
                    ra[t % 2] = chunk(ma + cur, 16 * ((t + 2) % 8), t + 2 < 8 ? low : high);
                }
                if constexpr (t == 6) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) rb[j] = chunk(mb + cur, 16 * j, high);
                }
                bf16x8 x0, x1;
                each4([&](auto J) {
                    constexpr int j = decltype(J)::value;
                    acc[i][j] = mfma(wa[0], wb[j][0], acc[i][j]);
                    if (t < 15 && j == 1) x0 = widen8(ra[(t + 1) % 2][0], ra[(t + 1) % 2][1], scale_of<n % 4>(sa[n / 4]));
                    if (t < 15 && j == 3) x1 = widen8(ra[(t + 1) % 2][2], ra[(t + 1) % 2][3], scale_of<n % 4>(sa[n / 4]));
                });
                each4([&](auto J) {
                    constexpr int j = decltype(J)::value;
                    acc[i][j] = mfma(wa[1], wb[j][1], acc[i][j]);
                    if constexpr (i == 7) widen_b(sb, J);
                });
                if constexpr (t == 15) {
                    x0 = widen8(ra[0][0], ra[0][1], scale_of<0>(sa[0]));
                    x1 = widen8(ra[0][2], ra[0][3], scale_of<0>(sa[0]));
                }
                wa[0] = x0;
                wa[1] = x1;
                in_order();
            };
            each4([&](auto T) { turn(T); });
            each4([&](auto T) { turn(std::integral_constant<int, 4 + decltype(T)::value>{}); });
            each4([&](auto T) { turn(std::integral_constant<int, 8 + decltype(T)::value>{}); });
            each4([&](auto T) { turn(std::integral_constant<int, 12 + decltype(T)::value>{}); });
        }
    }
    settle();
    store_tile<true>(A, m0 + wm * 128, n0 + wn * 64, acc);
}

// ---- few rows ---------------------------------------------------------------------

// Up to 16 rows of a: b is read once, and what bounds the call is how fast.  A
// workgroup takes 16 columns of the output, its waves share the steps along k, and
// their sums are joined through shared memory.  A wave has the operands of
// kFewDepth steps under way before it multiplies the first.  It adds in fp32 whoever calls: 1 x 14336 x 4096
// takes 14.5 us so and 13.8 with the codes' own instruction, 1 x 4096 x 14336 15.4 and 15.2.  With that instruction
// 1 x 14336 x 4096 took 3 us more without steps under way, 14 more with 8 of them, whose waves are too few, and 3 more with b read
// around the caches; 17 to 64 rows so, with a read anew by every workgroup, 28 us (32 rows) and 43 (64) where
// k_gemm_tile takes 17.
constexpr int kFewDepth = 4;

template <int WAVES, bool BROW>
__global__ __launch_bounds__(WAVES * 64) void k_gemm_few(GemmArgs A) {
    __shared__ __align__(16) float s_sum[WAVES][256];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int r = lane % 16, quarter = lane / 16;
    const int n0 = blockIdx.x * 16, split = blockIdx.y;
    const int first = split * A.split_steps, end = min(first + A.split_steps, A.steps);
    const int row = min(r, A.m - 1), col = min(n0 + r, A.n - 1), scale_col = BROW ? col : n0 / DOPT_FP8_BLOCK;
    const uint8_t *pa = A.a + static_cast<int64_t>(row) * A.a_ld + 16 * quarter;
    const uint8_t *pb = A.b + static_cast<int64_t>(col) * A.b_ld + 16 * quarter;
    f32x4 acc = {0, 0, 0, 0};
    for (int k0 = first + wave; k0 < end; k0 += kFewDepth * WAVES) {
        i32x4 b[kFewDepth][2], a[kFewDepth][2];
        int sb[kFewDepth], sa[kFewDepth];
#pragma unroll
        for (int u = 0; u < kFewDepth; ++u) {
            const int64_t k = min(k0 + u * WAVES, end - 1);  // steps past the last are read as the last, and not multiplied
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                b[u][h] = *reinterpret_cast<const i32x4 *>(pb + k * kStep + 64 * h);
                a[u][h] = *reinterpret_cast<const i32x4 *>(pa + k * kStep + 64 * h);
            }
            sa[u] = A.as[k * A.as_ld + row];
            sb[u] = A.bs[k * A.bs_ld + scale_col];
        }
        in_order();
#pragma unroll
        for (int u = 0; u < kFewDepth; ++u) {
            if (k0 + u * WAVES >= end) break;
            const float fa = scale_of<0>(sa[u]), fb = scale_of<0>(sb[u]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc = mfma(widen8(a[u][j / 2][2 * (j % 2)], a[u][j / 2][2 * (j % 2) + 1], fa),
                           widen8(b[u][j / 2][2 * (j % 2)], b[u][j / 2][2 * (j % 2) + 1], fb), acc);
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) s_sum[wave][(4 * quarter + v) * 16 + r] = acc[v];
    __syncthreads();
    if (wave > 0) return;
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) x += *reinterpret_cast<const f32x4 *>(&s_sum[w][4 * lane]);
    if (A.splits > 1) put4_part(A, split, lane / 4, n0 + 4 * (lane % 4), x);
    else put4(A, lane / 4, n0 + 4 * (lane % 4), x);
}

// ---- which kernel -------------------------------------------------------------------

struct Plan {
    int rows, cols;  // of a tile
    bool few;
    int stages;  // of k_gemm_tile
    int waves;   // of k_gemm_few
    int splits, split_steps;
};

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kCus = 256;

static Plan plan_of(int64_t m, int64_t n, int64_t k) {
    Plan p{};
    const int64_t steps = std::max<int64_t>(ceil_div(k, kStep), 1);
    p.few = m <= 16;
    p.stages = 2;
    int64_t splits = 1;
    if (p.few) {
        // One batch of kFewDepth steps to a wave, up to 8 waves: 4096 columns, 8 steps: 4.4 us with 2
        // waves, 4.6 with 4, 5.7 with 8; 6000 columns, 16 steps: 6.8, 6.4, 8.5; 11008 columns, 32 steps: 12.6, 13.2, 11.7;
        // 8192 columns, 32 steps: 11.0, 10.8, 9.5.  More steps than that are shared by several workgroups where
        // the columns are few: 768 columns, 128 steps: 13.0 us, split in 4 9.5, in 8 12.1; 2048 columns, 64 steps: 8.6, in 2 9.3.
        p.rows = p.cols = 16;
        p.waves = steps <= 12 ? 2 : steps <= 24 ? 4 : 8;
        if (ceil_div(n, p.cols) <= 64) splits = steps / (8 * kFewDepth);
    } else {
        const int64_t small = ceil_div(m, kSmall) * ceil_div(n, kSmall), big = ceil_div(m, kBig) * ceil_div(n, kBig);
        if (small <= kCus) {
            // A tile or less to a CU: what counts is how soon a step's loads are back, so three steps are under way,
            // and with 8 steps or more to each the steps are shared by several workgroups.
            // 1024 x 4096 x 4096: 42 us with 2 stages, 33 with 3 (coarse 26.6, 21.7).  128 x 4096 x 4096: 40 with 2 stages, 29.7
            // with 3; split in 2, 4, 8: 22.4, 19.2, 20.8 (coarse 24.6, 16.4; 15.7, 15.7, 18.8).  768 x 768 x 8192 added to fp32, split in 1, 2, 4,
            // 7, 8 (the rule's 7): 53, 33.6, 23.4, 21.7, 28.4; 768 x 2304 x 8192 unsplit, in 2, 3, 4, 7 (the rule's 2): 53.5, 39.1, 47.4, 43.6, 54.1.
            p.rows = p.cols = kSmall;
            p.stages = 3;
            splits = std::min(kCus / small, steps / 8);
        } else {
            // With coarse sums a round of big tiles takes about 7 us and 1.25 for each step, one of twice as many small
            // ones 2.5 and 0.92 (measured at 256 to 1024 small tiles and 8 to 32 steps); sums in fp32 take longer in about the same proportion.
            // Small and big, us: 2048 x 4096 x 4096 60, 81; 3073 x 4096 x 4096 101, 83; 4096 x 4096 x 4096 114, 95;
            // 8192 x 2304 x 768 34, 41; 4096 x 14336 x 128 36, 38; coarse 34, 48; 57, 48; 62, 56; 25, 32; 32, 41; fp32 out 59, 80; 105, 85; 116, 102;
            // 37, 45; 54, 61.
            const int64_t as_big = ceil_div(big, kCus) * (28 + 5 * steps), as_small = ceil_div(small, 2 * kCus) * (100 + 37 * steps);
            p.rows = p.cols = as_big * 10 <= as_small ? kBig : kSmall;
        }
    }
    splits = std::max<int64_t>(splits, 1);
    p.split_steps = static_cast<int>(ceil_div(steps, splits));
    p.splits = static_cast<int>(ceil_div(steps, p.split_steps));
    return p;
}

static int64_t part_ld_of(int64_t n) { return (n + 3) / 4 * 4; }

// Threads of a workgroup.
static unsigned threads_of(const Plan &p, bool exact) { return p.few ? 64 * p.waves : p.rows == kBig && exact ? 512 : 256; }

template <bool BROW, bool EXACT>
static void launch_gemm(const GemmArgs &A, const Plan &p, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(A.tiles_m * A.tiles_n), static_cast<unsigned>(A.splits));
    const unsigned threads = threads_of(p, EXACT);
    if (p.few) {
        if (p.waves == 2) k_gemm_few<2, BROW><<<grid, threads, 0, stream>>>(A);
        else if (p.waves == 4) k_gemm_few<4, BROW><<<grid, threads, 0, stream>>>(A);
        else k_gemm_few<8, BROW><<<grid, threads, 0, stream>>>(A);
    } else if (p.rows == kBig) {
        if constexpr (EXACT) k_gemm_wide<BROW><<<grid, threads, 0, stream>>>(A);
        else k_gemm_big<BROW><<<grid, threads, 0, stream>>>(A);
    } else {
        if (p.stages == 2) k_gemm_tile<2, BROW, EXACT><<<grid, threads, 0, stream>>>(A);
        else k_gemm_tile<3, BROW, EXACT><<<grid, threads, 0, stream>>>(A);
    }
}

static bool size_ok(int64_t m, int64_t n, int64_t k) {
    return m >= 0 && n >= 0 && k >= 0 && m <= DOPT_FP8_MAX_ROWS && n < (1 << 23) && k <= DOPT_FP8_MAX_COLS;
}

}  // namespace dopt

using namespace dopt;

extern "C" int64_t dopt_fp8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (!size_ok(m, n, k)) return fail(DOPT_ERR_INVALID, "bad size");
    if (m == 0 || n == 0) return 0;
    const Plan p = plan_of(m, n, k);
    return p.splits > 1 ? int64_t(p.splits) * m * part_ld_of(n) * 4 : 0;
}

static int gemm(bool exact, const dopt_fp8_matrix *a, const dopt_fp8_matrix *b, const dopt_dense *out, int32_t accumulate,
                void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (int rc = check_fp8("a", a)) return rc;
    if (int rc = check_fp8("b", b)) return rc;
    if (int rc = check_dense("out", out)) return rc;
    if (a->kind != DOPT_FP8_ROW) return fail(DOPT_ERR_INVALID, "a: not of kind ROW");
    if (a->cols != b->cols) return fail(DOPT_ERR_INVALID, "a and b differ in columns");
    if (!exact && out->dtype == DOPT_F32) return fail(DOPT_ERR_INVALID, "out: fp32, which coarse sums are not for");
    if (out->rows != a->rows || out->cols != b->rows) return fail(DOPT_ERR_INVALID, "out: not of a's rows x b's rows");
    const int64_t m = a->rows, n = b->rows, k = a->cols;
    if (!size_ok(m, n, k)) return fail(DOPT_ERR_INVALID, "too large");
    if (m == 0 || n == 0 || (k == 0 && accumulate)) return DOPT_OK;
    const int64_t need = dopt_fp8_gemm_workspace_bytes(m, n, k);
    if (need > 0 && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16))
        return fail(DOPT_ERR_INVALID, "workspace: null, not 16-byte aligned or too small (" + std::to_string(need) + " bytes)");
    const Span o[] = {dense_span("out", out), span_of("workspace", workspace, need)};
    const Span in[] = {codes_span("a", a), scales_span("a's scales", a), codes_span("b", b), scales_span("b's scales", b)};
    if (int rc = check_apart(o, 2, in, 4)) return rc;

    const Plan p = plan_of(m, n, k);
    const int64_t tiles_m = ceil_div(m, p.rows), tiles_n = ceil_div(n, p.cols);
    if (tiles_m * tiles_n * threads_of(p, exact) >= kMaxThreads) return fail(DOPT_ERR_INVALID, "out: too large");
    GemmArgs A{};
    A.a = static_cast<const uint8_t *>(a->codes);
    A.b = static_cast<const uint8_t *>(b->codes);
    A.as = static_cast<const uint8_t *>(a->scales);
    A.bs = static_cast<const uint8_t *>(b->scales);
    A.out = out->data;
    A.part = static_cast<float *>(workspace);
    A.as_ld = a->scale_ld;
    A.bs_ld = b->scale_ld;
    A.out_ld = out->ld;
    A.part_ld = part_ld_of(n);
    A.a_ld = static_cast<int32_t>(a->ld);
    A.b_ld = static_cast<int32_t>(b->ld);
    A.m = static_cast<int32_t>(m);
    A.n = static_cast<int32_t>(n);
    A.steps = static_cast<int32_t>(ceil_div(k, kStep));
    A.tiles_m = static_cast<int32_t>(tiles_m);
    A.tiles_n = static_cast<int32_t>(tiles_n);
    A.splits = p.splits;
    A.split_steps = p.split_steps;
    A.dtype = out->dtype;
    A.accumulate = accumulate != 0;
    const bool row = b->kind == DOPT_FP8_ROW;
    if (row && exact) launch_gemm<true, true>(A, p, stream);
    else if (row) launch_gemm<true, false>(A, p, stream);
    else if (exact) launch_gemm<false, true>(A, p, stream);
    else launch_gemm<false, false>(A, p, stream);
    if (int rc = launched("dopt_fp8_gemm")) return rc;
    if (p.splits > 1) {
        const int64_t vectors = m * (A.part_ld / 4);
        k_gemm_join<<<static_cast<unsigned>(ceil_div(vectors, 256)), 256, 0, stream>>>(A);
        return launched("dopt_fp8_gemm");
    }
    return DOPT_OK;
}

extern "C" int dopt_fp8_gemm(const dopt_fp8_matrix *a, const dopt_fp8_matrix *b, const dopt_dense *out, int32_t accumulate,
                             void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    return gemm(true, a, b, out, accumulate, workspace, workspace_bytes, stream);
}

extern "C" int dopt_fp8_gemm_coarse(const dopt_fp8_matrix *a, const dopt_fp8_matrix *b, const dopt_dense *out, int32_t accumulate,
                                    void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    return gemm(false, a, b, out, accumulate, workspace, workspace_bytes, stream);
}
