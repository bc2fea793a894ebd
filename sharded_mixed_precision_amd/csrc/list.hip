// The AdamW step over a list of tensors for gfx950 (MI355X): kernels and
// entry points of dopt_list.h.
//
// Per element, in fp32 and in this order (adamw_root in device.h):
//   g = fp32(raw) * inv_scale;  g = g * clip              (when clipping)
//   p = p * (1 - lr*wd);  m = b1*m + (1-b1)*g;  v = b2*v + (1-b2)*(g*g)
//   p = p - step_size * (m / (sqrt(v) / sqrt(1-b2^t) + eps))
// with m and v fp32 arrays, or m = c*S and v = (c*S)^2 from e4m3 codes c and
// the scale S of a block of 128 elements; the new m and sqrt(v) are encoded
// with their block's new scale.  p uses them before they are rounded.
//
// Every pass streams its arrays once and is bound by HBM: pass 2 without its
// arithmetic takes the same time.  A list is cut into tiles of 2048 elements,
// one workgroup each, and what the layout decides is how well the
// streams run.  Measured on MI355X, pass 2 of 1.1e9 bf16 params with fp32
// moments / of 1.0e9 with fp32 grads and e4m3 moments:
//   grid-stride over 16384 workgroups, 8 consecutive elements per lane   5.65 / 3.85 ms
//   one workgroup per tile                                               5.46 / 3.52 ms
//   a lane owns 4 elements in each half of its wave's 512: each
//   16-byte access of a wave covers a whole KB, all accesses nontemporal 5.02 / 3.16 ms
//   runs of 16 consecutive tiles on one XCD (tile_of)                    4.95 / 3.04 ms
//   512 threads to a tile, a lane with 4 elements, launched in pieces    4.95 / 2.85 ms
// Nontemporal accesses lose in the first layout, whose instructions leave
// half of every line they touch to the next one.  Pass 1 reads the grads of a
// list that is not too long with ordinary loads (kListKeep in list.h): pass 2
// then finds them in the last-level cache.
//
// A block of 128 elements is then a half-wave: the DPP lane permutes reduce
// over 16 lanes, one swizzle joins the two halves, and LDS is not used.
// Tensors start anywhere their element type allows, so params and grads go
// through accesses of element alignment (gfx950 takes unaligned global
// accesses); the arena arrays are aligned.  The last lane of a tensor takes
// single elements: nothing outside a tensor is read.
#include "device.h"

#include "list.h"

namespace dopt {

// ---- tensor addresses ---------------------------------------------------------

// The addresses of a launch's tensors: distances from the lowest of the
// launch in units of 2^shift bytes, or a table of the class in the workspace.
struct GradAddr {
    const dopt_list_ptrs *table;
    const char *grad0;
    uint32_t grad_shift, pad;
    uint32_t grad[kListGradSlots];
};
struct ListSlot {
    uint32_t grad, param;
};
struct ListAddr {
    const dopt_list_ptrs *table;
    const char *grad0;
    char *param0;
    uint32_t grad_shift, param_shift;
    ListSlot s[kListSlots];
};
struct PutAddr {
    dopt_list_ptrs p[kListPut];
};

__global__ void __launch_bounds__(kBlock) k_list_put(dopt_list_ptrs *__restrict__ dst, int32_t n, PutAddr a) {
    if (static_cast<int>(threadIdx.x) < n) dst[threadIdx.x] = a.p[threadIdx.x];
}
static_assert(kListPut <= kBlock, "one thread an address");

// Tensor `index` of the class, in a launch that begins with tensor `first`.
// The distances are read whether they are used or not, beside the table's
// address rather than after it.
__device__ __forceinline__ dopt_list_ptrs ptrs_of(const ListAddr &a, uint32_t index, int32_t first) {
    const ListSlot s = a.s[index - first];
    dopt_list_ptrs p{a.grad0 + (uint64_t(s.grad) << a.grad_shift), a.param0 + (uint64_t(s.param) << a.param_shift)};
    if (__builtin_expect(a.table != nullptr, 0)) p = a.table[index];
    return p;
}
__device__ __forceinline__ const void *grad_of(const GradAddr &a, uint32_t index, int32_t first) {
    const void *p = a.grad0 + (uint64_t(a.grad[index - first]) << a.grad_shift);
    if (__builtin_expect(a.table != nullptr, 0)) p = a.table[index].grad;
    return p;
}

// ---- element I/O at element alignment -------------------------------------------

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kQuad = 4;               // consecutive elements of a lane
constexpr int kGroup = 64 * kQuad;     // what a wave's access covers
constexpr int kGroups = kVec / kQuad;  // groups of a wave, back to back, where kBlock threads share a tile
constexpr int kWide = kTile / kQuad;   // threads that share a tile with one group to a wave

// The raw bytes of 4 consecutive elements, and their type at the element's alignment.
template <int DT>
struct Quad {
    typedef uint16_t T;
    typedef u32x2 Raw;
    typedef u32x2 At __attribute__((aligned(2)));
};
template <>
struct Quad<DOPT_F32> {
    typedef float T;
    typedef u32x4 Raw;
    typedef u32x4 At __attribute__((aligned(4)));
};

template <int DT>
__device__ __forceinline__ float up1(typename Quad<DT>::T x) {
    if constexpr (DT == DOPT_F32) return x;
    else if constexpr (DT == DOPT_BF16) return __uint_as_float(uint32_t(x) << 16);
    else return Elem<DOPT_F16>::up(x);
}

template <int DT>
__device__ __forceinline__ typename Quad<DT>::T down1(float x) {
    if constexpr (DT == DOPT_F32) return x;
    else return static_cast<uint16_t>(Elem<DT>::bits(x));
}

// A pointer into device memory, said to the compiler: one that came out of a
// table would otherwise be accessed with flat instructions (pass 2 of 1.2e8
// fp32 params on MI355X 603 us, 587 with global ones).
template <class T>
__device__ __forceinline__ __attribute__((address_space(1))) T *global(T *p) {
    return (__attribute__((address_space(1))) T *)p;
}

// Elements i .. i+3 of a tensor, of which the first n exist (n <= 0: none);
// the others read as 0.  KEEP: an ordinary load, for what a later pass reads
// again from the last-level cache.
template <int DT, bool KEEP = false>
__device__ __forceinline__ typename Quad<DT>::Raw load4(const void *base, int64_t i, int n) {
    typedef Quad<DT> Q;
    const auto *p = global(static_cast<const typename Q::T *>(base)) + i;
    typename Q::Raw r{};
    if (n >= kQuad) {
        const auto *q = (const __attribute__((address_space(1))) typename Q::At *)p;
        if constexpr (KEEP) r = *q;
        else r = __builtin_nontemporal_load(q);
    } else {
#pragma unroll
        for (int j = 0; j < kQuad - 1; ++j) {
            if (j < n) {
                if constexpr (DT == DOPT_F32) r[j] = __float_as_uint(p[j]);
                else r[j >> 1] |= uint32_t(p[j]) << (16 * (j & 1));
            }
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void unpack4(typename Quad<DT>::Raw r, float (&x)[kQuad]) {
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
        if constexpr (DT == DOPT_F32) x[j] = __uint_as_float(r[j]);
        else x[j] = up1<DT>(static_cast<uint16_t>(r[j >> 1] >> (16 * (j & 1))));
    }
}

template <int DT>
__device__ __forceinline__ void store4(void *base, int64_t i, int n, const float (&x)[kQuad]) {
    typedef Quad<DT> Q;
    auto *p = global(static_cast<typename Q::T *>(base)) + i;
    if (n >= kQuad) {
        typename Q::Raw r;
        if constexpr (DT == DOPT_F32) {
#pragma unroll
            for (int j = 0; j < kQuad; ++j) r[j] = __float_as_uint(x[j]);
        } else {
            r[0] = Elem<DT>::bits(x[0]) | (Elem<DT>::bits(x[1]) << 16);
            r[1] = Elem<DT>::bits(x[2]) | (Elem<DT>::bits(x[3]) << 16);
        }
        __builtin_nontemporal_store(r, (__attribute__((address_space(1))) typename Q::At *)p);
    } else {
#pragma unroll
        for (int j = 0; j < kQuad - 1; ++j)
            if (j < n) p[j] = down1<DT>(x[j]);
    }
}

// ---- e4m3 blocks ----------------------------------------------------------------

constexpr float kLeastScaled = 0x1p-100f;  // a block whose largest magnitude is below is held as zeros
constexpr float kCapM = 0x1p127f;
constexpr float kCapRoot = 0x1.fffffep63f;  // the largest fp32 number whose square is finite
constexpr float kTop = 448.0f, kLeast = 0x1p-9f;  // e4m3's largest and smallest magnitudes
constexpr float kLeastNormal = 0x1p-6f;           // below it e4m3's numbers are 2^-9 apart

__device__ __forceinline__ void decode4(uint32_t c, float scale, float (&x)[kQuad]) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), true);
    x[0] = a[0] * scale;
    x[1] = a[1] * scale;
    x[2] = b[0] * scale;
    x[3] = b[1] * scale;
}

template <int CTRL>
__device__ __forceinline__ uint32_t row_max(uint32_t u) {
    const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, false));
    return u > o ? u : o;
}

// The largest magnitude over a half-wave, as fp32 bits: an unsigned maximum of
// the bits without their sign, in which NaN is above infinity and both above
// every number, so a NaN is never dropped.
__device__ __forceinline__ float block_max(const float (&x)[kQuad]) {
    uint32_t u = 0;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
        const uint32_t b = __float_as_uint(x[j]) & 0x7fffffffu;
        u = u > b ? u : b;
    }
    u = row_max<0xb1>(u);   // quad_perm 1,0,3,2
    u = row_max<0x4e>(u);   // quad_perm 2,3,0,1
    u = row_max<0x141>(u);  // row_half_mirror
    u = row_max<0x140>(u);  // row_mirror
    const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(u), 0x401f));  // lane ^ 16
    return __uint_as_float(u > o ? u : o);
}

// How a lane's 4 values in units of their scale become e4m3 numbers: to the
// nearest, which the conversion does, or to one of the two neighbours by
// chance with the mean kept.  m and sqrt(v) take a half of one random word each
// (ROOT: the upper): the mean of 2^16 equal chances is within 2^-17 of a step.
struct Nearest {
    template <bool ROOT>
    __device__ __forceinline__ float round(float q, int) const {
        return q;
    }
};

struct Dither {
    uint32_t w[kQuad];

    // |q| <= 448 with 3 bits behind its leading one, as the conversion keeps them:
    // a chance below 1 of a step is added and the bits below are cut.  Numbers
    // below 2^-6, whose step stays 2^-9, are raised to 2^-6 for it, where
    // the step is that.  448 has no bits to carry into, so nothing passes it.
    template <bool ROOT>
    __device__ __forceinline__ float round(float q, int j) const {
        const float a = fabsf(q);
        const bool low = a < kLeastNormal;
        const uint32_t b = __float_as_uint(low ? a + kLeastNormal : a);
        const uint32_t u = ROOT ? w[j] >> 16 : w[j] & 0xffffu;
        const float y = __uint_as_float((b + (u << 4) + 8) & 0xfff00000u);
        return copysignf(low ? y - kLeastNormal : y, q);
    }
};

// The random words of 4 elements: Philox4x32 with 7 rounds (Salmon, Moraes,
// Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3, 2011), whose counter is the place of the 4
// in the arena and the number of the step, and whose key is the list's seed.
// 7 rounds are the fewest that the paper finds without fault.  On MI355X a step with
// rounding by chance and to nearest: 1.0e9 bf16 params with fp32 grads 3.74 and 3.41 ms, 1.2e8
// bf16 426 and 369 us, 1.8e7 fp16 in 500 tensors 79.7 and 72.7 us, 2,608 elements the same 10 us:
// the words' multiplications no longer hide behind the memory.
__device__ __forceinline__ Dither random4(uint64_t quad, uint64_t step, uint64_t seed) {
    uint32_t c[4] = {static_cast<uint32_t>(quad), static_cast<uint32_t>(quad >> 32), static_cast<uint32_t>(step),
                     static_cast<uint32_t>(step >> 32)};
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const uint64_t a = uint64_t(0xd2511f53u) * c[0], b = uint64_t(0xcd9e8d57u) * c[2];
        c[0] = static_cast<uint32_t>(b >> 32) ^ c[1] ^ k0;
        c[1] = static_cast<uint32_t>(b);
        c[2] = static_cast<uint32_t>(a >> 32) ^ c[3] ^ k1;
        c[3] = static_cast<uint32_t>(a);
        k0 += 0x9e3779b9u;
        k1 += 0xbb67ae85u;
    }
    return Dither{{c[0], c[1], c[2], c[3]}};
}

// Codes and scale of a block, all 32 lanes of its half-wave together.  ROOT:
// a square root of v, whose nonzero values keep a nonzero code.
template <bool ROOT, class R>
__device__ __forceinline__ uint32_t encode4(const float (&x)[kQuad], float &scale, const R &how) {
    const float a = block_max(x);
    const float cap = ROOT ? kCapRoot : kCapM;
    const bool live = !(a < kLeastScaled);
    scale = live ? (a > cap ? cap : a) * (1.0f / kTop) : 0.0f;  // a NaN passes both comparisons
    const float inv = live ? 1.0f / scale : 0.0f;
    float q[kQuad];
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
        q[j] = how.template round<ROOT>(__builtin_amdgcn_fmed3f(x[j] * inv, -kTop, kTop), j);
        if (ROOT) q[j] = x[j] > 0.0f ? fmaxf(q[j], kLeast) : q[j];
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    return live ? static_cast<uint32_t>(w) : 0u;
}

// 4 codes at arena element e, of which the first n exist (the others keep
// their bytes).
__device__ __forceinline__ void store_codes(void *base, int64_t e, int n, uint32_t c) {
    uint8_t *p = static_cast<uint8_t *>(base) + e;
    if (n >= kQuad) {
        __builtin_nontemporal_store(c, reinterpret_cast<uint32_t *>(p));
    } else {
#pragma unroll
        for (int j = 0; j < kQuad - 1; ++j)
            if (j < n) p[j] = static_cast<uint8_t>(c >> (8 * j));
    }
}

// ---- tiles and lanes --------------------------------------------------------------

// The tile of workgroup b of n.  Workgroups go to the 8 XCDs in turn; runs of
// kXcdRun consecutive tiles are dealt to one XCD, so that the lines two tiles
// share (a tile's scales are half a line) meet in one L2, and each XCD's
// requests run along the arrays.  On MI355X, runs of 4 / 8 / 16 / 32 / 64 tiles:
// pass 2 with e4m3 moments of 1.0e9 elements 3.05 / 2.91 / 2.91 / 2.90 / 2.91 ms, with fp32
// ones of 1.1e9 4.94 / 4.90 / 4.90 / 4.91 / 5.00, export of 1.0e9 2.98 / 3.00 / 2.90 / 2.96 / 3.07.
constexpr int64_t kXcds = 8, kXcdRun = 16;
__device__ __forceinline__ int64_t tile_of(int64_t b, int64_t n) {
    const int64_t whole = n / (kXcds * kXcdRun) * (kXcds * kXcdRun);
    if (b >= whole) return b;
    return b / (kXcds * kXcdRun) * (kXcds * kXcdRun) + b % kXcds * kXcdRun + b / kXcds % kXcdRun;
}

// A lane's 4 elements of one group of its tile.
struct Place {
    int64_t e;      // the first within the tensor
    int64_t arena;  // and in the arena
    int n;          // how many of them exist (<= 0: none)
};

// Where a lane's 4 elements of a group start in the tile; `thread` is among
// the kTile / (GROUPS * kQuad) that share it.
template <int GROUPS>
__device__ __forceinline__ int lane_offset(int group, int thread) {
    return (thread >> 6) * (kGroup * GROUPS) + group * kGroup + (thread & 63) * kQuad;
}
template <int GROUPS>
__device__ __forceinline__ Place place_of(const ListTile &d, int group, int thread) {
    const int l = lane_offset<GROUPS>(group, thread);
    return Place{int64_t(d.tile) * kTile + l, int64_t(d.block) * kListBlock + l, static_cast<int>(d.packed & 0xffffu) - l};
}

// Whether a wave's group of a tile holds an element (wave-uniform).
__device__ __forceinline__ bool group_lives(const ListTile &d, int group, int thread) {
    return __builtin_amdgcn_readfirstlane(thread >> 6) * (kGroup * kGroups) + group * kGroup <
           static_cast<int>(d.packed & 0xffffu);
}

struct StateArrays {
    float *master;
    void *m, *v;
    float *ms, *vs;
};

// m and v of a lane's 4 elements as they are held: loaded together, decoded later.
template <int ST>
struct Moments;

template <>
struct Moments<DOPT_STATE_F32> {
    u32x4 m, v;
    __device__ __forceinline__ void load(const StateArrays &s, const Place &L) {
        m = load4<DOPT_F32>(s.m, L.arena, L.n);
        v = load4<DOPT_F32>(s.v, L.arena, L.n);
    }
    __device__ __forceinline__ void decode(float (&a)[kQuad], float (&b)[kQuad]) const {
        unpack4<DOPT_F32>(m, a);
        unpack4<DOPT_F32>(v, b);
    }
    // r = sqrt(v)
    static __device__ __forceinline__ void store(const StateArrays &s, const Place &L, float (&a)[kQuad],
                                                 const float (&b)[kQuad], float (&)[kQuad], const Nearest &) {
        store4<DOPT_F32>(s.m, L.arena, L.n, a);
        store4<DOPT_F32>(s.v, L.arena, L.n, b);
    }
};

template <>
struct Moments<DOPT_STATE_E4M3> {
    uint32_t m, v;
    float ms, vs;
    __device__ __forceinline__ void load(const StateArrays &s, const Place &L) {
        m = v = 0;
        ms = vs = 0.0f;
        if (L.n > 0) {  // a block's slots past the tensor's end are arena memory: whole 4-byte loads
            m = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(s.m) + L.arena));
            v = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(s.v) + L.arena));
            ms = s.ms[L.arena / kListBlock];
            vs = s.vs[L.arena / kListBlock];
        }
    }
    __device__ __forceinline__ void decode(float (&a)[kQuad], float (&b)[kQuad]) const {
        decode4(m, ms, a);
        decode4(v, vs, b);
#pragma unroll
        for (int j = 0; j < kQuad; ++j) b[j] = b[j] * b[j];
    }
    template <class R>
    static __device__ __forceinline__ void store(const StateArrays &s, const Place &L, float (&a)[kQuad],
                                                 const float (&)[kQuad], float (&r)[kQuad], const R &how) {
#pragma unroll
        for (int j = 0; j < kQuad; ++j) {  // what is not of the tensor does not enter its block's maximum
            a[j] = j < L.n ? a[j] : 0.0f;
            r[j] = j < L.n ? r[j] : 0.0f;
        }
        float sm, sr;
        const uint32_t cm = encode4<false>(a, sm, how), cr = encode4<true>(r, sr, how);
        store_codes(s.m, L.arena, L.n, cm);
        store_codes(s.v, L.arena, L.n, cr);
        if ((threadIdx.x & 31) == 0 && L.n > 0) {
            s.ms[L.arena / kListBlock] = sm;
            s.vs[L.arena / kListBlock] = sr;
        }
    }
};

template <>
struct Moments<DOPT_STATE_E4M3_SR> : Moments<DOPT_STATE_E4M3> {};

// How a step of a kind rounds, for the 4 elements at L; t: its number.
template <int ST>
__device__ __forceinline__ auto rounding(const Place &L, int64_t t, const void *seed) {
    if constexpr (ST == DOPT_STATE_E4M3_SR)
        return random4(static_cast<uint64_t>(L.arena) / kQuad, static_cast<uint64_t>(t),
                       *static_cast<const uint64_t *>(seed));
    else return Nearest{};
}

// ---- pass 1: sum of squares and zero count ----------------------------------------
//
// As the flat step's pass 1: g = fp32(raw) * inv_scale, g*g exact in double,
// one partial per workgroup, added in index order.  A workgroup reads
// kListStatsTiles consecutive tiles per iteration, all loads before the first
// use.  The partials of a small list are added by the workgroup that finishes
// last, those of a larger one by a kernel of their own (kListFused).

struct StatsArgs {
    const ListTile *tiles;
    int64_t t_begin, t_end;
    int32_t first, part0;   // first tensor and first partial of the launch
    int32_t total;          // partials of all launches of the pass
    int32_t finalize;       // 0: the record only
    DevState *st;
    Partial *part;
    uint32_t *done;         // FUSED: workgroups that have finished; zero between passes
    Record *rec;
    StepRec *sr;
    dopt_stats *out;
    FinalizeArgs fa;
};
static_assert(sizeof(ListAddr) <= 3936 && sizeof(GradAddr) + sizeof(StatsArgs) <= 4096,
              "addresses must fit the kernel argument space");

// A wave's sums by a fixed butterfly.
__device__ __forceinline__ void wave_sum(double &acc, unsigned long long &z) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        acc += __shfl_xor(acc, off, 64);
        z += __shfl_xor(z, off, 64);
    }
}

// The sum of the partials in a fixed order (thread i adds partials i, i +
// THREADS, ...; each wave folds its lanes; thread 0 adds the waves), the
// record and the finalize, by one whole workgroup.  The hyper-groups' scalars
// are formed for the step that follows a clean pass while the loads are in
// flight, and stored if the pass was clean.
// AGENT: the partials were written by workgroups of this launch, on any XCD.
template <int THREADS, int BATCH, bool AGENT>
__device__ __forceinline__ void finish_stats(const StatsArgs &a) {
    __shared__ double f_acc[THREADS / 64];
    __shared__ unsigned long long f_z[THREADS / 64];
    __shared__ int f_skip;
    const DevState cur = *a.st;
    double acc = 0.0;
    unsigned long long z = 0;
    Hp mine{};
    for (int32_t i0 = threadIdx.x; i0 < a.total; i0 += BATCH * THREADS) {
        double s[BATCH];
        unsigned long long q[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int32_t i = i0 + j * THREADS < a.total ? i0 + j * THREADS : a.total - 1;
            if (AGENT) {
                s[j] = __hip_atomic_load(&a.part[i].sumsq, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                q[j] = __hip_atomic_load(&a.part[i].zeros, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            } else {
                const Partial x = a.part[i];
                s[j] = x.sumsq;
                q[j] = x.zeros;
            }
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const bool in = i0 + j * THREADS < a.total;  // a clamped duplicate adds +0
            acc += in ? s[j] : 0.0;
            z += in ? q[j] : 0ull;
        }
    }
    // the last wave, whose partials are the fewest
    const int h = static_cast<int>(threadIdx.x) - (THREADS - 64);
    if (a.finalize && h >= 0 && h < a.fa.nh) mine = step_scalars(a.fa.hp[h], static_cast<double>(cur.t + 1));
    wave_sum(acc, z);
    if ((threadIdx.x & 63) == 0) {
        f_acc[threadIdx.x >> 6] = acc;
        f_z[threadIdx.x >> 6] = z;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        unsigned long long tz = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            t += f_acc[w];
            tz += f_z[w];
        }
        a.rec->sumsq = t;
        a.rec->zeros = static_cast<double>(tz);
        f_skip = isfinite(t) ? 0 : 1;
        if (a.finalize) decide_step(t, static_cast<double>(tz), cur, a.st, a.sr, a.out, a.fa.max_norm);
    }
    __syncthreads();
    if (a.finalize && !f_skip && h >= 0 && h < a.fa.nh) store_scalars(a.sr, h, mine);
}

// One unscaled grad; a slot of no element (in false) holds 0 and adds +0.
__device__ __forceinline__ void add_grad(float x, bool in, double &acc, uint32_t &zeros) {
    const double xd = static_cast<double>(x);
    acc = fma(xd, xd, acc);
    zeros += (in && x == 0.0f) ? 1u : 0u;
}

// One round adds 4096 partials; on MI355X the statistics of 1.2e8 grads (3803 of them)
// took 46.4 us with 512 threads, 46.8 with 256 and 48.0 with 1024.
constexpr int kFinishThreads = 512;
template <int THREADS, int BATCH>
__global__ void __launch_bounds__(THREADS) k_list_finish(StatsArgs a) {
    finish_stats<THREADS, BATCH, false>(a);
}

template <int GD, bool FUSED, bool KEEP>
__global__ void __launch_bounds__(kBlock) k_list_stats(StatsArgs a, GradAddr addr) {
    const float inv = a.st->inv_scale;
    double acc = 0.0;
    uint32_t zeros = 0;  // of one lane: at most its share of 2^38 elements over its workgroup's 256
    for (int64_t t0 = a.t_begin + int64_t(blockIdx.x) * kListStatsTiles; t0 < a.t_end;
         t0 += int64_t(gridDim.x) * kListStatsTiles) {
        typename Quad<GD>::Raw raw[kListStatsTiles][kGroups];
        int n[kListStatsTiles][kGroups];
#pragma unroll
        for (int u = 0; u < kListStatsTiles; ++u) {
            const ListTile d = a.tiles[t0 + u < a.t_end ? t0 + u : a.t_end - 1];
            const void *g = grad_of(addr, d.index, a.first);
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                const Place L = place_of<kGroups>(d, k, threadIdx.x);
                n[u][k] = t0 + u < a.t_end ? L.n : 0;
                raw[u][k] = load4<GD, KEEP>(g, L.e, n[u][k]);
            }
        }
#pragma unroll
        for (int u = 0; u < kListStatsTiles; ++u)
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                float g[kQuad];
                unpack4<GD>(raw[u][k], g);
#pragma unroll
                for (int j = 0; j < kQuad; ++j) add_grad(g[j] * inv, j < n[u][k], acc, zeros);
            }
    }
    __shared__ double s_acc[kBlock / 64];
    __shared__ unsigned long long s_z[kBlock / 64];
    __shared__ bool s_last;
    unsigned long long z = zeros;
    wave_sum(acc, z);
    if ((threadIdx.x & 63) == 0) {
        s_acc[threadIdx.x >> 6] = acc;
        s_z[threadIdx.x >> 6] = z;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        unsigned long long tz = 0;
#pragma unroll
        for (int w = 0; w < kBlock / 64; ++w) {
            t += s_acc[w];
            tz += s_z[w];
        }
        Partial *dst = a.part + a.part0 + blockIdx.x;
        if (!FUSED) {
            dst->sumsq = t;
            dst->zeros = tz;
        } else {
            // the partial goes past this XCD's L2, and the count is released after it
            __hip_atomic_store(&dst->sumsq, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&dst->zeros, tz, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            s_last = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == uint32_t(a.total) - 1;
        }
    }
    if constexpr (FUSED) {
        __syncthreads();
        if (!s_last) return;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        if (threadIdx.x == 0) __hip_atomic_store(a.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        finish_stats<kBlock, 1, true>(a);
    }
}

__global__ void k_list_done(uint32_t *done) {
    if (threadIdx.x == 0) *done = 0;
}

__global__ void k_list_seed(uint64_t *dst, uint64_t seed) {
    if (threadIdx.x == 0) *dst = seed;
}

// ---- pass 2 -------------------------------------------------------------------------

// 512 threads to a tile, one group to a wave: as fast as 256 with two for fp32
// moments and faster for e4m3 ones (1.0e9 elements 2.85 and 2.92 ms, 1.8e7 in 500
// tensors 56.9 and 59.0 us; 128 with four lose 1 to 8%).
template <int PD, int GD, int ST>
__global__ void __launch_bounds__(kWide) k_list_apply(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                     int64_t t_end, int32_t first, StateArrays s,
                                                     const StepRec *__restrict__ rec, ListAddr addr) {
    // the records lie at fixed distances from one another
    const char *ws = reinterpret_cast<const char *>(rec) - kWsStepRec;
    const int skip = rec->skip;  // loaded beside the tile: a skipped step touches no data
    const ListTile d = tiles[t_begin + tile_of(blockIdx.x, t_end - t_begin)];
    if (skip) return;
    const dopt_list_ptrs q = ptrs_of(addr, d.index, first);
    const Hp h = load_hp(rec, d.packed >> 16);
    const Place L = place_of<1>(d, 0, threadIdx.x);
    const auto graw = load4<GD>(q.grad, L.e, L.n);
    const u32x4 praw = PD == DOPT_F32 ? load4<DOPT_F32>(q.param, L.e, L.n) : load4<DOPT_F32>(s.master, L.arena, L.n);
    Moments<ST> mom;
    mom.load(s, L);
    float g[kQuad], p[kQuad], a[kQuad], b[kQuad], r[kQuad];
    unpack4<GD>(graw, g);
    unpack4<DOPT_F32>(praw, p);
    mom.decode(a, b);
#pragma unroll
    for (int j = 0; j < kQuad; ++j)
        r[j] = adamw_root(g[j], p[j], a[j], b[j], rec->inv_scale, rec->clip_on, rec->clip, h);
    Moments<ST>::store(s, L, a, b, r,
                       rounding<ST>(L, reinterpret_cast<const DevState *>(ws + kWsState)->t, ws + kWsListSeed));
    if (PD != DOPT_F32) store4<DOPT_F32>(s.master, L.arena, L.n, p);
    store4<PD>(q.param, L.e, L.n, p);
}

// ---- the whole step of a small list ---------------------------------------------------
//
// At most kSmallTiles tiles: one workgroup of that many times kBlock threads
// takes both passes, a quarter a tile, and sums, stats and results are those
// of the two launches bit for bit.  Everything is read once, before anything
// is waited for; pass 1 takes the grads over LDS in the order of its own
// kernel, and the hyper-groups' scalars are formed meanwhile.  Latency is all
// there is here, and what four waves of a SIMD compute one after the other:
// groups without elements are left out (pass 2 of a large list, where they
// are rare, ran 1.5% slower with that test).  On MI355X, back to back, a step
// of 4 bf16 tensors of 500 elements takes 7.7 us with e4m3 moments and 6.8 with fp32
// ones, 12.2 and 11.8 in two launches; four whole tiles take 11.3 and 9.3,
// 11.6 and 10.5 in two.
// Arrays of the arguments are indexed with scalars: their elements are whole
// words, for scalar loads ignore the low two bits of each part of an address.
struct SmallTile {
    ListTile t;
    dopt_list_ptrs p;
    int32_t pd, gd;
};
struct SmallRun {
    int32_t first, n;
};
struct SmallArgs {
    StateArrays s;
    DevState *st;
    Record *rec;
    StepRec *sr;
    dopt_stats *out;
    int32_t n_tiles, n_runs;
    SmallTile tiles[kSmallTiles];
    SmallRun runs[kSmallTiles];  // the tiles of pass 1's partials
    FinalizeArgs fa;
};
static_assert(sizeof(SmallTile) % 4 == 0 && sizeof(SmallRun) % 4 == 0, "scalar loads take whole words");
static_assert(sizeof(SmallArgs) <= 4096, "the list must fit the kernel argument space");

// load4, unpack4 and store4 of a type that is an argument.
__device__ __forceinline__ u32x4 load4_any(int dt, const void *base, int64_t i, int n) {
    if (dt == DOPT_F32) return load4<DOPT_F32>(base, i, n);
    const u32x2 r = load4<DOPT_BF16>(base, i, n);  // the bits of either 16-bit type
    return u32x4{r[0], r[1], 0, 0};
}
__device__ __forceinline__ void unpack4_any(int dt, u32x4 r, float (&x)[kQuad]) {
    if (dt == DOPT_F32) unpack4<DOPT_F32>(r, x);
    else if (dt == DOPT_BF16) unpack4<DOPT_BF16>(u32x2{r[0], r[1]}, x);
    else unpack4<DOPT_F16>(u32x2{r[0], r[1]}, x);
}
__device__ __forceinline__ void store4_any(int dt, void *base, int64_t i, int n, const float (&x)[kQuad]) {
    if (dt == DOPT_F32) store4<DOPT_F32>(base, i, n, x);
    else if (dt == DOPT_BF16) store4<DOPT_BF16>(base, i, n, x);
    else store4<DOPT_F16>(base, i, n, x);
}

template <int ST>
__global__ void __launch_bounds__(kSmallTiles * kBlock) k_list_small(SmallArgs a) {
    __shared__ float s_g[kSmallTiles][kGroups][kQuad][kBlock];
    __shared__ double s_acc[kSmallTiles][kBlock / 64];
    __shared__ unsigned long long s_z[kSmallTiles][kBlock / 64];
    __shared__ StepRec s_rec;
    const int mine = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kBlock);  // this quarter's tile
    // its threads, a wave further round in each quarter: wave w of a workgroup runs on
    // SIMD w % 4, and the first waves of small tiles, often the only ones with work, would
    // all wait for one
    const int thread = (static_cast<int>(threadIdx.x) + mine * 64) % kBlock;
    const SmallTile t = a.tiles[mine];  // of no element beyond n_tiles
    float *const master = a.s.master;
    const DevState cur = *a.st;
    Place L[kGroups];
    u32x4 graw[kGroups], praw[kGroups];
    Moments<ST> mom[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        if (!group_lives(t.t, k, thread)) continue;
        L[k] = place_of<kGroups>(t.t, k, thread);
        graw[k] = load4_any(t.gd, t.p.grad, L[k].e, L[k].n);
        praw[k] = t.pd == DOPT_F32 ? load4<DOPT_F32>(t.p.param, L[k].e, L[k].n)
                                   : load4<DOPT_F32>(master, L[k].arena, L[k].n);
        mom[k].load(a.s, L[k]);
    }
    Hp scal{};
    const int h = static_cast<int>(threadIdx.x) - (kSmallTiles * kBlock - 64);  // the last wave's lanes
    if (h >= 0 && h < a.fa.nh) scal = step_scalars(a.fa.hp[h], static_cast<double>(cur.t + 1));
    float g[kGroups][kQuad];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        if (!group_lives(t.t, k, thread)) continue;
        unpack4_any(t.gd, graw[k], g[k]);
#pragma unroll
        for (int j = 0; j < kQuad; ++j) s_g[mine][k][j][thread] = g[k][j];
    }
    __syncthreads();
    // pass 1: quarter r adds partial r
    if (mine < a.n_runs) {
        double acc = 0.0;
        uint32_t zeros = 0;
        for (int u = a.runs[mine].first; u < a.runs[mine].first + a.runs[mine].n; ++u) {
            const ListTile d = a.tiles[u].t;
            const int count = static_cast<int>(d.packed & 0xffffu);
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                if (!group_lives(d, k, thread)) continue;  // it would add +0
#pragma unroll
                for (int j = 0; j < kQuad; ++j)
                    add_grad(s_g[u][k][j][thread] * cur.inv_scale, lane_offset<kGroups>(k, thread) + j < count, acc, zeros);
            }
        }
        unsigned long long z = zeros;
        wave_sum(acc, z);
        if ((thread & 63) == 0) {
            s_acc[mine][thread >> 6] = acc;
            s_z[mine][thread >> 6] = z;
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        double acc = 0.0;
        unsigned long long z = 0;
        if (static_cast<int>(threadIdx.x) < a.n_runs)
#pragma unroll
            for (int w = 0; w < kBlock / 64; ++w) {
                acc += s_acc[threadIdx.x][w];
                z += s_z[threadIdx.x][w];
            }
        wave_sum(acc, z);
        if (threadIdx.x == 0) {
            a.rec->sumsq = acc;
            a.rec->zeros = static_cast<double>(z);
            decide_step(acc, static_cast<double>(z), cur, a.st, &s_rec, a.out, a.fa.max_norm);
            a.sr->skip = s_rec.skip;
            a.sr->inv_scale = s_rec.inv_scale;
            a.sr->clip_on = s_rec.clip_on;
            a.sr->clip = s_rec.clip;
        }
    }
    if (h >= 0 && h < a.fa.nh) store_scalars(&s_rec, h, scal);
    __syncthreads();
    if (s_rec.skip) return;
    if (h >= 0 && h < a.fa.nh) store_scalars(a.sr, h, scal);
    // pass 2
    const Hp hp = load_hp(&s_rec, t.t.packed >> 16);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        if (!group_lives(t.t, k, thread)) continue;
        float p[kQuad], x[kQuad], y[kQuad], root[kQuad];
        unpack4<DOPT_F32>(praw[k], p);
        mom[k].decode(x, y);
#pragma unroll
        for (int j = 0; j < kQuad; ++j)
            root[j] = adamw_root(g[k][j], p[j], x[j], y[j], s_rec.inv_scale, s_rec.clip_on, s_rec.clip, hp);
        Moments<ST>::store(a.s, L[k], x, y, root,
                           rounding<ST>(L[k], cur.t + 1,
                                        reinterpret_cast<const char *>(a.rec) + (kWsListSeed - kWsRecord)));
        if (t.pd != DOPT_F32) store4<DOPT_F32>(master, L[k].arena, L[k].n, p);
        store4_any(t.pd, t.p.param, L[k].e, L[k].n, p);
    }
}

// ---- export, import, init -----------------------------------------------------------

struct ExportArrays {
    float *p, *m, *v;
};

// The import takes a lane of a tile's 512 per 4 elements, as pass 2; the
// export, which writes three arrays for one and a half that it reads, runs
// better with 256 and two groups each (1.2e8 elements on MI355X: import 395 and
// 411 us, export 401 and 377).
template <int PD, int ST>
__global__ void __launch_bounds__(kBlock) k_list_export(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                       int64_t t_end, int32_t first,
                                                       const int64_t *__restrict__ xoff, StateArrays s,
                                                       ExportArrays x, ListAddr addr) {
    const ListTile d = tiles[t_begin + tile_of(blockIdx.x, t_end - t_begin)];
    const void *param = ptrs_of(addr, d.index, first).param;
    const int64_t o = xoff[d.index];
    Place L[kGroups];
    u32x4 praw[kGroups];
    Moments<ST> mom[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        L[k] = place_of<kGroups>(d, k, threadIdx.x);
        praw[k] = PD == DOPT_F32 ? load4<DOPT_F32>(param, L[k].e, L[k].n) : load4<DOPT_F32>(s.master, L[k].arena, L[k].n);
        mom[k].load(s, L[k]);
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        float p[kQuad], a[kQuad], b[kQuad];
        unpack4<DOPT_F32>(praw[k], p);
        mom[k].decode(a, b);
        store4<DOPT_F32>(x.p, o + L[k].e, L[k].n, p);
        store4<DOPT_F32>(x.m, o + L[k].e, L[k].n, a);
        store4<DOPT_F32>(x.v, o + L[k].e, L[k].n, b);
    }
}

template <int PD, int ST>
__global__ void __launch_bounds__(kWide) k_list_import(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                      int64_t t_end, int32_t first,
                                                      const int64_t *__restrict__ xoff, StateArrays s,
                                                      ExportArrays x, ListAddr addr) {
    const ListTile d = tiles[t_begin + tile_of(blockIdx.x, t_end - t_begin)];
    void *param = ptrs_of(addr, d.index, first).param;
    const int64_t o = xoff[d.index];
    const Place L = place_of<1>(d, 0, threadIdx.x);
    const u32x4 praw = load4<DOPT_F32>(x.p, o + L.e, L.n);
    const u32x4 araw = load4<DOPT_F32>(x.m, o + L.e, L.n);
    const u32x4 braw = load4<DOPT_F32>(x.v, o + L.e, L.n);
    float p[kQuad], a[kQuad], b[kQuad], r[kQuad];
    unpack4<DOPT_F32>(praw, p);
    unpack4<DOPT_F32>(araw, a);
    unpack4<DOPT_F32>(braw, b);
    if (PD != DOPT_F32) store4<DOPT_F32>(s.master, L.arena, L.n, p);
    store4<PD>(param, L.e, L.n, p);
#pragma unroll
    for (int j = 0; j < kQuad; ++j) r[j] = ST == DOPT_STATE_E4M3 ? sqrtf(b[j]) : 0.0f;
    Moments<ST>::store(s, L, a, b, r, Nearest{});
}

// Masters from the params, everything else zero, whole blocks of the arena.
template <int PD, int ST>
__global__ void __launch_bounds__(kWide) k_list_init(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                    int32_t first, bool masters, StateArrays s, ListAddr addr) {
    const float z[kQuad] = {0, 0, 0, 0};
    const ListTile d = tiles[t_begin + blockIdx.x];
    const int count = static_cast<int>(d.packed & 0xffffu);
    const Place L = place_of<1>(d, 0, threadIdx.x);
    const int n = L.n + (count + kListBlock - 1) / kListBlock * kListBlock - count;  // slots of the tensor's blocks
    if (n <= 0) return;
    if (masters) {
        float p[kQuad] = {0, 0, 0, 0};
        if (PD != DOPT_F32) unpack4<PD>(load4<PD>(ptrs_of(addr, d.index, first).param, L.e, L.n), p);
        store4<DOPT_F32>(s.master, L.arena, n, p);
    }
    if constexpr (ST == DOPT_STATE_E4M3) {
        store_codes(s.m, L.arena, n, 0);
        store_codes(s.v, L.arena, n, 0);
        if ((threadIdx.x & 31) == 0) {
            s.ms[L.arena / kListBlock] = 0.0f;
            s.vs[L.arena / kListBlock] = 0.0f;
        }
    } else {
        store4<DOPT_F32>(s.m, L.arena, n, z);
        store4<DOPT_F32>(s.v, L.arena, n, z);
    }
}

// ---- host side ------------------------------------------------------------------------

static int check_list(const dopt_list *P, const void *ws) {
    if (!P || !ws) return fail(DOPT_ERR_INVALID, "null list or workspace");
    if (!aligned(ws)) return fail(DOPT_ERR_INVALID, "workspace is not 256-byte aligned");
    return DOPT_OK;
}

static int check_tensors(const dopt_list *P, const dopt_list_ptrs *ts, bool grads, bool params) {
    if (!ts && !P->tensors.empty()) return fail(DOPT_ERR_INVALID, "null tensor array");
    for (size_t i = 0; i < P->tensors.size(); ++i) {
        const ListTensor &T = P->tensors[i];
        if (T.numel == 0) continue;
        const uintptr_t g = reinterpret_cast<uintptr_t>(ts[i].grad), p = reinterpret_cast<uintptr_t>(ts[i].param);
        if ((grads && !g) || (params && !p))
            return fail(DOPT_ERR_INVALID, "tensor " + std::to_string(i) + ": null device pointer");
        if ((grads && g % (T.gd == DOPT_F32 ? 4 : 2)) || (params && p % (T.pd == DOPT_F32 ? 4 : 2)))
            return fail(DOPT_ERR_INVALID, "tensor " + std::to_string(i) + ": device pointer not aligned to its element");
    }
    return DOPT_OK;
}

static int check_state(const dopt_list *P, const dopt_list_state *s, StateArrays &out) {
    if (!s) return fail(DOPT_ERR_INVALID, "null state");
    const bool e = P->state_kind != DOPT_STATE_F32;
    if (P->arena_numel > 0) {
        const void *need[] = {s->exp_avg, s->exp_avg_sq, P->has_master ? s->master : s->exp_avg,
                              e ? static_cast<const void *>(s->exp_avg_scale) : s->exp_avg,
                              e ? static_cast<const void *>(s->exp_avg_sq_scale) : s->exp_avg};
        for (const void *p : need) {
            if (!p) return fail(DOPT_ERR_INVALID, "state: null device pointer");
            if (!aligned(p)) return fail(DOPT_ERR_INVALID, "state: device pointer not 256-byte aligned");
        }
    }
    out = StateArrays{s->master, s->exp_avg, s->exp_avg_sq, s->exp_avg_scale, s->exp_avg_sq_scale};
    return DOPT_OK;
}

static bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + static_cast<uint64_t>(b_bytes) && y < x + static_cast<uint64_t>(a_bytes);
}

// The arrays of an export or import against one another, the params and the
// state, which the same launches read and write in another order.  A master
// array may be the fp32 params themselves: their elements go onto themselves.
static int check_copies(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *st, const float *const (&x)[3],
                        bool written) {
    static const char *const kNames[3] = {"master", "exp_avg", "exp_avg_sq"};
    const int64_t bytes = P->numel * 4;
    if (P->numel == 0) return DOPT_OK;
    for (const float *p : x)
        if (!p) return fail(DOPT_ERR_INVALID, "null export array");
    for (const float *p : x)
        if (reinterpret_cast<uintptr_t>(p) % 4) return fail(DOPT_ERR_INVALID, "export array not 4-byte aligned");
    const bool e = P->state_kind != DOPT_STATE_F32;
    const int64_t held = P->arena_numel * (e ? 1 : 4), scales = e ? P->arena_numel / kListBlock * 4 : 0;
    const struct {
        const char *name;
        const void *p;
        int64_t bytes;
    } state[] = {{"master", st->master, P->has_master ? P->arena_numel * 4 : 0},
                 {"exp_avg", st->exp_avg, held},
                 {"exp_avg_sq", st->exp_avg_sq, held},
                 {"exp_avg_scale", st->exp_avg_scale, scales},
                 {"exp_avg_sq_scale", st->exp_avg_sq_scale, scales}};
    for (int i = 0; i < 3; ++i) {
        for (int k = 0; written && k < i; ++k)
            if (overlap(x[i], bytes, x[k], bytes))
                return fail(DOPT_ERR_INVALID, std::string(kNames[i]) + " array overlaps the " + kNames[k] + " array");
        for (const auto &s : state)
            if (s.bytes > 0 && overlap(x[i], bytes, s.p, s.bytes))
                return fail(DOPT_ERR_INVALID, std::string(kNames[i]) + " array overlaps state " + s.name);
        for (size_t t = 0; t < P->tensors.size(); ++t) {
            const ListTensor &T = P->tensors[t];
            if (T.numel == 0 || !overlap(x[i], bytes, ts[t].param, T.numel * (T.pd == DOPT_F32 ? 4 : 2))) continue;
            if (i == 0 && T.pd == DOPT_F32 && static_cast<const void *>(x[0] + T.xoff) == ts[t].param) continue;
            return fail(DOPT_ERR_INVALID, std::string(kNames[i]) + " array overlaps param " + std::to_string(t));
        }
    }
    return DOPT_OK;
}

static const ListTile *tiles_of(const ListClass &C, const void *ws) {
    return reinterpret_cast<const ListTile *>(static_cast<const char *>(ws) + C.ws_tiles);
}

// The lowest address of n of a kind, and the others' distances from it in
// units of the largest power of two that divides them all.
struct Span {
    uintptr_t lo = UINTPTR_MAX, hi = 0, bits = 0;
    template <class At>  // the i-th address
    Span(int32_t n, At at) {
        for (int32_t i = 0; i < n; ++i) {
            lo = std::min(lo, reinterpret_cast<uintptr_t>(at(i)));
            hi = std::max(hi, reinterpret_cast<uintptr_t>(at(i)));
        }
        for (int32_t i = 0; i < n; ++i) bits |= reinterpret_cast<uintptr_t>(at(i)) - lo;
    }
    uint32_t shift() const { return bits ? static_cast<uint32_t>(__builtin_ctzll(bits)) : 0; }
    bool fits() const { return !bits || (hi - lo) >> shift() <= UINT32_MAX; }
    uint32_t from(const void *p) const {
        return static_cast<uint32_t>((reinterpret_cast<uintptr_t>(p) - lo) >> shift());
    }
};

static Span grad_span(const ListClass &C, const ListRange &r, const dopt_list_ptrs *ts) {
    return Span(r.count, [&](int32_t i) { return ts[C.tensors[static_cast<size_t>(r.first + i)]].grad; });
}
static Span param_span(const ListClass &C, const ListRange &r, const dopt_list_ptrs *ts) {
    return Span(r.count, [&](int32_t i) { return ts[C.tensors[static_cast<size_t>(r.first + i)]].param; });
}

// Per class the table of its addresses in the workspace, or null where every
// launch's addresses fit its arguments.
struct Tables {
    const dopt_list_ptrs *of[kDtypes * kDtypes];  // a class per pair of element types
};

static bool fits(const ListClass &C, const std::vector<ListRange> &ranges, const dopt_list_ptrs *ts, bool grads,
                 bool params) {
    for (const ListRange &r : ranges)
        if ((grads && !grad_span(C, r, ts).fits()) || (params && !param_span(C, r, ts).fits())) return false;
    return true;
}

// Writes the addresses of the classes that need it into the workspace, for
// pass 1, pass 2 (or a copy, which takes no grads) or both.
static int place_addresses(const dopt_list *P, const dopt_list_ptrs *ts, bool pass1, bool pass2, bool grads, void *ws,
                           hipStream_t stream, Tables &tables) {
    for (size_t c = 0; c < P->classes.size(); ++c) {
        const ListClass &C = P->classes[c];
        tables.of[c] = nullptr;
        if ((!pass1 || fits(C, C.stats, ts, true, false)) && (!pass2 || fits(C, C.apply, ts, grads, true))) continue;
        dopt_list_ptrs *dst = reinterpret_cast<dopt_list_ptrs *>(ws_ptr(ws, C.ws_addr));
        const int32_t n = static_cast<int32_t>(C.tensors.size());
        for (int32_t f = 0; f < n; f += kListPut) {
            PutAddr a;
            std::memset(&a, 0, sizeof a);
            const int32_t m = std::min(kListPut, n - f);
            for (int32_t i = 0; i < m; ++i) a.p[i] = ts[C.tensors[static_cast<size_t>(f + i)]];
            k_list_put<<<1, kBlock, 0, stream>>>(dst + f, m, a);
            const int rc = check_launch("launch k_list_put");
            if (rc) return rc;
        }
        tables.of[c] = dst;
    }
    return DOPT_OK;
}

static void fill(ListAddr &a, const ListClass &C, const ListRange &r, const dopt_list_ptrs *ts, bool grads,
                 const dopt_list_ptrs *table) {
    std::memset(&a, 0, sizeof a);
    a.table = table;
    if (table) return;
    const Span p = param_span(C, r, ts);
    a.param0 = reinterpret_cast<char *>(p.lo);
    a.param_shift = p.shift();
    for (int32_t i = 0; i < r.count; ++i) a.s[i].param = p.from(ts[C.tensors[static_cast<size_t>(r.first + i)]].param);
    if (!grads) return;
    const Span g = grad_span(C, r, ts);
    a.grad0 = reinterpret_cast<const char *>(g.lo);
    a.grad_shift = g.shift();
    for (int32_t i = 0; i < r.count; ++i) a.s[i].grad = g.from(ts[C.tensors[static_cast<size_t>(r.first + i)]].grad);
}

static void fill(GradAddr &a, const ListClass &C, const ListRange &r, const dopt_list_ptrs *ts,
                 const dopt_list_ptrs *table) {
    std::memset(&a, 0, sizeof a);
    a.table = table;
    if (table) return;
    const Span g = grad_span(C, r, ts);
    a.grad0 = reinterpret_cast<const char *>(g.lo);
    a.grad_shift = g.shift();
    for (int32_t i = 0; i < r.count; ++i) a.grad[i] = g.from(ts[C.tensors[static_cast<size_t>(r.first + i)]].grad);
}

// Calls f with an element type as a compile-time constant.
template <int DT>
struct Const {
    static constexpr int value = DT;
};
template <class F>
static void with_dtype(int dt, F f) {
    if (dt == DOPT_BF16) f(Const<DOPT_BF16>());
    else if (dt == DOPT_F16) f(Const<DOPT_F16>());
    else f(Const<DOPT_F32>());
}
// The kind of a list's moments, in a step: how they are held and rounded.
template <class F>
static void with_state(int kind, F f) {
    if (kind == DOPT_STATE_E4M3) f(Const<DOPT_STATE_E4M3>());
    else if (kind == DOPT_STATE_E4M3_SR) f(Const<DOPT_STATE_E4M3_SR>());
    else f(Const<DOPT_STATE_F32>());
}
// In the calls that round to nearest or not at all: how they are held.
template <class F>
static void with_held(int kind, F f) {
    if (kind != DOPT_STATE_F32) f(Const<DOPT_STATE_E4M3>());
    else f(Const<DOPT_STATE_F32>());
}

// Pass 1 over every class; fa null: the record only.
static int launch_list_stats(const dopt_list *P, const dopt_list_ptrs *ts, const Tables &tables, void *ws,
                             hipStream_t stream, const FinalizeArgs *fa) {
    StatsArgs a;
    std::memset(&a, 0, sizeof a);
    a.total = P->total_partials;
    const bool fused = a.total > 0 && a.total <= kListFused;
    a.finalize = fa != nullptr;
    const bool keep = P->grad_bytes <= kListKeep;
    if (fa) a.fa = *fa;
    a.st = reinterpret_cast<DevState *>(ws_ptr(ws, kWsState));
    a.part = reinterpret_cast<Partial *>(ws_ptr(ws, kWsPartials));
    a.done = reinterpret_cast<uint32_t *>(ws_ptr(ws, kWsListDone));
    a.rec = reinterpret_cast<Record *>(ws_ptr(ws, kWsRecord));
    a.sr = reinterpret_cast<StepRec *>(ws_ptr(ws, kWsStepRec));
    a.out = reinterpret_cast<dopt_stats *>(ws_ptr(ws, kWsStats));
    for (size_t c = 0; c < P->classes.size(); ++c) {
        const ListClass &C = P->classes[c];
        a.tiles = tiles_of(C, ws);
        for (const ListRange &r : C.stats) {
            GradAddr g;
            fill(g, C, r, ts, tables.of[c]);
            a.t_begin = r.t0;
            a.t_end = r.t1;
            a.first = r.first;
            a.part0 = r.partial_base;
            with_dtype(C.gd, [&](auto gd) {
                constexpr int GD = decltype(gd)::value;
                if (fused) k_list_stats<GD, true, true><<<r.grid, kBlock, 0, stream>>>(a, g);
                else if (keep) k_list_stats<GD, false, true><<<r.grid, kBlock, 0, stream>>>(a, g);
                else k_list_stats<GD, false, false><<<r.grid, kBlock, 0, stream>>>(a, g);
            });
            const int rc = check_launch("launch k_list_stats");
            if (rc) {
                k_list_done<<<1, 64, 0, stream>>>(a.done);  // the pass is not complete: forget its count
                return rc;
            }
        }
    }
    if (fused) return DOPT_OK;
    k_list_finish<kFinishThreads, kFinishBatch><<<1, kFinishThreads, 0, stream>>>(a);
    return check_launch("launch k_list_finish");
}

// Pass 2 over every class.
static int launch_list_apply(const dopt_list *P, const dopt_list_ptrs *ts, const Tables &tables, const StateArrays &s,
                             void *ws, hipStream_t stream) {
    const StepRec *rec = reinterpret_cast<const StepRec *>(ws_ptr(ws, kWsStepRec));
    for (size_t c = 0; c < P->classes.size(); ++c) {
        const ListClass &C = P->classes[c];
        for (const ListRange &r : C.apply) {
            ListAddr a;
            fill(a, C, r, ts, true, tables.of[c]);
            with_dtype(C.pd, [&](auto pd) {
                with_dtype(C.gd, [&](auto gd) {
                    with_state(P->state_kind, [&](auto st) {
                        k_list_apply<decltype(pd)::value, decltype(gd)::value, decltype(st)::value>
                            <<<r.grid, kWide, 0, stream>>>(tiles_of(C, ws), r.t0, r.t1, r.first, s, rec, a);
                    });
                });
            });
            const int rc = check_launch("launch k_list_apply");
            if (rc) return rc;
        }
    }
    return DOPT_OK;
}

// Both passes of a list of at most kSmallTiles tiles.
static int launch_list_small(const dopt_list *P, const dopt_list_ptrs *ts, const StateArrays &s, const FinalizeArgs &fa,
                             void *ws, hipStream_t stream) {
    SmallArgs a;
    std::memset(&a, 0, sizeof a);
    a.s = s;
    a.st = reinterpret_cast<DevState *>(ws_ptr(ws, kWsState));
    a.rec = reinterpret_cast<Record *>(ws_ptr(ws, kWsRecord));
    a.sr = reinterpret_cast<StepRec *>(ws_ptr(ws, kWsStepRec));
    a.out = reinterpret_cast<dopt_stats *>(ws_ptr(ws, kWsStats));
    a.fa = fa;
    for (const ListClass &C : P->classes) {
        const int n = static_cast<int>(C.tiles.size());
        for (int t = 0; t < n; ++t) {
            const int i = a.n_tiles + t;
            const ListTile &d = C.tiles[static_cast<size_t>(t)];
            a.tiles[i] = SmallTile{d, ts[C.tensors[d.index]], C.pd, C.gd};
        }
        for (int t = 0; t < n; t += kListStatsTiles)
            a.runs[a.n_runs++] = SmallRun{a.n_tiles + t, std::min(kListStatsTiles, n - t)};
        a.n_tiles += n;
    }
    with_state(P->state_kind,
               [&](auto st) { k_list_small<decltype(st)::value><<<1, kSmallTiles * kBlock, 0, stream>>>(a); });
    return check_launch("launch k_list_small");
}

template <bool IMPORT>
static int list_copy(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, ExportArrays x,
                     void *ws, hipStream_t stream) {
    StateArrays s;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, false, true)) || (rc = check_state(P, state, s))) return rc;
    if ((rc = check_copies(P, ts, state, {x.p, x.m, x.v}, !IMPORT))) return rc;
    Tables tables;
    if ((rc = place_addresses(P, ts, false, true, false, ws, stream, tables))) return rc;
    for (size_t c = 0; c < P->classes.size(); ++c) {
        const ListClass &C = P->classes[c];
        for (const ListRange &r : C.apply) {
            ListAddr a;
            fill(a, C, r, ts, false, tables.of[c]);
            const int64_t *xoff = reinterpret_cast<const int64_t *>(ws_ptr(ws, C.ws_xoff));
            with_dtype(C.pd, [&](auto pd) {
                with_held(P->state_kind, [&](auto st) {
                    constexpr int PD = decltype(pd)::value, ST = decltype(st)::value;
                    if (IMPORT)
                        k_list_import<PD, ST><<<r.grid, kWide, 0, stream>>>(tiles_of(C, ws), r.t0, r.t1, r.first, xoff, s, x, a);
                    else
                        k_list_export<PD, ST><<<r.grid, kBlock, 0, stream>>>(tiles_of(C, ws), r.t0, r.t1, r.first, xoff, s, x, a);
                });
            });
            if ((rc = check_launch(IMPORT ? "launch k_list_import" : "launch k_list_export"))) return rc;
        }
    }
    return DOPT_OK;
}

}  // namespace dopt

using namespace dopt;

extern "C" {

int dopt_list_init(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state,
                   const dopt_scaler_cfg *sc, void *ws, hipStream_t stream) {
    StateArrays s;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, false, true)) || (rc = check_state(P, state, s)) || (rc = check_scaler(sc)))
        return rc;
    Tables tables;
    if ((rc = place_addresses(P, ts, false, true, false, ws, stream, tables))) return rc;
    for (size_t c = 0; c < P->classes.size(); ++c) {
        const ListClass &C = P->classes[c];
        rc = hip_check(hipMemcpyAsync(ws_ptr(ws, C.ws_tiles), C.tiles.data(), C.tiles.size() * sizeof(ListTile),
                                      hipMemcpyHostToDevice, stream),
                       "copy list tiles");
        if (rc) return rc;
        rc = hip_check(hipMemcpyAsync(ws_ptr(ws, C.ws_xoff), C.xoff.data(), C.xoff.size() * sizeof(int64_t),
                                      hipMemcpyHostToDevice, stream),
                       "copy list export offsets");
        if (rc) return rc;
        for (const ListRange &r : C.apply) {
            ListAddr a;
            fill(a, C, r, ts, false, tables.of[c]);
            with_dtype(C.pd, [&](auto pd) {
                with_held(P->state_kind, [&](auto st) {
                    k_list_init<decltype(pd)::value, decltype(st)::value><<<r.grid, kWide, 0, stream>>>(
                        tiles_of(C, ws), r.t0, r.first, P->has_master, s, a);
                });
            });
            if ((rc = check_launch("launch k_list_init"))) return rc;
        }
    }
    if ((rc = launch_init_records(*sc, ws, stream))) return rc;
    k_list_done<<<1, 64, 0, stream>>>(reinterpret_cast<uint32_t *>(ws_ptr(ws, kWsListDone)));
    if ((rc = check_launch("launch k_list_done"))) return rc;
    k_list_seed<<<1, 64, 0, stream>>>(reinterpret_cast<uint64_t *>(ws_ptr(ws, kWsListSeed)), 0);
    if ((rc = check_launch("launch k_list_seed"))) return rc;
    return hip_check(hipStreamSynchronize(stream), "synchronize after list init");
}

int dopt_list_stats(const dopt_list *P, const dopt_list_ptrs *ts, void *ws, hipStream_t stream) {
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, true, false))) return rc;
    Tables tables;
    if ((rc = place_addresses(P, ts, true, false, true, ws, stream, tables))) return rc;
    return launch_list_stats(P, ts, tables, ws, stream, nullptr);
}

int dopt_list_finalize(const dopt_list *P, const dopt_hparams *hp, int32_t n_hgroups, double max_grad_norm, void *ws,
                       hipStream_t stream) {
    FinalizeArgs a;
    int rc = check_list(P, ws);
    if (rc || (rc = build_finalize_args(P->max_hgroup, hp, n_hgroups, max_grad_norm, a))) return rc;
    return launch_finalize(a, ws, stream);
}

int dopt_list_prepare(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_hparams *hp, int32_t n_hgroups,
                      double max_grad_norm, void *ws, hipStream_t stream) {
    FinalizeArgs a;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, true, false)) ||
        (rc = build_finalize_args(P->max_hgroup, hp, n_hgroups, max_grad_norm, a)))
        return rc;
    Tables tables;
    if ((rc = place_addresses(P, ts, true, false, true, ws, stream, tables))) return rc;
    return launch_list_stats(P, ts, tables, ws, stream, &a);
}

int dopt_list_apply(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, void *ws,
                    hipStream_t stream) {
    StateArrays s;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, true, true)) || (rc = check_state(P, state, s))) return rc;
    Tables tables;
    if ((rc = place_addresses(P, ts, false, true, true, ws, stream, tables))) return rc;
    return launch_list_apply(P, ts, tables, s, ws, stream);
}

int dopt_list_step(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, const dopt_hparams *hp,
                   int32_t n_hgroups, double max_grad_norm, void *ws, hipStream_t stream, dopt_stats *out) {
    // everything is checked before the first launch: a refused call leaves the scaler and step count alone
    StateArrays s;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, true, true)) || (rc = check_state(P, state, s))) return rc;
    FinalizeArgs a;
    if ((rc = build_finalize_args(P->max_hgroup, hp, n_hgroups, max_grad_norm, a))) return rc;
    if (P->total_tiles > 0 && P->total_tiles <= kSmallTiles) {
        rc = launch_list_small(P, ts, s, a, ws, stream);
    } else {
        Tables tables;
        rc = place_addresses(P, ts, true, true, true, ws, stream, tables);  // once for both passes
        if (rc == DOPT_OK) rc = launch_list_stats(P, ts, tables, ws, stream, &a);
        if (rc == DOPT_OK) rc = launch_list_apply(P, ts, tables, s, ws, stream);
    }
    if (rc) return rc;
    return out ? copy_stats(ws, stream, out) : DOPT_OK;
}

int dopt_list_export(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, float *master,
                     float *exp_avg, float *exp_avg_sq, void *ws, hipStream_t stream) {
    return list_copy<false>(P, ts, state, ExportArrays{master, exp_avg, exp_avg_sq}, ws, stream);
}

int dopt_list_import(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, const float *master,
                     const float *exp_avg, const float *exp_avg_sq, void *ws, hipStream_t stream) {
    return list_copy<true>(P, ts, state,
                           ExportArrays{const_cast<float *>(master), const_cast<float *>(exp_avg),
                                        const_cast<float *>(exp_avg_sq)},
                           ws, stream);
}

int dopt_list_set_seed(const dopt_list *P, uint64_t seed, void *ws, hipStream_t stream) {
    const int rc = check_list(P, ws);
    if (rc) return rc;
    if (P->state_kind != DOPT_STATE_E4M3_SR) return fail(DOPT_ERR_INVALID, "only lists of kind E4M3_SR take a seed");
    k_list_seed<<<1, 64, 0, stream>>>(reinterpret_cast<uint64_t *>(ws_ptr(ws, kWsListSeed)), seed);
    return check_launch("launch k_list_seed");
}

int dopt_list_scalars_get(const dopt_list *P, const void *ws, hipStream_t stream, dopt_state_scalars *out) {
    if (!P || !ws || !out) return fail(DOPT_ERR_INVALID, "null list, workspace or output");
    return read_scalars(ws, stream, out);
}

int dopt_list_scalars_set(const dopt_list *P, void *ws, hipStream_t stream, const dopt_state_scalars *in) {
    if (!P || !ws || !in) return fail(DOPT_ERR_INVALID, "null list, workspace or input");
    return write_scalars(ws, stream, in);
}

int dopt_list_read_stats(const dopt_list *P, const void *ws, hipStream_t stream, dopt_stats *out) {
    if (!P || !ws || !out) return fail(DOPT_ERR_INVALID, "null list, workspace or output");
    return copy_stats(ws, stream, out);
}

}  // extern "C"
