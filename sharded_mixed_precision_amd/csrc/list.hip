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
// A list is cut into tiles of 2048 elements, one workgroup each, 8
// consecutive elements per lane: a block of 128 elements is then one row of
// 16 lanes, the group that the DPP lane permutes reduce over without LDS.
// Tensors start anywhere their element type allows, so params and grads go
// through 16-byte accesses of element alignment (gfx950 takes unaligned
// global accesses); the arena arrays are aligned.  The last lanes of a
// tensor's last tile take single elements: nothing outside a tensor is read.
#include "device.h"

#include "list.h"

namespace dopt {

// ---- tensor addresses ---------------------------------------------------------

struct ListPtrs {
    dopt_list_ptrs p[kListSlots];
};
struct GradPtrs {
    const void *p[kListGradSlots];
};
static_assert(sizeof(ListPtrs) <= 3840 && sizeof(GradPtrs) <= 3840, "addresses must fit the kernel argument space");

// ---- element I/O at element alignment -------------------------------------------

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x4 ldu(const uint16_t *p) { return *reinterpret_cast<const u32x4_a2 *>(p); }
__device__ __forceinline__ u32x4 ldu(const float *p) { return *reinterpret_cast<const u32x4_a4 *>(p); }
__device__ __forceinline__ void stu(uint16_t *p, u32x4 x) { *reinterpret_cast<u32x4_a2 *>(p) = x; }
__device__ __forceinline__ void stu(float *p, u32x4 x) { *reinterpret_cast<u32x4_a4 *>(p) = x; }

template <int DT>
struct Store {
    typedef uint16_t T;
};
template <>
struct Store<DOPT_F32> {
    typedef float T;
};

template <int DT>
__device__ __forceinline__ float up1(typename Store<DT>::T x) {
    if constexpr (DT == DOPT_F32) return x;
    else if constexpr (DT == DOPT_BF16) return __uint_as_float(uint32_t(x) << 16);
    else return Elem<DOPT_F16>::up(x);
}

template <int DT>
__device__ __forceinline__ typename Store<DT>::T down1(float x) {
    if constexpr (DT == DOPT_F32) return x;
    else return static_cast<uint16_t>(Elem<DT>::bits(x));
}

// Elements i .. i+7 of a tensor, of which the first n exist (n <= 0: none);
// the others read as 0.
template <int DT>
__device__ __forceinline__ Raw8 load_raw_n(const void *base, int64_t i, int n) {
    typedef typename Store<DT>::T T;
    const T *p = static_cast<const T *>(base) + i;
    Raw8 r{u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
    if (n >= kVec) {
        r.lo = ldu(p);
        if (DT == DOPT_F32) r.hi = ldu(p + 4);
    } else {
        for (int j = 0; j < kVec; ++j) {
            if (j >= n) break;
            if constexpr (DT == DOPT_F32) {
                if (j < 4) r.lo[j] = __float_as_uint(p[j]);
                else r.hi[j - 4] = __float_as_uint(p[j]);
            } else {
                r.lo[j >> 1] |= uint32_t(p[j]) << (16 * (j & 1));
            }
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void store_n(void *base, int64_t i, int n, const float (&x)[kVec]) {
    typedef typename Store<DT>::T T;
    T *p = static_cast<T *>(base) + i;
    if (n >= kVec) {
        if constexpr (DT == DOPT_F32) {
            stu(p, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])});
            stu(p + 4, u32x4{__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])});
        } else {
            u32x4 u;
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = Elem<DT>::bits(x[2 * j]) | (Elem<DT>::bits(x[2 * j + 1]) << 16);
            stu(p, u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[j] = down1<DT>(x[j]);
    }
}

// ---- e4m3 blocks ----------------------------------------------------------------

constexpr float kLeastScaled = 0x1p-100f;  // a block whose largest magnitude is below is held as zeros
constexpr float kCapM = 0x1p127f;
constexpr float kCapRoot = 0x1.fffffep63f;  // the largest fp32 number whose square is finite
constexpr float kTop = 448.0f, kLeast = 0x1p-9f;  // e4m3's largest and smallest magnitudes

__device__ __forceinline__ void decode8(u32x2 c, float scale, float (&x)[kVec]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[j]), false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[j]), true);
        x[4 * j] = a[0] * scale;
        x[4 * j + 1] = a[1] * scale;
        x[4 * j + 2] = b[0] * scale;
        x[4 * j + 3] = b[1] * scale;
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t row_max(uint32_t u) {
    const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, false));
    return u > o ? u : o;
}

// The largest magnitude over a row of 16 lanes, as fp32 bits: an unsigned
// maximum of the bits without their sign, in which NaN is above infinity and
// both above every number, so a NaN is never dropped.
__device__ __forceinline__ float block_max(const float (&x)[kVec]) {
    uint32_t u = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const uint32_t b = __float_as_uint(x[j]) & 0x7fffffffu;
        u = u > b ? u : b;
    }
    u = row_max<0xb1>(u);   // quad_perm 1,0,3,2
    u = row_max<0x4e>(u);   // quad_perm 2,3,0,1
    u = row_max<0x141>(u);  // row_half_mirror
    u = row_max<0x140>(u);  // row_mirror
    return __uint_as_float(u);
}

// Codes and scale of a block, all 16 lanes of its row together.  ROOT: a
// square root of v, whose nonzero values keep a nonzero code.
template <bool ROOT>
__device__ __forceinline__ u32x2 encode8(const float (&x)[kVec], float &scale) {
    const float a = block_max(x);
    const float cap = ROOT ? kCapRoot : kCapM;
    const bool live = !(a < kLeastScaled);
    scale = live ? (a > cap ? cap : a) * (1.0f / kTop) : 0.0f;  // a NaN passes both comparisons
    const float inv = live ? 1.0f / scale : 0.0f;
    u32x2 c;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float v = x[4 * j + k];
            q[k] = __builtin_amdgcn_fmed3f(v * inv, -kTop, kTop);
            if (ROOT) q[k] = v > 0.0f ? fmaxf(q[k], kLeast) : q[k];
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
        c[j] = live ? static_cast<uint32_t>(w) : 0u;
    }
    return c;
}

// 8 codes at arena element e, of which the first n exist (the others keep
// their bytes).
__device__ __forceinline__ void store_codes(void *base, int64_t e, int n, u32x2 c) {
    uint8_t *p = static_cast<uint8_t *>(base) + e;
    if (n >= kVec) {
        *reinterpret_cast<u32x2 *>(p) = c;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[j] = static_cast<uint8_t>(c[j >> 2] >> (8 * (j & 3)));
    }
}

// A lane's place in its tile.
struct Lane {
    int64_t e;      // the first of its 8 elements within the tensor
    int64_t arena;  // and in the arena
    int n;          // how many of them exist (<= 0: none)
    bool heads;     // first lane of a block that holds an element
};

__device__ __forceinline__ Lane lane_of(const ListTile &d) {
    const int l = static_cast<int>(threadIdx.x) * kVec;
    const int n = static_cast<int>(d.packed & 0xffffu) - l;
    return Lane{int64_t(d.tile) * kTile + l, int64_t(d.block) * kListBlock + l, n,
                (threadIdx.x & (kListBlock / kVec - 1)) == 0 && n > 0};
}

// ---- pass 1: sum of squares and zero count ----------------------------------------
//
// As the flat step's pass 1: g = fp32(raw) * inv_scale, g*g exact in double,
// one partial per workgroup, added in index order by k_finish.  It reads
// kListStatsTiles consecutive tiles per iteration.
template <int GD>
__global__ void __launch_bounds__(kBlock) k_list_stats(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                      int64_t t_end, int32_t first, const DevState *__restrict__ st,
                                                      Partial *__restrict__ out, GradPtrs ptrs) {
    const float inv = st->inv_scale;
    double acc = 0.0;
    uint32_t zeros = 0;
    for (int64_t t0 = t_begin + int64_t(blockIdx.x) * kListStatsTiles; t0 < t_end;
         t0 += int64_t(gridDim.x) * kListStatsTiles) {
        Raw8 raw[kListStatsTiles];
        int n[kListStatsTiles];
#pragma unroll
        for (int u = 0; u < kListStatsTiles; ++u) {
            n[u] = 0;
            if (t0 + u < t_end) {
                const ListTile d = tiles[t0 + u];
                const Lane L = lane_of(d);
                n[u] = L.n;
                raw[u] = load_raw_n<GD>(ptrs.p[d.index - first], L.e, L.n);
            }
        }
#pragma unroll
        for (int u = 0; u < kListStatsTiles; ++u) {
            float g[kVec];
            Elem<GD>::unpack(raw[u], g);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (j >= n[u]) continue;
                const float x = g[j] * inv;
                const double xd = static_cast<double>(x);
                acc = fma(xd, xd, acc);
                zeros += x == 0.0f ? 1u : 0u;
            }
        }
    }
    block_sum_store(acc, zeros, out + blockIdx.x);
}

// ---- pass 2 -------------------------------------------------------------------------

struct StateArrays {
    float *master;
    void *m, *v;
    float *ms, *vs;
};

template <int PD, int GD, int ST>
__global__ void __launch_bounds__(kBlock) k_list_apply(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                      int64_t t_end, int32_t first, StateArrays s,
                                                      const StepRec *__restrict__ rec, ListPtrs ptrs) {
    if (rec->skip) return;
    const float inv = rec->inv_scale;
    const int clip_on = rec->clip_on;
    const float clip = rec->clip;
    for (int64_t t = t_begin + blockIdx.x; t < t_end; t += gridDim.x) {
        const ListTile d = tiles[t];
        const Lane L = lane_of(d);
        const dopt_list_ptrs q = ptrs.p[d.index - first];
        const Hp h = load_hp(rec, d.packed >> 16);
        const Raw8 graw = load_raw_n<GD>(q.grad, L.e, L.n);
        float g[kVec], p[kVec], a[kVec], b[kVec];
        const Raw8 praw = PD == DOPT_F32 ? load_raw_n<DOPT_F32>(q.param, L.e, L.n)
                                         : load_raw_n<DOPT_F32>(s.master, L.arena, L.n);
        if constexpr (ST == DOPT_STATE_E4M3) {
            u32x2 cm{0, 0}, cv{0, 0};
            float sm = 0.0f, sv = 0.0f;
            if (L.n > 0) {  // a block's slots past the tensor's end are arena memory: whole 8-byte loads
                cm = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(s.m) + L.arena);
                cv = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(s.v) + L.arena);
                sm = s.ms[L.arena / kListBlock];
                sv = s.vs[L.arena / kListBlock];
            }
            decode8(cm, sm, a);
            decode8(cv, sv, b);
#pragma unroll
            for (int j = 0; j < kVec; ++j) b[j] = b[j] * b[j];
        } else {
            Elem<DOPT_F32>::unpack(load_raw_n<DOPT_F32>(s.m, L.arena, L.n), a);
            Elem<DOPT_F32>::unpack(load_raw_n<DOPT_F32>(s.v, L.arena, L.n), b);
        }
        Elem<GD>::unpack(graw, g);
        Elem<DOPT_F32>::unpack(praw, p);
        float r[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) r[j] = adamw_root(g[j], p[j], a[j], b[j], inv, clip_on, clip, h);
        if constexpr (ST == DOPT_STATE_E4M3) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {  // what is not of the tensor does not enter its block's maximum
                a[j] = j < L.n ? a[j] : 0.0f;
                r[j] = j < L.n ? r[j] : 0.0f;
            }
            float sm, sv;
            const u32x2 cm = encode8<false>(a, sm), cv = encode8<true>(r, sv);
            store_codes(s.m, L.arena, L.n, cm);
            store_codes(s.v, L.arena, L.n, cv);
            if (L.heads) {
                s.ms[L.arena / kListBlock] = sm;
                s.vs[L.arena / kListBlock] = sv;
            }
        } else {
            store_n<DOPT_F32>(s.m, L.arena, L.n, a);
            store_n<DOPT_F32>(s.v, L.arena, L.n, b);
        }
        if (PD != DOPT_F32) store_n<DOPT_F32>(s.master, L.arena, L.n, p);
        store_n<PD>(q.param, L.e, L.n, p);
    }
}

// ---- export, import, init -----------------------------------------------------------

struct ExportArrays {
    float *p, *m, *v;
};

template <int PD, int ST>
__global__ void __launch_bounds__(kBlock) k_list_export(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                       int64_t t_end, int32_t first,
                                                       const int64_t *__restrict__ xoff, StateArrays s,
                                                       ExportArrays x, ListPtrs ptrs) {
    for (int64_t t = t_begin + blockIdx.x; t < t_end; t += gridDim.x) {
        const ListTile d = tiles[t];
        const Lane L = lane_of(d);
        const int64_t o = xoff[d.index] + L.e;
        float p[kVec], a[kVec], b[kVec];
        Elem<DOPT_F32>::unpack(PD == DOPT_F32 ? load_raw_n<DOPT_F32>(ptrs.p[d.index - first].param, L.e, L.n)
                                              : load_raw_n<DOPT_F32>(s.master, L.arena, L.n), p);
        if constexpr (ST == DOPT_STATE_E4M3) {
            u32x2 cm{0, 0}, cv{0, 0};
            float sm = 0.0f, sv = 0.0f;
            if (L.n > 0) {
                cm = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(s.m) + L.arena);
                cv = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(s.v) + L.arena);
                sm = s.ms[L.arena / kListBlock];
                sv = s.vs[L.arena / kListBlock];
            }
            decode8(cm, sm, a);
            decode8(cv, sv, b);
#pragma unroll
            for (int j = 0; j < kVec; ++j) b[j] = b[j] * b[j];
        } else {
            Elem<DOPT_F32>::unpack(load_raw_n<DOPT_F32>(s.m, L.arena, L.n), a);
            Elem<DOPT_F32>::unpack(load_raw_n<DOPT_F32>(s.v, L.arena, L.n), b);
        }
        store_n<DOPT_F32>(x.p, o, L.n, p);
        store_n<DOPT_F32>(x.m, o, L.n, a);
        store_n<DOPT_F32>(x.v, o, L.n, b);
    }
}

template <int PD, int ST>
__global__ void __launch_bounds__(kBlock) k_list_import(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                       int64_t t_end, int32_t first,
                                                       const int64_t *__restrict__ xoff, StateArrays s,
                                                       ExportArrays x, ListPtrs ptrs) {
    for (int64_t t = t_begin + blockIdx.x; t < t_end; t += gridDim.x) {
        const ListTile d = tiles[t];
        const Lane L = lane_of(d);
        const int64_t o = xoff[d.index] + L.e;
        float p[kVec], a[kVec], b[kVec];
        Elem<DOPT_F32>::unpack(load_raw_n<DOPT_F32>(x.p, o, L.n), p);
        Elem<DOPT_F32>::unpack(load_raw_n<DOPT_F32>(x.m, o, L.n), a);
        Elem<DOPT_F32>::unpack(load_raw_n<DOPT_F32>(x.v, o, L.n), b);
        if (PD != DOPT_F32) store_n<DOPT_F32>(s.master, L.arena, L.n, p);
        store_n<PD>(ptrs.p[d.index - first].param, L.e, L.n, p);
        if constexpr (ST == DOPT_STATE_E4M3) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) b[j] = sqrtf(b[j]);
            float sm, sv;
            const u32x2 cm = encode8<false>(a, sm), cv = encode8<true>(b, sv);
            store_codes(s.m, L.arena, L.n, cm);
            store_codes(s.v, L.arena, L.n, cv);
            if (L.heads) {
                s.ms[L.arena / kListBlock] = sm;
                s.vs[L.arena / kListBlock] = sv;
            }
        } else {
            store_n<DOPT_F32>(s.m, L.arena, L.n, a);
            store_n<DOPT_F32>(s.v, L.arena, L.n, b);
        }
    }
}

// Masters from the params, everything else zero, whole blocks of the arena.
template <int PD, int ST>
__global__ void __launch_bounds__(kBlock) k_list_init(const ListTile *__restrict__ tiles, int64_t t_begin,
                                                     int64_t t_end, int32_t first, bool masters, StateArrays s,
                                                     ListPtrs ptrs) {
    const float z[kVec] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t t = t_begin + blockIdx.x; t < t_end; t += gridDim.x) {
        const ListTile d = tiles[t];
        const Lane L = lane_of(d);
        // the lane's slots lie in a block of the tensor
        const int whole = (static_cast<int>(d.packed & 0xffffu) + kListBlock - 1) / kListBlock * kListBlock;
        if (static_cast<int>(threadIdx.x) * kVec >= whole) continue;
        if (masters) {
            float p[kVec] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (PD != DOPT_F32) Elem<PD>::unpack(load_raw_n<PD>(ptrs.p[d.index - first].param, L.e, L.n), p);
            store8f(s.master, L.arena, p);
        }
        if constexpr (ST == DOPT_STATE_E4M3) {
            store_codes(s.m, L.arena, kVec, u32x2{0, 0});
            store_codes(s.v, L.arena, kVec, u32x2{0, 0});
            if (L.heads) {
                s.ms[L.arena / kListBlock] = 0.0f;
                s.vs[L.arena / kListBlock] = 0.0f;
            }
        } else {
            store8f(static_cast<float *>(s.m), L.arena, z);
            store8f(static_cast<float *>(s.v), L.arena, z);
        }
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
    const bool e = P->state_kind == DOPT_STATE_E4M3;
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

static const ListTile *tiles_of(const ListClass &C, const void *ws) {
    return reinterpret_cast<const ListTile *>(static_cast<const char *>(ws) + C.ws_tiles);
}

static ListPtrs slots(const ListClass &C, const ListRange &r, const dopt_list_ptrs *ts) {
    ListPtrs a;
    std::memset(&a, 0, sizeof a);
    for (int32_t i = 0; i < r.count; ++i) a.p[i] = ts[C.tensors[static_cast<size_t>(r.first + i)]];
    return a;
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
template <class F>
static void with_state(int kind, F f) {
    if (kind == DOPT_STATE_E4M3) f(Const<DOPT_STATE_E4M3>());
    else f(Const<DOPT_STATE_F32>());
}

template <bool FINALIZE>
static int launch_list_stats(const dopt_list *P, const dopt_list_ptrs *ts, void *ws, hipStream_t stream,
                             const FinalizeArgs &fa) {
    const DevState *st = reinterpret_cast<const DevState *>(ws_ptr(ws, kWsState));
    Partial *part = reinterpret_cast<Partial *>(ws_ptr(ws, kWsPartials));
    for (const ListClass &C : P->classes)
        for (const ListRange &r : C.stats) {
            GradPtrs a;
            std::memset(&a, 0, sizeof a);
            for (int32_t i = 0; i < r.count; ++i) a.p[i] = ts[C.tensors[static_cast<size_t>(r.first + i)]].grad;
            with_dtype(C.gd, [&](auto gd) {
                k_list_stats<decltype(gd)::value><<<r.grid, kBlock, 0, stream>>>(tiles_of(C, ws), r.t0, r.t1, r.first, st,
                                                                                 part + r.partial_base, a);
            });
            const int rc = check_launch("launch k_list_stats");
            if (rc) return rc;
        }
    return launch_finish<FINALIZE>(P->total_partials, ws, stream, fa);
}

template <bool IMPORT>
static int list_copy(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, ExportArrays x,
                     void *ws, hipStream_t stream) {
    StateArrays s;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, false, true)) || (rc = check_state(P, state, s))) return rc;
    if (P->numel > 0) {
        if (!x.p || !x.m || !x.v) return fail(DOPT_ERR_INVALID, "null export array");
        if ((reinterpret_cast<uintptr_t>(x.p) | reinterpret_cast<uintptr_t>(x.m) | reinterpret_cast<uintptr_t>(x.v)) % 4)
            return fail(DOPT_ERR_INVALID, "export array not 4-byte aligned");
    }
    for (const ListClass &C : P->classes)
        for (const ListRange &r : C.apply) {
            const ListPtrs a = slots(C, r, ts);
            const int64_t *xoff = reinterpret_cast<const int64_t *>(ws_ptr(ws, C.ws_xoff));
            with_dtype(C.pd, [&](auto pd) {
                with_state(P->state_kind, [&](auto st) {
                    constexpr int PD = decltype(pd)::value, ST = decltype(st)::value;
                    if (IMPORT)
                        k_list_import<PD, ST><<<r.grid, kBlock, 0, stream>>>(tiles_of(C, ws), r.t0, r.t1, r.first, xoff, s, x, a);
                    else
                        k_list_export<PD, ST><<<r.grid, kBlock, 0, stream>>>(tiles_of(C, ws), r.t0, r.t1, r.first, xoff, s, x, a);
                });
            });
            if ((rc = check_launch(IMPORT ? "launch k_list_import" : "launch k_list_export"))) return rc;
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
    for (const ListClass &C : P->classes) {
        rc = hip_check(hipMemcpyAsync(ws_ptr(ws, C.ws_tiles), C.tiles.data(), C.tiles.size() * sizeof(ListTile),
                                      hipMemcpyHostToDevice, stream),
                       "copy list tiles");
        if (rc) return rc;
        rc = hip_check(hipMemcpyAsync(ws_ptr(ws, C.ws_xoff), C.xoff.data(), C.xoff.size() * sizeof(int64_t),
                                      hipMemcpyHostToDevice, stream),
                       "copy list export offsets");
        if (rc) return rc;
        for (const ListRange &r : C.apply) {
            const ListPtrs a = slots(C, r, ts);
            with_dtype(C.pd, [&](auto pd) {
                with_state(P->state_kind, [&](auto st) {
                    k_list_init<decltype(pd)::value, decltype(st)::value><<<r.grid, kBlock, 0, stream>>>(
                        tiles_of(C, ws), r.t0, r.t1, r.first, P->has_master, s, a);
                });
            });
            if ((rc = check_launch("launch k_list_init"))) return rc;
        }
    }
    if ((rc = launch_init_records(*sc, ws, stream))) return rc;
    return hip_check(hipStreamSynchronize(stream), "synchronize after list init");
}

int dopt_list_stats(const dopt_list *P, const dopt_list_ptrs *ts, void *ws, hipStream_t stream) {
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, true, false))) return rc;
    FinalizeArgs none;
    std::memset(&none, 0, sizeof none);
    return launch_list_stats<false>(P, ts, ws, stream, none);
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
    return launch_list_stats<true>(P, ts, ws, stream, a);
}

int dopt_list_apply(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, void *ws,
                    hipStream_t stream) {
    StateArrays s;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, true, true)) || (rc = check_state(P, state, s))) return rc;
    const StepRec *rec = reinterpret_cast<const StepRec *>(ws_ptr(ws, kWsStepRec));
    for (const ListClass &C : P->classes)
        for (const ListRange &r : C.apply) {
            const ListPtrs a = slots(C, r, ts);
            with_dtype(C.pd, [&](auto pd) {
                with_dtype(C.gd, [&](auto gd) {
                    with_state(P->state_kind, [&](auto st) {
                        k_list_apply<decltype(pd)::value, decltype(gd)::value, decltype(st)::value>
                            <<<r.grid, kBlock, 0, stream>>>(tiles_of(C, ws), r.t0, r.t1, r.first, s, rec, a);
                    });
                });
            });
            if ((rc = check_launch("launch k_list_apply"))) return rc;
        }
    return DOPT_OK;
}

int dopt_list_step(const dopt_list *P, const dopt_list_ptrs *ts, const dopt_list_state *state, const dopt_hparams *hp,
                   int32_t n_hgroups, double max_grad_norm, void *ws, hipStream_t stream, dopt_stats *out) {
    // everything is checked before the first launch: a refused call leaves the scaler and step count alone
    StateArrays s;
    int rc = check_list(P, ws);
    if (rc || (rc = check_tensors(P, ts, true, true)) || (rc = check_state(P, state, s))) return rc;
    if ((rc = dopt_list_prepare(P, ts, hp, n_hgroups, max_grad_norm, ws, stream))) return rc;
    if ((rc = dopt_list_apply(P, ts, state, ws, stream))) return rc;
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
