// Device side shared by the flat-buffer step (step.hip) and the tensor-list
// step (list.hip): the records in the workspace, element I/O, the update
// formula, the fixed-order reduction with the step's finalize, and the host
// routines around them.
//
// Pages cited: [DO] "Megatron-LM distrib_optimizer.py 源码精读";
// [DS] "Megatron-LM与DeepSpeed的分布式训练源码里，模型和优化器到底是怎么切分的？".
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"

namespace dopt {

// ---- device records in the workspace -------------------------------------

struct DevState {  // persists across steps
    double scale, growth_factor, backoff_factor, min_scale;
    int64_t t;  // successful steps
    int64_t growth_tracker, hysteresis_tracker, growth_interval;
    float inv_scale;  // fp32(1 / scale): the unscale factor of the coming step
    int32_t kind, hysteresis, pad;
};
static_assert(sizeof(DevState) <= kWsStepRec - kWsState, "state record too large");

struct StepRec {  // scalars of the apply pass of the current step
    int32_t skip, clip_on;
    float inv_scale, clip;
    float decay[DOPT_MAX_HGROUPS], beta1[DOPT_MAX_HGROUPS], omb1[DOPT_MAX_HGROUPS];
    float beta2[DOPT_MAX_HGROUPS], omb2[DOPT_MAX_HGROUPS], eps[DOPT_MAX_HGROUPS];
    float step_size[DOPT_MAX_HGROUPS], sqrt_bc2[DOPT_MAX_HGROUPS];
};
static_assert(sizeof(StepRec) <= kWsStats - kWsStepRec, "step record too large");
static_assert(sizeof(dopt_stats) <= kWsRecord - kWsStats, "stats record too large");

struct Partial {
    double sumsq;
    unsigned long long zeros;
};
static_assert(sizeof(Partial) == 16, "partial record size");

struct Record {
    double sumsq, zeros;
};

struct FinalizeArgs {
    dopt_hparams hp[DOPT_MAX_HGROUPS];
    int32_t nh, pad;
    double max_norm;
};

struct InitArgs {
    DevState st;
};

// ---- element I/O -----------------------------------------------------------

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 16-byte load; NT marks the line as streamed (read once), which lets the
// memory system keep it out of the caches.
template <bool NT>
__device__ __forceinline__ u32x4 ld16(const void *p) {
    if (NT) return __builtin_nontemporal_load(static_cast<const u32x4 *>(p));
    return *static_cast<const u32x4 *>(p);
}

// Tile-local buffer access (pass 2).  A resource descriptor covers one
// 2048-element tile of one stream: the tile base is wave-uniform and sits in
// scalar registers, so every stream of a tile shares one per-lane byte offset
// instead of holding a 64-bit address per lane.  The descriptor is raw
// (stride 0, range in bytes) with the 32-bit data format that untyped dword
// accesses take on this ISA; an access past the range would read zero and
// write nothing, and none is made.
constexpr int32_t kRsrcWord3 = 0x00020000;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const void *tile_base, int32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(tile_base), 0, bytes, kRsrcWord3);
}
__device__ __forceinline__ u32x4 bld16(__amdgpu_buffer_rsrc_t r, int32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
}
__device__ __forceinline__ void bst16(__amdgpu_buffer_rsrc_t r, int32_t off, u32x4 x) {
    __builtin_amdgcn_raw_buffer_store_b128(x, r, off, 0, 0);
}
__device__ __forceinline__ float bld4(__amdgpu_buffer_rsrc_t r, int32_t off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
__device__ __forceinline__ void bst4(__amdgpu_buffer_rsrc_t r, int32_t off, float x) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, off, 0, 0);
}

template <int DT>
struct Elem;

// The raw bytes of 8 consecutive elements (16-bit types use `lo` only).
// Kernels load raw packets first and convert after a scheduling barrier, so
// that all of a batch's loads are in flight before the first one is waited
// for.
struct Raw8 {
    u32x4 lo, hi;
};

template <>
struct Elem<DOPT_BF16> {
    static constexpr int64_t kBytes = 2;
    template <bool NT = false>
    static __device__ __forceinline__ Raw8 load_raw(const void *base, int64_t i) {
        return Raw8{ld16<NT>(static_cast<const uint16_t *>(base) + i), u32x4{0, 0, 0, 0}};
    }
    static __device__ __forceinline__ void unpack(const Raw8 &r, float (&x)[kVec]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(r.lo[j] << 16);
            x[2 * j + 1] = __uint_as_float(r.lo[j] & 0xffff0000u);
        }
    }
    template <bool NT = false>
    static __device__ __forceinline__ void load8(const void *base, int64_t i, float (&x)[kVec]) {
        unpack(load_raw<NT>(base, i), x);
    }
    static __device__ __forceinline__ uint32_t bits(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    }
    static __device__ __forceinline__ void store8(void *base, int64_t i, const float (&x)[kVec]) {
        u32x4 u;
        u[0] = bits(x[0]) | (bits(x[1]) << 16);
        u[1] = bits(x[2]) | (bits(x[3]) << 16);
        u[2] = bits(x[4]) | (bits(x[5]) << 16);
        u[3] = bits(x[6]) | (bits(x[7]) << 16);
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(base) + i) = u;
    }
    static __device__ __forceinline__ void store1(void *base, int64_t i, float x) {
        static_cast<uint16_t *>(base)[i] = static_cast<uint16_t>(bits(x));
    }
    // lane's 8 elements of a tile through its resource descriptor
    static __device__ __forceinline__ void bload8(__amdgpu_buffer_rsrc_t r, int32_t lane, float (&x)[kVec]) {
        unpack(Raw8{bld16(r, lane * 16), u32x4{0, 0, 0, 0}}, x);
    }
    static __device__ __forceinline__ float bload1(__amdgpu_buffer_rsrc_t r, int32_t lane, int j) {
        return __uint_as_float(uint32_t(__builtin_amdgcn_raw_buffer_load_b16(r, lane * 16 + j * 2, 0, 0)) << 16);
    }
    static __device__ __forceinline__ void bstore1(__amdgpu_buffer_rsrc_t r, int32_t lane, int j, float x) {
        __builtin_amdgcn_raw_buffer_store_b16(static_cast<unsigned short>(bits(x)), r, lane * 16 + j * 2, 0, 0);
    }
    static __device__ __forceinline__ void bstore8(__amdgpu_buffer_rsrc_t r, int32_t lane, const float (&x)[kVec]) {
        u32x4 u;
        u[0] = bits(x[0]) | (bits(x[1]) << 16);
        u[1] = bits(x[2]) | (bits(x[3]) << 16);
        u[2] = bits(x[4]) | (bits(x[5]) << 16);
        u[3] = bits(x[6]) | (bits(x[7]) << 16);
        bst16(r, lane * 16, u);
    }
};

template <>
struct Elem<DOPT_F16> {
    static constexpr int64_t kBytes = 2;
    static __device__ __forceinline__ float up(uint32_t h) {
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
    }
    template <bool NT = false>
    static __device__ __forceinline__ Raw8 load_raw(const void *base, int64_t i) {
        return Raw8{ld16<NT>(static_cast<const uint16_t *>(base) + i), u32x4{0, 0, 0, 0}};
    }
    static __device__ __forceinline__ void unpack(const Raw8 &r, float (&x)[kVec]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = up(r.lo[j] & 0xffffu);
            x[2 * j + 1] = up(r.lo[j] >> 16);
        }
    }
    template <bool NT = false>
    static __device__ __forceinline__ void load8(const void *base, int64_t i, float (&x)[kVec]) {
        unpack(load_raw<NT>(base, i), x);
    }
    static __device__ __forceinline__ uint32_t bits(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
    }
    static __device__ __forceinline__ void store8(void *base, int64_t i, const float (&x)[kVec]) {
        u32x4 u;
        u[0] = bits(x[0]) | (bits(x[1]) << 16);
        u[1] = bits(x[2]) | (bits(x[3]) << 16);
        u[2] = bits(x[4]) | (bits(x[5]) << 16);
        u[3] = bits(x[6]) | (bits(x[7]) << 16);
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(base) + i) = u;
    }
    static __device__ __forceinline__ void store1(void *base, int64_t i, float x) {
        static_cast<uint16_t *>(base)[i] = static_cast<uint16_t>(bits(x));
    }
    // lane's 8 elements of a tile through its resource descriptor
    static __device__ __forceinline__ void bload8(__amdgpu_buffer_rsrc_t r, int32_t lane, float (&x)[kVec]) {
        unpack(Raw8{bld16(r, lane * 16), u32x4{0, 0, 0, 0}}, x);
    }
    static __device__ __forceinline__ float bload1(__amdgpu_buffer_rsrc_t r, int32_t lane, int j) {
        return up(__builtin_amdgcn_raw_buffer_load_b16(r, lane * 16 + j * 2, 0, 0));
    }
    static __device__ __forceinline__ void bstore1(__amdgpu_buffer_rsrc_t r, int32_t lane, int j, float x) {
        __builtin_amdgcn_raw_buffer_store_b16(static_cast<unsigned short>(bits(x)), r, lane * 16 + j * 2, 0, 0);
    }
    static __device__ __forceinline__ void bstore8(__amdgpu_buffer_rsrc_t r, int32_t lane, const float (&x)[kVec]) {
        u32x4 u;
        u[0] = bits(x[0]) | (bits(x[1]) << 16);
        u[1] = bits(x[2]) | (bits(x[3]) << 16);
        u[2] = bits(x[4]) | (bits(x[5]) << 16);
        u[3] = bits(x[6]) | (bits(x[7]) << 16);
        bst16(r, lane * 16, u);
    }
};

template <bool NT = false>
__device__ __forceinline__ void load8f(const float *base, int64_t i, float (&x)[kVec]) {
    const u32x4 a = ld16<NT>(base + i);
    const u32x4 b = ld16<NT>(base + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = __uint_as_float(a[j]);
        x[4 + j] = __uint_as_float(b[j]);
    }
}

__device__ __forceinline__ void store8f(float *base, int64_t i, const float (&x)[kVec]) {
    *reinterpret_cast<f32x4 *>(base + i) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4 *>(base + i + 4) = f32x4{x[4], x[5], x[6], x[7]};
}

// Elem<GD>::store8 with the nontemporal hint (16-byte stores), called by all
// 64 lanes of a wave together, lane l holding elements i .. i+7 with
// i = (the wave's first element) + 8l.  For fp32 each store instruction
// covers one contiguous KiB: lane l writes elements 4l .. 4l+3 and
// 256+4l .. 256+4l+3 of the wave's 512, taken from the lanes that hold them
// (l>>1 and 32 + (l>>1)).  Two stores of a lane's own halves would leave
// every other 16 bytes of each instruction's lines unwritten, and streaming
// stores of such partial lines raised the reduce's write traffic by 11%.
template <int GD>
__device__ __forceinline__ void store8_nt(void *base, int64_t i, const float (&x)[kVec]) {
    if constexpr (GD == DOPT_F32) {
        const int l = static_cast<int>(threadIdx.x & 63);
        const int s0 = l >> 1, s1 = 32 + (l >> 1);
        const bool odd = (l & 1) != 0;
        f32x4 a, c;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float lo0 = __shfl(x[q], s0, 64), hi0 = __shfl(x[4 + q], s0, 64);
            const float lo1 = __shfl(x[q], s1, 64), hi1 = __shfl(x[4 + q], s1, 64);
            a[q] = odd ? hi0 : lo0;
            c[q] = odd ? hi1 : lo1;
        }
        float *w = static_cast<float *>(base) + (i - int64_t(l) * kVec);
        __builtin_nontemporal_store(a, reinterpret_cast<f32x4 *>(w + 4 * l));
        __builtin_nontemporal_store(c, reinterpret_cast<f32x4 *>(w + 256 + 4 * l));
    } else {
        u32x4 u;
        u[0] = Elem<GD>::bits(x[0]) | (Elem<GD>::bits(x[1]) << 16);
        u[1] = Elem<GD>::bits(x[2]) | (Elem<GD>::bits(x[3]) << 16);
        u[2] = Elem<GD>::bits(x[4]) | (Elem<GD>::bits(x[5]) << 16);
        u[3] = Elem<GD>::bits(x[6]) | (Elem<GD>::bits(x[7]) << 16);
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(base) + i));
    }
}

__device__ __forceinline__ void bload8f(__amdgpu_buffer_rsrc_t r, int32_t lane, float (&x)[kVec]) {
    const u32x4 a = bld16(r, lane * 32);
    const u32x4 b = bld16(r, lane * 32 + 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = __uint_as_float(a[j]);
        x[4 + j] = __uint_as_float(b[j]);
    }
}

__device__ __forceinline__ void bstore8f(__amdgpu_buffer_rsrc_t r, int32_t lane, const float (&x)[kVec]) {
    bst16(r, lane * 32, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])});
    bst16(r, lane * 32 + 16,
          u32x4{__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])});
}

template <>
struct Elem<DOPT_F32> {
    static constexpr int64_t kBytes = 4;
    static __device__ __forceinline__ void bload8(__amdgpu_buffer_rsrc_t r, int32_t lane, float (&x)[kVec]) {
        bload8f(r, lane, x);
    }
    static __device__ __forceinline__ void bstore8(__amdgpu_buffer_rsrc_t r, int32_t lane, const float (&x)[kVec]) {
        bstore8f(r, lane, x);
    }
    static __device__ __forceinline__ float bload1(__amdgpu_buffer_rsrc_t r, int32_t lane, int j) {
        return bld4(r, lane * 32 + j * 4);
    }
    static __device__ __forceinline__ void bstore1(__amdgpu_buffer_rsrc_t r, int32_t lane, int j, float x) {
        bst4(r, lane * 32 + j * 4, x);
    }
    template <bool NT = false>
    static __device__ __forceinline__ Raw8 load_raw(const void *base, int64_t i) {
        const float *f = static_cast<const float *>(base) + i;
        return Raw8{ld16<NT>(f), ld16<NT>(f + 4)};
    }
    static __device__ __forceinline__ void unpack(const Raw8 &r, float (&x)[kVec]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = __uint_as_float(r.lo[j]);
            x[4 + j] = __uint_as_float(r.hi[j]);
        }
    }
    template <bool NT = false>
    static __device__ __forceinline__ void load8(const void *base, int64_t i, float (&x)[kVec]) {
        load8f<NT>(static_cast<const float *>(base), i, x);
    }
    static __device__ __forceinline__ void store8(void *base, int64_t i, const float (&x)[kVec]) {
        store8f(static_cast<float *>(base), i, x);
    }
    static __device__ __forceinline__ void store1(void *base, int64_t i, float x) { static_cast<float *>(base)[i] = x; }
};

// An optimizer param group's scalars of one step.
struct Hp {
    float decay, b1, omb1, b2, omb2, eps, step, sbc2;
};

// ---- finalize: skip, norm, clip, loss scale, step count, AdamW scalars ------
//
// [DO] "三层继承体系": an overflow skips the inner step; clipping uses the
// global norm.  [DS] §3 config: dynamic loss scale starting at 2^16.  Clip
// coefficient max_norm / (norm + 1e-6), applied when below 1; the dynamic
// scale backs off (after `hysteresis` overflows) and grows every
// growth_interval clean steps; AdamW scalars are computed in double and
// rounded once to fp32.  `cur` is the caller's copy of *st, read at kernel
// start so that its load overlaps the reduction; the new state is written to
// *st.

// The decision, by one thread; returns the step count after it.
static __device__ __forceinline__ int64_t decide_step(double sumsq, double zeros, const DevState &cur, DevState *st,
                                                      StepRec *sr, dopt_stats *out, double max_norm) {
    DevState n = cur;
    const int found_inf = isfinite(sumsq) ? 0 : 1;
    const double norm = sqrt(sumsq);
    out->found_inf = found_inf;
    out->skipped = found_inf;
    out->reserved = 0;
    out->sumsq = sumsq;
    out->grad_norm = norm;
    out->num_zeros = static_cast<uint64_t>(zeros);
    out->loss_scale_used = n.scale;
    sr->skip = found_inf;
    sr->inv_scale = n.inv_scale;
    if (n.kind == DOPT_SCALER_DYNAMIC) {
        if (found_inf) {
            n.growth_tracker = 0;
            n.hysteresis_tracker -= 1;
            if (n.hysteresis_tracker <= 0) n.scale = fmax(n.scale * n.backoff_factor, n.min_scale);
        } else {
            n.growth_tracker += 1;
            if (n.growth_tracker == n.growth_interval) {
                n.growth_tracker = 0;
                n.hysteresis_tracker = n.hysteresis;
                n.scale = n.scale * n.growth_factor;
            }
        }
        n.inv_scale = static_cast<float>(1.0 / n.scale);
    }
    out->loss_scale_next = n.scale;
    double clip = 1.0;
    int clip_on = 0;
    if (!found_inf) {
        n.t += 1;
        if (max_norm > 0.0) {
            clip = max_norm / (norm + 1e-6);
            clip_on = clip < 1.0 ? 1 : 0;
        }
    }
    out->clip_coef = clip;
    out->clip_applied = clip_on;
    sr->clip_on = clip_on;
    sr->clip = clip_on ? static_cast<float>(clip) : 0.0f;
    out->step_count = n.t;
    *st = n;
    return n.t;
}

// One hyper-group's scalars for step t.
static __device__ __forceinline__ Hp step_scalars(const dopt_hparams &hp, double t) {
    return Hp{static_cast<float>(1.0 - hp.lr * hp.weight_decay), static_cast<float>(hp.beta1),
              static_cast<float>(1.0 - hp.beta1), static_cast<float>(hp.beta2), static_cast<float>(1.0 - hp.beta2),
              static_cast<float>(hp.eps), static_cast<float>(hp.lr / (1.0 - pow(hp.beta1, t))),
              static_cast<float>(sqrt(1.0 - pow(hp.beta2, t)))};
}

static __device__ __forceinline__ void store_scalars(StepRec *sr, int h, const Hp &x) {
    sr->decay[h] = x.decay;
    sr->beta1[h] = x.b1;
    sr->omb1[h] = x.omb1;
    sr->beta2[h] = x.b2;
    sr->omb2[h] = x.omb2;
    sr->eps[h] = x.eps;
    sr->step_size[h] = x.step;
    sr->sqrt_bc2[h] = x.sbc2;
}

// Called by every thread of one workgroup: thread 0 takes the step decision,
// then thread h fills the scalars of hyper-group h.
static __device__ void finalize_block(double sumsq, double zeros, const DevState &cur, DevState *st, StepRec *sr,
                                      dopt_stats *out, const FinalizeArgs &a) {
    __shared__ double s_t;
    __shared__ int s_skip;
    if (threadIdx.x == 0) {
        s_t = static_cast<double>(decide_step(sumsq, zeros, cur, st, sr, out, a.max_norm));
        s_skip = isfinite(sumsq) ? 0 : 1;
    }
    __syncthreads();
    const int h = threadIdx.x;
    if (!s_skip && h < a.nh) store_scalars(sr, h, step_scalars(a.hp[h], s_t));
}

static __global__ void __launch_bounds__(64) k_finalize(const Record *rec, DevState *st, StepRec *sr, dopt_stats *out,
                                                        FinalizeArgs a) {
    const DevState cur = *st;
    finalize_block(rec->sumsq, rec->zeros, cur, st, sr, out, a);
}

// ---- partial sums -------------------------------------------------------------

__device__ __forceinline__ void block_sum_store(double acc, unsigned long long z, Partial *__restrict__ dst) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        acc += __shfl_xor(acc, off, 64);
        z += __shfl_xor(z, off, 64);
    }
    __shared__ double s_acc[kBlock / 64];
    __shared__ unsigned long long s_z[kBlock / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) {
        s_acc[wave] = acc;
        s_z[wave] = z;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double a = 0.0;
        unsigned long long zz = 0;
#pragma unroll
        for (int w = 0; w < kBlock / 64; ++w) {
            a += s_acc[w];
            zz += s_z[w];
        }
        dst->sumsq = a;
        dst->zeros = zz;
    }
}

// One workgroup of THREADS: the fixed-order sum of all partials into the
// record, and in the fused form the finalize of the step.  Thread i adds
// partials i, i+THREADS, ... in order (loads issued together, BATCH at a
// time), each wave folds its 64 lanes with a fixed butterfly, and thread 0
// adds the wave sums in order.  Up to kFinishSmall partials (small windows)
// take 256 threads x 8 loads; more (large windows, up to kStatsMaxBlocks per
// buffer) take 1024 threads x 16 loads, one round for 16384 partials.
constexpr int kFinishSmall = 2048;
constexpr int kFinishBatch = 8;  // loads in flight per thread in k_check_finish

template <bool FINALIZE, int THREADS, int BATCH>
static __global__ void __launch_bounds__(THREADS) k_finish(const Partial *__restrict__ part, int32_t n,
                                                          Record *__restrict__ rec, DevState *__restrict__ st,
                                                          StepRec *__restrict__ sr, dopt_stats *__restrict__ out,
                                                          FinalizeArgs fa) {
    const DevState cur = *st;  // loaded now, used after the reduction
    double a = 0.0;
    unsigned long long z = 0;
    for (int32_t i0 = threadIdx.x; i0 < n; i0 += BATCH * THREADS) {
        Partial q[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int32_t i = i0 + j * THREADS;
            q[j] = part[i < n ? i : n - 1];
        }
        __builtin_amdgcn_sched_barrier(0);  // all loads in flight before the first add
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const bool in = i0 + j * THREADS < n;  // a clamped duplicate adds +0
            a += in ? q[j].sumsq : 0.0;
            z += in ? q[j].zeros : 0ull;
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        a += __shfl_xor(a, off, 64);
        z += __shfl_xor(z, off, 64);
    }
    __shared__ double s_acc[THREADS / 64];
    __shared__ unsigned long long s_z[THREADS / 64];
    __shared__ double s_tot[2];
    if ((threadIdx.x & 63) == 0) {
        s_acc[threadIdx.x >> 6] = a;
        s_z[threadIdx.x >> 6] = z;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        unsigned long long tz = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            t += s_acc[w];
            tz += s_z[w];
        }
        rec->sumsq = t;
        rec->zeros = static_cast<double>(tz);
        s_tot[0] = t;
        s_tot[1] = static_cast<double>(tz);
    }
    if (FINALIZE) {
        __syncthreads();
        finalize_block(s_tot[0], s_tot[1], cur, st, sr, out, fa);
    }
}

// ---- the update formula (fp32, in the order stated at pass 2) -------------------

__device__ __forceinline__ Hp load_hp(const StepRec *__restrict__ r, int h) {
    return Hp{r->decay[h], r->beta1[h], r->omb1[h], r->beta2[h], r->omb2[h], r->eps[h], r->step_size[h], r->sqrt_bc2[h]};
}

// Returns sqrt(v) of the new v.
__device__ __forceinline__ float adamw_root(float raw, float &p, float &m, float &v, float inv, int clip_on, float clip,
                                            const Hp &h) {
    float g = raw * inv;
    if (clip_on) g = g * clip;
    p = p * h.decay;
    m = h.b1 * m + h.omb1 * g;
    v = h.b2 * v + h.omb2 * (g * g);
    const float r = sqrtf(v);
    const float d = r / h.sbc2 + h.eps;
    p = p - h.step * (m / d);
    return r;
}

__device__ __forceinline__ void adamw(float raw, float &p, float &m, float &v, float inv, int clip_on, float clip,
                                      const Hp &h) {
    adamw_root(raw, p, m, v, inv, clip_on, clip, h);
}

// ---- records at init ------------------------------------------------------------

static __global__ void k_init_state(DevState *st, StepRec *sr, dopt_stats *stats, Record *rec, InitArgs a) {
    if (threadIdx.x != 0) return;
    *st = a.st;
    StepRec r;
    memset(&r, 0, sizeof r);
    r.skip = 1;
    *sr = r;
    dopt_stats o;
    memset(&o, 0, sizeof o);
    o.loss_scale_next = a.st.scale;
    *stats = o;
    rec->sumsq = 0.0;
    rec->zeros = 0.0;
}

// ---- host side --------------------------------------------------------------

inline int hip_check(hipError_t e, const char *what) {
    if (e == hipSuccess) return DOPT_OK;
    return fail(DOPT_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

inline int check_launch(const char *what) { return hip_check(hipGetLastError(), what); }

inline bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) % DOPT_PTR_ALIGN) == 0; }

inline char *ws_ptr(void *ws, int64_t off) { return static_cast<char *>(ws) + off; }

inline int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// max_hgroup: the largest hyper-group in use.
inline int build_finalize_args(int32_t max_hgroup, const dopt_hparams *hp, int32_t n_hgroups, double max_grad_norm,
                               FinalizeArgs &a) {
    if (!hp) return fail(DOPT_ERR_INVALID, "null hparams");
    if (n_hgroups < max_hgroup + 1 || n_hgroups > DOPT_MAX_HGROUPS)
        return fail(DOPT_ERR_INVALID, "n_hgroups must cover every hgroup of the params (<= DOPT_MAX_HGROUPS)");
    std::memset(&a, 0, sizeof a);
    for (int32_t h = 0; h < n_hgroups; ++h) {
        const dopt_hparams &x = hp[h];
        if (!(x.lr >= 0.0) || !(x.beta1 >= 0.0 && x.beta1 < 1.0) || !(x.beta2 >= 0.0 && x.beta2 < 1.0) ||
            !(x.eps > 0.0) || !(x.weight_decay >= 0.0))
            return fail(DOPT_ERR_INVALID,
                        "hparams " + std::to_string(h) + ": need lr >= 0, 0 <= betas < 1, eps > 0, wd >= 0");
        a.hp[h] = x;
    }
    a.nh = n_hgroups;
    a.max_norm = max_grad_norm;
    return DOPT_OK;
}

// The fixed-order reduction of all pass-1 partials, and the finalize when
// FINALIZE is set.
template <bool FINALIZE>
static int launch_finish(int32_t n_partials, void *ws, hipStream_t stream, const FinalizeArgs &fa) {
    const Partial *part = reinterpret_cast<const Partial *>(ws_ptr(ws, kWsPartials));
    Record *rec = reinterpret_cast<Record *>(ws_ptr(ws, kWsRecord));
    DevState *st = reinterpret_cast<DevState *>(ws_ptr(ws, kWsState));
    StepRec *sr = reinterpret_cast<StepRec *>(ws_ptr(ws, kWsStepRec));
    dopt_stats *out = reinterpret_cast<dopt_stats *>(ws_ptr(ws, kWsStats));
    if (n_partials <= kFinishSmall)
        k_finish<FINALIZE, 256, 8><<<1, 256, 0, stream>>>(part, n_partials, rec, st, sr, out, fa);
    else
        k_finish<FINALIZE, 1024, 16><<<1, 1024, 0, stream>>>(part, n_partials, rec, st, sr, out, fa);
    return check_launch("launch k_finish");
}

// A loss scale the step can run with: positive and finite, with a
// reciprocal (the factor every grad is unscaled by, kept in fp32) that is a
// finite nonzero fp32 number.
inline bool usable_scale(double s) {
    if (!(s > 0.0) || !std::isfinite(s)) return false;
    const float inv = static_cast<float>(1.0 / s);
    return inv > 0.0f && std::isfinite(inv);
}

inline int check_scaler(const dopt_scaler_cfg *sc) {
    if (!sc) return fail(DOPT_ERR_INVALID, "null scaler config");
    if (!usable_scale(sc->initial_scale) || (sc->kind != DOPT_SCALER_CONSTANT && sc->kind != DOPT_SCALER_DYNAMIC))
        return fail(DOPT_ERR_INVALID, "scaler: kind must be constant or dynamic, and initial_scale finite and > 0 "
                                      "with a finite nonzero fp32 reciprocal");
    if (sc->kind == DOPT_SCALER_DYNAMIC &&
        (sc->hysteresis < 1 || sc->growth_interval < 1 || !(sc->growth_factor > 1.0) || !std::isfinite(sc->growth_factor) ||
         !(sc->backoff_factor > 0.0) || !(sc->backoff_factor < 1.0) || !usable_scale(sc->min_scale)))
        return fail(DOPT_ERR_INVALID, "dynamic scaler: bad hysteresis, interval or factors");
    return DOPT_OK;
}

// The persistent state and the step records at step 0.
inline int launch_init_records(const dopt_scaler_cfg &sc, void *ws, hipStream_t stream) {
    InitArgs a;
    std::memset(&a, 0, sizeof a);
    a.st.scale = sc.initial_scale;
    a.st.growth_factor = sc.growth_factor;
    a.st.backoff_factor = sc.backoff_factor;
    a.st.min_scale = sc.min_scale;
    a.st.t = 0;
    a.st.growth_tracker = 0;
    a.st.hysteresis_tracker = sc.hysteresis;
    a.st.growth_interval = sc.growth_interval;
    a.st.inv_scale = static_cast<float>(1.0 / sc.initial_scale);
    a.st.kind = sc.kind;
    a.st.hysteresis = sc.hysteresis;
    k_init_state<<<1, 64, 0, stream>>>(reinterpret_cast<DevState *>(ws_ptr(ws, kWsState)),
                                       reinterpret_cast<StepRec *>(ws_ptr(ws, kWsStepRec)),
                                       reinterpret_cast<dopt_stats *>(ws_ptr(ws, kWsStats)),
                                       reinterpret_cast<Record *>(ws_ptr(ws, kWsRecord)), a);
    return check_launch("launch k_init_state");
}

inline int launch_finalize(const FinalizeArgs &a, void *ws, hipStream_t stream) {
    k_finalize<<<1, 64, 0, stream>>>(reinterpret_cast<const Record *>(ws_ptr(ws, kWsRecord)),
                                     reinterpret_cast<DevState *>(ws_ptr(ws, kWsState)),
                                     reinterpret_cast<StepRec *>(ws_ptr(ws, kWsStepRec)),
                                     reinterpret_cast<dopt_stats *>(ws_ptr(ws, kWsStats)), a);
    return check_launch("launch k_finalize");
}

// Synchronizing reads and writes of the records (dopt_state_scalars_get / _set,
// dopt_read_stats and their list counterparts).
inline int read_scalars(const void *ws, hipStream_t stream, dopt_state_scalars *out) {
    DevState st;
    int rc = hip_check(hipMemcpyAsync(&st, static_cast<const char *>(ws) + kWsState, sizeof st,
                                      hipMemcpyDeviceToHost, stream),
                       "copy scalar state");
    if (rc) return rc;
    if ((rc = hip_check(hipStreamSynchronize(stream), "synchronize for scalar state"))) return rc;
    out->step_count = st.t;
    out->loss_scale = st.scale;
    out->growth_tracker = st.growth_tracker;
    out->hysteresis_tracker = st.hysteresis_tracker;
    return DOPT_OK;
}

inline int write_scalars(void *ws, hipStream_t stream, const dopt_state_scalars *in) {
    if (!usable_scale(in->loss_scale) || in->step_count < 0)
        return fail(DOPT_ERR_INVALID, "scalar state: loss_scale must be finite and > 0 with a finite nonzero fp32 "
                                      "reciprocal, and step_count >= 0");
    DevState st;
    int rc = hip_check(hipMemcpyAsync(&st, ws_ptr(ws, kWsState), sizeof st, hipMemcpyDeviceToHost, stream),
                       "copy scalar state");
    if (rc) return rc;
    if ((rc = hip_check(hipStreamSynchronize(stream), "synchronize for scalar state"))) return rc;
    st.t = in->step_count;
    st.scale = in->loss_scale;
    st.inv_scale = static_cast<float>(1.0 / in->loss_scale);
    st.growth_tracker = in->growth_tracker;
    st.hysteresis_tracker = in->hysteresis_tracker;
    if ((rc = hip_check(hipMemcpyAsync(ws_ptr(ws, kWsState), &st, sizeof st, hipMemcpyHostToDevice, stream),
                        "write scalar state")))
        return rc;
    return hip_check(hipStreamSynchronize(stream), "synchronize after scalar state");
}

inline int copy_stats(const void *ws, hipStream_t stream, dopt_stats *out) {
    int rc = hip_check(hipMemcpyAsync(out, static_cast<const char *>(ws) + kWsStats, sizeof(dopt_stats),
                                      hipMemcpyDeviceToHost, stream),
                       "copy stats");
    if (rc) return rc;
    return hip_check(hipStreamSynchronize(stream), "synchronize for stats");
}

}  // namespace dopt
