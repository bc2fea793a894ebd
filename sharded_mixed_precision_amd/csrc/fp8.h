// Shared by the 8-bit operators (fp8.hip, norm.hip, gemm.hip): the checks of
// their arguments, element I/O at any alignment, and the block-scaled e4m3 format.
#pragma once

#include <hip/hip_runtime.h>

#include <cstring>

#include "dopt_fp8.h"
#include "internal.h"

namespace dopt {

// ---- host: checks of arguments ---------------------------------------------------

// What an argument covers: from lo to before hi, and of that `width` bytes in
// each `pitch`, so that columns side by side in one matrix do not overlap.
struct Span {
    const char *name;
    uintptr_t lo, hi;
    int64_t pitch, width;
};

inline Span span_of(const char *name, const void *p, int64_t bytes, int64_t pitch = 0, int64_t width = 0) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{name, a, p ? a + static_cast<uint64_t>(bytes > 0 ? bytes : 0) : a, pitch, width};
}

inline int element_bytes(int32_t dtype) { return dtype == DOPT_F32 ? 4 : 2; }

inline bool is_dtype(int32_t t) { return t == DOPT_F32 || t == DOPT_BF16 || t == DOPT_F16; }

int check_dense(const char *name, const dopt_dense *x);
int check_fp8(const char *name, const dopt_fp8_matrix *x);
int check_vector(const char *name, const void *p, int64_t n, int32_t dtype);
Span dense_span(const char *name, const dopt_dense *x);
Span codes_span(const char *name, const dopt_fp8_matrix *x);
Span scales_span(const char *name, const dopt_fp8_matrix *x);
// Refuses an output that overlaps an input or another output (n_out spans, then the inputs).
int check_apart(const Span *out, int n_out, const Span *in, int n_in);
int launched(const char *what);

// A launch has less than this many threads along a dimension of its grid.
constexpr int64_t kMaxThreads = int64_t(1) << 32;

// ---- device: elements -------------------------------------------------------------

using i32x4 = __attribute__((ext_vector_type(4))) int;
using i32x8 = __attribute__((ext_vector_type(8))) int;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x2 = __attribute__((ext_vector_type(2))) uint32_t;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;

// 16 bytes at any address that is a multiple of 2: global accesses need no
// alignment here, so odd strides take the same wide loads.
struct __attribute__((packed, aligned(2))) Bytes16 {
    u32x4 v;
};
struct __attribute__((packed, aligned(2))) Bytes8 {
    u32x2 v;
};

struct __attribute__((packed, aligned(4))) Float4 {
    f32x4 v;
};

// Number of 16-byte words that 8 elements take.
template <int T>
constexpr int kWords8 = T == DOPT_F32 ? 2 : 1;

// 8 consecutive elements as they lie in memory.
template <int T>
struct Raw8 {
    u32x4 w[kWords8<T>];
};

template <int T>
__device__ __forceinline__ float to_float(uint32_t bits) {
    if constexpr (T == DOPT_F32) return __uint_as_float(bits);
    if constexpr (T == DOPT_BF16) return __uint_as_float(bits << 16);
    if constexpr (T == DOPT_F16) {
        const uint16_t h = static_cast<uint16_t>(bits);
        return static_cast<float>(__builtin_bit_cast(_Float16, h));
    }
}

template <int T>
__device__ __forceinline__ uint32_t from_float(float x) {
    if constexpr (T == DOPT_F32) return __float_as_uint(x);
    if constexpr (T == DOPT_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    if constexpr (T == DOPT_F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

// As Bytes16 for accesses that pass the caches by: a vector type of that alignment.
using u32x4_any = __attribute__((ext_vector_type(4), aligned(2))) uint32_t;

// A matrix of 16-bit elements of more bytes than the 8 L2 caches hold (4 MB each) is read around them where it
// is read once: its lines are gone before anyone could ask again, and what the call
// writes for the next one stays longer.  Of fp32 elements a lane reads 32 bytes in two loads, and around the caches a line
// may be fetched for each: there only the cast does so, from 96 MB on.
constexpr int64_t kStreamBytes = int64_t(32) << 20;
constexpr int64_t kStreamBytesF32 = int64_t(96) << 20;

// Elements [0, n) of the 8 at p, n <= 8, the others zero.
template <int T, bool STREAM = false>
__device__ __forceinline__ Raw8<T> load8(const void *base, int64_t e, int n) {
    Raw8<T> r;
    if (n >= 8) {
        const char *p = static_cast<const char *>(base) + e * (T == DOPT_F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < kWords8<T>; ++i) {
            if constexpr (STREAM) r.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p) + i);
            else r.w[i] = reinterpret_cast<const Bytes16 *>(p)[i].v;
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < kWords8<T>; ++i) r.w[i] = u32x4{0, 0, 0, 0};
    if constexpr (T == DOPT_F32) {
        const uint32_t *p = static_cast<const uint32_t *>(base) + e;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) r.w[i / 4][i % 4] = p[i];
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + e;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) r.w[0][i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i % 2));
    }
    return r;
}

template <int T>
__device__ __forceinline__ float element(const Raw8<T> &r, int i) {
    if constexpr (T == DOPT_F32) return __uint_as_float(r.w[i / 4][i % 4]);
    else return to_float<T>(i % 2 ? r.w[0][i / 2] >> 16 : r.w[0][i / 2] & 0xffffu);
}

template <int T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = element<T>(r, i);
}

template <int T>
__device__ __forceinline__ Raw8<T> pack8(const float (&x)[8]) {
    Raw8<T> r;
    if constexpr (T == DOPT_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i / 4][i % 4] = __float_as_uint(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[0][i] = from_float<T>(x[2 * i]) | from_float<T>(x[2 * i + 1]) << 16;
    }
    return r;
}

template <int T, bool STREAM = false>
__device__ __forceinline__ void store8(void *base, int64_t e, int n, const Raw8<T> &r) {
    if (n >= 8) {
        char *p = static_cast<char *>(base) + e * (T == DOPT_F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < kWords8<T>; ++i) {
            if constexpr (STREAM) __builtin_nontemporal_store(r.w[i], reinterpret_cast<u32x4_any *>(p) + i);
            else reinterpret_cast<Bytes16 *>(p)[i].v = r.w[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) break;
        if constexpr (T == DOPT_F32) static_cast<uint32_t *>(base)[e + i] = r.w[i / 4][i % 4];
        else static_cast<uint16_t *>(base)[e + i] = static_cast<uint16_t>(r.w[0][i / 2] >> (16 * (i % 2)));
    }
}

// 8 consecutive elements of a vector of a type known at run time only.
__device__ __forceinline__ void load_vector8(const void *p, int32_t dtype, int64_t e, int n, float (&x)[8]) {
    if (dtype == DOPT_F32) unpack8<DOPT_F32>(load8<DOPT_F32>(p, e, n), x);
    else if (dtype == DOPT_BF16) unpack8<DOPT_BF16>(load8<DOPT_BF16>(p, e, n), x);
    else unpack8<DOPT_F16>(load8<DOPT_F16>(p, e, n), x);
}

// x * r * w in 64 bits, where x * r is exact and in range, rounded to fp32 at the
// end.  In 32 bits x * r may be infinite or lose bits where the whole would not, and a second rounding
// makes twice as many codes differ from the formula's, since a code lies next to a border as often
// as its value is off.  8192 x 8192 bf16 norm with a residual: 92.5 us; in 32 bits with what
// the first product loses added to the second, 90.6; so, and again in 64 bits where
// a product of the 8 left the range, 95.2.
__device__ __forceinline__ float product3(float x, float r, float w) {
    return static_cast<float>(static_cast<double>(x) * r * w);
}

// ---- device: the 8-bit format -----------------------------------------------------

constexpr uint32_t kInfBits = 0x7f800000u;

// The magnitude's bits, 0 for what is not finite: bits of magnitudes are ordered as they are.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < kInfBits ? b : 0u;
}

// The scale's byte from a block's largest magnitude: 448 = 1.75 * 2^8, so e is
// the exponent of the magnitude, plus one where its mantissa is above 1.75
// (0x600000, which the sum carries into the exponent), minus 8, at least -126.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int e = static_cast<int>((top + 0x1fffffu) >> 23) - 8;
    return e < 1 ? 1u : static_cast<uint32_t>(e);
}

// 2^-e; the byte is in [1, 247], so this is a normal number.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two values as codes in the lower or upper half of `old`.  What is not finite
// becomes a NaN by itself: the conversion turns infinities into NaN.
template <bool HIGH>
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv, uint32_t old) {
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, static_cast<int>(old), HIGH));
}

template <bool STREAM>
__device__ __forceinline__ void store_codes8(uint8_t *p, u32x2 q) {
    if constexpr (STREAM) __builtin_nontemporal_store(q, reinterpret_cast<u32x2 *>(p));
    else *reinterpret_cast<u32x2 *>(p) = q;
}

__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float inv) {
    u32x2 r;
    r[0] = codes2<true>(x[2], x[3], inv, codes2<false>(x[0], x[1], inv, 0));
    r[1] = codes2<true>(x[6], x[7], inv, codes2<false>(x[4], x[5], inv, 0));
    return r;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t u) {
    const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, false));
    return u > o ? u : o;
}

// The largest over each 16 lanes, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t u) {
    u = dpp_max<0xb1>(u);   // quad_perm 1,0,3,2
    u = dpp_max<0x4e>(u);   // quad_perm 2,3,0,1
    u = dpp_max<0x141>(u);  // row_half_mirror
    return dpp_max<0x140>(u);  // row_mirror
}

}  // namespace dopt
