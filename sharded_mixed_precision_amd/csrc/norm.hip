// The RMS norm with an 8-bit output (dopt_rmsnorm) and its backward pass (dopt_rmsnorm_grad).
// Both read a row once and keep it in registers across its sum, and both are
// bound by memory.  On MI355X (a copy reaches 5.1 TB/s): 8192 x 8192 bf16 with a residual 90.3 us a call (5.2 TB/s);
// backward of 8192 x 4096 bf16 with a residual's grad 56.5, 52 of them its own kernel (5.2 TB/s) and 5 for the weight's grad; one row of 4096
// 4 us on the GPU, 1023 x 768 backward 5 and 3, both less than the call's host time.
#include <algorithm>
#include <string>

#include "fp8.h"

namespace dopt {

constexpr int kNormThreads = 256;
constexpr int kLoop = 0;  // NV of the kernels for rows too long for registers

// A row is taken by LANES threads, a wave or a workgroup, each with NV vectors
// of 8 elements: vector v of a row belongs to thread v % LANES, so 16
// neighbouring lanes hold a block of 128 elements and every access of a wave
// is contiguous.  Rows of more than 256 * 8 * 8 elements are read twice.
struct Shape {
    int lanes, nv;
};

static Shape shape_of(int64_t cols) {
    if (cols <= 512) return {64, 1};
    if (cols <= 1024) return {64, 2};
    if (cols <= 2048) return {256, 1};
    if (cols <= 4096) return {256, 2};
    if (cols <= 8192) return {256, 4};
    if (cols <= 16384) return {256, 8};
    return {256, kLoop};
}

template <int LANES, class F>
__device__ __forceinline__ F row_sum(F s, F *shared) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
    if constexpr (LANES > 64) {
        const int w = threadIdx.x / 64;
        __syncthreads();  // the sums of the row before have been read
        if (threadIdx.x % 64 == 0) shared[w] = s;
        __syncthreads();
        s = shared[0];
#pragma unroll
        for (int i = 1; i < LANES / 64; ++i) s += shared[i];
    }
    return s;
}

// The sum of 8 squares, in 64 bits: in 32 one number from 2^64 on would make it infinite, and numbers below
// 2^-75 would not count.
__device__ __forceinline__ double squares8(const float (&x)[8]) {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fma(static_cast<double>(x[j]), static_cast<double>(x[j]), s);
    return s;
}

// 1 / sqrt(sum / cols + eps) to half a step of fp32: an estimate and one Newton step
// in 64 bits, in which no sum of squares of fp32 numbers leaves the range.
__device__ __forceinline__ float rstd_of(double sum, int cols, double eps) {
    const double m = sum / cols + eps;
    const double r = __builtin_amdgcn_rsq(m);
    if (!(r > 0.0 && r < INFINITY)) return static_cast<float>(r);
    return static_cast<float>(r + 0.5 * r * fma(-m * r, r, 1.0));
}

// ---- forward ----------------------------------------------------------------------

struct NormArgs {
    const void *x, *res, *weight;
    void *h, *y;
    uint8_t *codes, *scales;
    float *rstd;
    int64_t x_ld, res_ld, h_ld, y_ld, codes_ld, scale_ld;
    int32_t rows, cols, wdtype;
    double eps;
};

// STREAM: x and the residual are read, and h, which the backward pass asks for, is
// written around the caches; y and its codes are the next product's operands.  8192 x 8192
// bf16 with a residual: 99.8 us with ordinary accesses, 92.1 so; 1024 x 4096: 10.2 and 10.5; 8192 x 4096 fp32 87.6 and 96.5,
// without a residual 40.1 and 41.7.
template <int T, bool STREAM>
__device__ __forceinline__ void load_h(const NormArgs &A, int64_t row, int64_t e, int n, float (&x)[8]) {
    unpack8<T>(load8<T, STREAM>(A.x, row * A.x_ld + e, n), x);
    if (A.res) {
        float r[8];
        unpack8<T>(load8<T, STREAM>(A.res, row * A.res_ld + e, n), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += r[j];
        const Raw8<T> h = pack8<T>(x);
        if (A.h) store8<T, STREAM>(A.h, row * A.h_ld + e, n, h);
        unpack8<T>(h, x);
    } else if (A.h) {
        store8<T, STREAM>(A.h, row * A.h_ld + e, n, pack8<T>(x));
    }
}

template <int T>
__device__ __forceinline__ void write_y(const NormArgs &A, int64_t row, int64_t e, int n, float rstd, const float (&x)[8]) {
    float w[8], y[8];
    load_vector8(A.weight, A.wdtype, e, n, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = j < n ? product3(x[j], rstd, w[j]) : 0.0f;
    if (A.y) store8<T>(A.y, row * A.y_ld + e, n, pack8<T>(y));
    if (A.codes) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, finite_bits(y[j]));
        const uint32_t byte = scale_byte(max16(top));
        if (e < (A.cols + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK * DOPT_FP8_BLOCK) {
            *reinterpret_cast<u32x2 *>(A.codes + row * A.codes_ld + e) = codes8(y, inverse_scale(byte));
            if (e % DOPT_FP8_BLOCK == 0) A.scales[e / DOPT_FP8_BLOCK * A.scale_ld + row] = static_cast<uint8_t>(byte);
        }
    }
}

__device__ __forceinline__ int count8(int64_t cols, int64_t e) {
    const int64_t n = cols - e;
    return n <= 0 ? 0 : n >= 8 ? 8 : static_cast<int>(n);
}

// Workgroups in a row of the grid: a launch has less than 2^32 threads along x, and up to
// 2^30 rows take 2^36 to 2^38.
constexpr int64_t kNormGridX = int64_t(1) << 23;

template <int T, int LANES, int NV, bool STREAM>
__global__ __launch_bounds__(kNormThreads) void k_norm(NormArgs A) {
    __shared__ double s_sum[4];
    const int t = threadIdx.x % LANES;
    const int64_t row = (blockIdx.y * kNormGridX + blockIdx.x) * (kNormThreads / LANES) + threadIdx.x / LANES;
    if (row >= A.rows) return;  // LANES = 256: all threads; 64: whole waves, which do not synchronise
    double s = 0.0;
    if constexpr (NV != kLoop) {
        float x[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t e = 8 * (t + int64_t(LANES) * v);
            load_h<T, STREAM>(A, row, e, count8(A.cols, e), x[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) s += squares8(x[v]);
        const float rstd = rstd_of(row_sum<LANES>(s, s_sum), A.cols, A.eps);
        if (A.rstd && t == 0) A.rstd[row] = rstd;
        // The row is kept as it was loaded, and widened again for y: kept in 64 bits since the squares it would take twice
        // the registers (8192 x 8192 with a residual: 93 us so, 115).
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int j = 0; j < 8; ++j) asm("" : "+v"(x[v][j]));
            const int64_t e = 8 * (t + int64_t(LANES) * v);
            write_y<T>(A, row, e, count8(A.cols, e), rstd, x[v]);
        }
    } else {
        const int64_t end = (A.cols + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK * DOPT_FP8_BLOCK;
        for (int64_t e = 8 * t; e < end; e += 8 * LANES) {
            float x[8];
            load_h<T, false>(A, row, e, count8(A.cols, e), x);
            s += squares8(x);
        }
        const float rstd = rstd_of(row_sum<LANES>(s, s_sum), A.cols, A.eps);
        if (A.rstd && t == 0) A.rstd[row] = rstd;
        NormArgs B = A;  // h is written: x may be h itself, and is not added to again
        if (A.h) {
            B.x = A.h;
            B.x_ld = A.h_ld;
            B.res = nullptr;
            B.h = nullptr;
        }
        // every lane of a block's 16 takes part in its maximum: end is a multiple of 128
        for (int64_t e = 8 * t; e < end; e += 8 * LANES) {
            float x[8];
            load_h<T, false>(B, row, e, count8(A.cols, e), x);
            write_y<T>(B, row, e, count8(A.cols, e), rstd, x);
        }
    }
}

template <int T, bool STREAM>
static void launch_norm_as(const NormArgs &A, hipStream_t stream) {
    const Shape s = shape_of(A.cols);
    const int64_t blocks = (int64_t(A.rows) * s.lanes + kNormThreads - 1) / kNormThreads;
    const dim3 grid(static_cast<unsigned>(std::min(blocks, kNormGridX)), static_cast<unsigned>((blocks + kNormGridX - 1) / kNormGridX));
    if (s.lanes == 64 && s.nv == 1) k_norm<T, 64, 1, STREAM><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.lanes == 64) k_norm<T, 64, 2, STREAM><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.nv == 1) k_norm<T, 256, 1, STREAM><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.nv == 2) k_norm<T, 256, 2, STREAM><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.nv == 4) k_norm<T, 256, 4, STREAM><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.nv == 8) k_norm<T, 256, 8, STREAM><<<grid, kNormThreads, 0, stream>>>(A);
    else k_norm<T, 256, kLoop, false><<<grid, kNormThreads, 0, stream>>>(A);
}

template <int T>
static void launch_norm(const NormArgs &A, hipStream_t stream) {
    if constexpr (T != DOPT_F32) {
        if (int64_t(A.rows) * A.cols * 2 > kStreamBytes) {
            launch_norm_as<T, true>(A, stream);
            return;
        }
    }
    launch_norm_as<T, false>(A, stream);
}

// ---- backward ---------------------------------------------------------------------

struct NormGradArgs {
    const void *dy, *h, *dh, *weight;
    const float *rstd;
    void *dx;
    float *part;  // a row of cols sums per worker
    int64_t dy_ld, h_ld, dh_ld, dx_ld;
    int32_t rows, cols, wdtype, workers;
};

// With n = h * rstd, which is at most sqrt(cols), dx = dh + rstd * (g - n * mean(g * n)): neither rstd^2
// nor g * h is formed, which may be out of range where dx is not.
//
// Workgroups share the rows, a row to a wave or to the whole workgroup, and
// hold the weight's grad of theirs in registers; a workgroup leaves one row of
// sums, which k_norm_weight joins in a fixed order.  512 of them, of at least 2 rows each: 2048 x 4096
// bf16 with a residual's grad takes 20.0 us with 512, 22.7 with 256, 30.9 with 128; 512 x 4096 13.9 with a
// row to each, 12.1 with two, 13.0 with four; 512 x 8192 19.1, 15.1, 16.1; 1023 x 768, of which a workgroup
// takes four rows at once, 8.8 with 256, 9.7 with 128.
constexpr int kMaxWorkers = 512;

// As shape_of, with wider workgroups in place of more vectors to a thread: a
// vector takes 40 registers here.
static Shape grad_shape_of(int64_t cols) {
    if (cols <= 4096) return shape_of(cols);
    if (cols <= 8192) return {512, 2};
    if (cols <= 16384) return {1024, 2};
    return {1024, kLoop};
}

static int64_t workers_of(int64_t rows, int64_t cols) {
    const int64_t at_once = std::max(2, kNormThreads / grad_shape_of(cols).lanes);
    return std::min<int64_t>((rows + at_once - 1) / at_once, kMaxWorkers);
}

template <int T, int TD, int LANES, int NV>
__global__ __launch_bounds__(LANES > kNormThreads ? LANES : kNormThreads) void k_norm_grad(NormGradArgs A) {
    constexpr int kAtOnce = LANES < kNormThreads ? kNormThreads / LANES : 1;
    __shared__ float s_sum[LANES / 64];
    __shared__ float s_dw[LANES == 64 ? kAtOnce - 1 : 1][LANES == 64 ? LANES * NV * 8 : 1];
    const int t = threadIdx.x % LANES, part_of = threadIdx.x / LANES;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kAtOnce + part_of, next = static_cast<int64_t>(A.workers) * kAtOnce;
    const float cols = static_cast<float>(A.cols);
    float *part = A.part + static_cast<int64_t>(blockIdx.x) * A.cols;
    if constexpr (NV != kLoop) {
        float w[NV][8], dw[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t e = 8 * (t + int64_t(LANES) * v);
            load_vector8(A.weight, A.wdtype, e, count8(A.cols, e), w[v]);
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[v][j] = 0.0f;
        }
        for (int64_t row = first; row < A.rows; row += next) {
            Raw8<TD> dy[NV];
            Raw8<T> h[NV], dh[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int64_t e = 8 * (t + int64_t(LANES) * v);
                const int n = count8(A.cols, e);
                dy[v] = load8<TD>(A.dy, row * A.dy_ld + e, n);
                h[v] = load8<T>(A.h, row * A.h_ld + e, n);
                if (A.dh) dh[v] = load8<T>(A.dh, row * A.dh_ld + e, n);
            }
            const float rstd = A.rstd[row];
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(element<TD>(dy[v], j) * w[v][j], element<T>(h[v], j) * rstd, s);
            const float c = row_sum<LANES>(s, s_sum) / cols;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int64_t e = 8 * (t + int64_t(LANES) * v);
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = element<TD>(dy[v], j), n = element<T>(h[v], j) * rstd;
                    dw[v][j] = fmaf(d, n, dw[v][j]);
                    x[j] = rstd * (d * w[v][j] - n * c);
                    if (A.dh) x[j] += element<T>(dh[v], j);
                }
                store8<T>(A.dx, row * A.dx_ld + e, count8(A.cols, e), pack8<T>(x));
            }
        }
        if constexpr (LANES == 64) {
            if (part_of > 0) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s_dw[part_of - 1][(8 * v + j) * 64 + t] = dw[v][j];
            }
            __syncthreads();
            if (part_of > 0) return;
#pragma unroll
            for (int i = 0; i < kAtOnce - 1; ++i)
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) dw[v][j] += s_dw[i][(8 * v + j) * 64 + t];
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t e = 8 * (t + int64_t(LANES) * v);
            store8<DOPT_F32>(part, e, count8(A.cols, e), pack8<DOPT_F32>(dw[v]));
        }
    } else {
        for (int64_t row = first; row < A.rows; row += next) {
            const float rstd = A.rstd[row];
            float s = 0.0f;
            for (int64_t e = 8 * t; e < A.cols; e += 8 * LANES) {
                const int n = count8(A.cols, e);
                float d[8], hx[8], w[8], q = 0.0f;
                unpack8<TD>(load8<TD>(A.dy, row * A.dy_ld + e, n), d);
                unpack8<T>(load8<T>(A.h, row * A.h_ld + e, n), hx);
                load_vector8(A.weight, A.wdtype, e, n, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) q = fmaf(d[j] * w[j], hx[j] * rstd, q);
                s += q;
            }
            const float c = row_sum<LANES>(s, s_sum) / cols;
            for (int64_t e = 8 * t; e < A.cols; e += 8 * LANES) {
                const int n = count8(A.cols, e);
                float d[8], hx[8], w[8], x[8], dw[8], r[8];
                unpack8<TD>(load8<TD>(A.dy, row * A.dy_ld + e, n), d);
                unpack8<T>(load8<T>(A.h, row * A.h_ld + e, n), hx);
                load_vector8(A.weight, A.wdtype, e, n, w);
                unpack8<DOPT_F32>(load8<DOPT_F32>(part, e, row == first ? 0 : n), dw);
                unpack8<T>(load8<T>(A.dh ? A.dh : A.h, row * (A.dh ? A.dh_ld : A.h_ld) + e, A.dh ? n : 0), r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float nj = hx[j] * rstd;
                    dw[j] = fmaf(d[j], nj, dw[j]);
                    x[j] = rstd * (d[j] * w[j] - nj * c);
                    if (A.dh) x[j] += r[j];
                }
                store8<T>(A.dx, row * A.dx_ld + e, n, pack8<T>(x));
                store8<DOPT_F32>(part, e, n, pack8<DOPT_F32>(dw));
            }
        }
    }
}

// The workers' sums of 32 columns: 8 lanes of 4 columns each, 128 slices of
// the workers, so that a thread has at most 4 loads, all under way at once.
constexpr int kJoinThreads = 1024;

__global__ __launch_bounds__(kJoinThreads) void k_norm_weight(const float *part, int workers, int cols, void *out,
                                                               int32_t dtype, int accumulate) {
    __shared__ f32x4 s_part[kJoinThreads / 64][8];
    const int lane = threadIdx.x % 8, slice = threadIdx.x / 8;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 32 + 4 * lane;
    const int n = c0 >= cols ? 0 : cols - c0 >= 4 ? 4 : static_cast<int>(cols - c0);
    f32x4 s = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kMaxWorkers / 128; ++i) {
        const int w = slice + 128 * i;
        if (w >= workers || n == 0) continue;
        const float *p = part + static_cast<int64_t>(w) * cols + c0;
        if (n == 4) {
            s += reinterpret_cast<const Float4 *>(p)->v;
        } else {
            for (int j = 0; j < n; ++j) s[j] += p[j];
        }
    }
#pragma unroll
    for (int m = 8; m < 64; m <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += __shfl_xor(s[j], m);
    if (threadIdx.x % 64 < 8) s_part[threadIdx.x / 64][lane] = s;
    __syncthreads();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    if (threadIdx.x >= 32 || c >= cols) return;
    float s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinThreads / 64; ++i) s1 += s_part[i][threadIdx.x / 4][threadIdx.x % 4];
    if (dtype == DOPT_F32) {
        float *p = static_cast<float *>(out) + c;
        *p = accumulate ? *p + s1 : s1;
    } else {
        uint16_t *p = static_cast<uint16_t *>(out) + c;
        if (dtype == DOPT_BF16) *p = static_cast<uint16_t>(from_float<DOPT_BF16>(accumulate ? to_float<DOPT_BF16>(*p) + s1 : s1));
        else *p = static_cast<uint16_t>(from_float<DOPT_F16>(accumulate ? to_float<DOPT_F16>(*p) + s1 : s1));
    }
}

template <int T, int TD>
static void launch_norm_grad(const NormGradArgs &A, hipStream_t stream) {
    const Shape s = grad_shape_of(A.cols);
    const unsigned grid = static_cast<unsigned>(A.workers);
    if (s.lanes == 64 && s.nv == 1) k_norm_grad<T, TD, 64, 1><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.lanes == 64) k_norm_grad<T, TD, 64, 2><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.lanes == 256 && s.nv == 1) k_norm_grad<T, TD, 256, 1><<<grid, kNormThreads, 0, stream>>>(A);
    else if (s.lanes == 256) k_norm_grad<T, TD, 256, 2><<<grid, 256, 0, stream>>>(A);
    else if (s.lanes == 512) k_norm_grad<T, TD, 512, 2><<<grid, 512, 0, stream>>>(A);
    else if (s.nv == 2) k_norm_grad<T, TD, 1024, 2><<<grid, 1024, 0, stream>>>(A);
    else k_norm_grad<T, TD, 1024, kLoop><<<grid, 1024, 0, stream>>>(A);
}

// `x` is of the size and type of `like`.
static int check_like(const char *name, const dopt_dense *x, const dopt_dense *like, bool type) {
    if (int rc = check_dense(name, x)) return rc;
    if (x->rows != like->rows || x->cols != like->cols) return fail(DOPT_ERR_INVALID, std::string(name) + ": of another size");
    if (type && x->dtype != like->dtype) return fail(DOPT_ERR_INVALID, std::string(name) + ": of another type");
    return DOPT_OK;
}

// Whether `a` is the same elements as `b`, so that a thread that has read them may write them.
static bool same(const dopt_dense *a, const dopt_dense *b) {
    return a && b && a->data == b->data && a->ld == b->ld && a->dtype == b->dtype;
}

}  // namespace dopt

using namespace dopt;

extern "C" int dopt_rmsnorm(const dopt_dense *x, const dopt_dense *residual, const void *weight, int32_t weight_dtype,
                            double eps, const dopt_dense *h, const dopt_dense *y, const dopt_fp8_matrix *q, float *rstd,
                            hipStream_t stream) {
    if (int rc = check_dense("x", x)) return rc;
    if (residual)
        if (int rc = check_like("residual", residual, x, true)) return rc;
    if (h)
        if (int rc = check_like("h", h, x, true)) return rc;
    if (y)
        if (int rc = check_like("y", y, x, true)) return rc;
    if (q) {
        if (int rc = check_fp8("q", q)) return rc;
        if (q->kind != DOPT_FP8_ROW) return fail(DOPT_ERR_INVALID, "q: not of kind ROW");
        if (q->rows != x->rows || q->cols != x->cols) return fail(DOPT_ERR_INVALID, "q: of another size");
    }
    if (!y && !q) return fail(DOPT_ERR_INVALID, "neither y nor q is asked for");
    if (!(eps >= 0.0)) return fail(DOPT_ERR_INVALID, "eps is negative or NaN");
    if (int rc = check_vector("weight", weight, x->cols, weight_dtype)) return rc;
    if (reinterpret_cast<uintptr_t>(rstd) % 4) return fail(DOPT_ERR_INVALID, "rstd: device pointer not aligned to its element");
    if (x->rows == 0 || x->cols == 0) return DOPT_OK;
    if (x->cols > DOPT_FP8_MAX_COLS) return fail(DOPT_ERR_INVALID, "x: too many columns");

    const Span out[] = {dense_span("h", h), dense_span("y", y), codes_span("q", q), scales_span("q's scales", q),
                        span_of("rstd", rstd, 4 * x->rows)};
    const Span none = span_of("", nullptr, 0), vec = span_of("weight", weight, element_bytes(weight_dtype) * x->cols);
    const Span in[] = {dense_span("x", x), dense_span("residual", residual), vec};
    const Span in_h[] = {same(h, x) ? none : in[0], same(h, residual) ? none : in[1], vec};
    if (int rc = check_apart(out, 5, nullptr, 0)) return rc;
    if (int rc = check_apart(out, 1, in_h, 3)) return rc;
    if (int rc = check_apart(out + 1, 4, in, 3)) return rc;

    NormArgs A{};
    A.x = x->data;
    A.x_ld = x->ld;
    if (residual) {
        A.res = residual->data;
        A.res_ld = residual->ld;
    }
    // without a residual h is x: nothing is written where it is x itself
    if (h && !(same(h, x) && !residual)) {
        A.h = h->data;
        A.h_ld = h->ld;
    }
    if (y) {
        A.y = y->data;
        A.y_ld = y->ld;
    }
    if (q) {
        A.codes = static_cast<uint8_t *>(q->codes);
        A.scales = static_cast<uint8_t *>(q->scales);
        A.codes_ld = q->ld;
        A.scale_ld = q->scale_ld;
    }
    A.weight = weight;
    A.wdtype = weight_dtype;
    A.rstd = rstd;
    A.rows = static_cast<int32_t>(x->rows);
    A.cols = static_cast<int32_t>(x->cols);
    A.eps = eps;
    if (x->dtype == DOPT_F32) launch_norm<DOPT_F32>(A, stream);
    else if (x->dtype == DOPT_BF16) launch_norm<DOPT_BF16>(A, stream);
    else launch_norm<DOPT_F16>(A, stream);
    return launched("dopt_rmsnorm");
}

extern "C" int64_t dopt_rmsnorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > DOPT_FP8_MAX_ROWS || cols > DOPT_FP8_MAX_COLS) return fail(DOPT_ERR_INVALID, "bad size");
    return workers_of(rows, cols) * cols * 4;
}

extern "C" int dopt_rmsnorm_grad(const dopt_dense *dy, const dopt_dense *h, const dopt_dense *dh, const void *weight,
                                 int32_t weight_dtype, const float *rstd, const dopt_dense *dx, void *dweight,
                                 int32_t dweight_dtype, int32_t accumulate, void *workspace, int64_t workspace_bytes,
                                 hipStream_t stream) {
    if (int rc = check_dense("h", h)) return rc;
    if (int rc = check_like("dy", dy, h, false)) return rc;
    if (dy->dtype != h->dtype && dy->dtype != DOPT_F32) return fail(DOPT_ERR_INVALID, "dy: neither of h's type nor fp32");
    if (dh)
        if (int rc = check_like("dh", dh, h, true)) return rc;
    if (int rc = check_like("dx", dx, h, true)) return rc;
    if (int rc = check_vector("weight", weight, h->cols, weight_dtype)) return rc;
    if (int rc = check_vector("dweight", dweight, h->cols, dweight_dtype)) return rc;
    if (int rc = check_vector("rstd", rstd, h->rows, DOPT_F32)) return rc;
    if (h->cols > DOPT_FP8_MAX_COLS) return fail(DOPT_ERR_INVALID, "h: too many columns");
    if (h->cols == 0) return DOPT_OK;
    const int64_t need = dopt_rmsnorm_grad_workspace_bytes(h->rows, h->cols);
    if (need > 0 && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16))
        return fail(DOPT_ERR_INVALID, "workspace: null, not 16-byte aligned or too small (" + std::to_string(need) + " bytes)");
    const Span out[] = {dense_span("dx", dx), span_of("dweight", dweight, element_bytes(dweight_dtype) * h->cols),
                        span_of("workspace", workspace, need)};
    const Span none = span_of("", nullptr, 0), vec = span_of("weight", weight, element_bytes(weight_dtype) * h->cols);
    const Span kept = span_of("rstd", rstd, 4 * h->rows);
    const Span in[] = {dense_span("dy", dy), dense_span("h", h), dense_span("dh", dh), vec, kept};
    const Span in_dx[] = {same(dx, dy) ? none : in[0], in[1], same(dx, dh) ? none : in[2], vec, kept};
    if (int rc = check_apart(out, 3, nullptr, 0)) return rc;
    if (int rc = check_apart(out, 1, in_dx, 5)) return rc;
    if (int rc = check_apart(out + 1, 2, in, 5)) return rc;

    const int64_t workers = h->rows > 0 ? workers_of(h->rows, h->cols) : 0;
    if (workers > 0) {
        NormGradArgs A{};
        A.dy = dy->data;
        A.dy_ld = dy->ld;
        A.h = h->data;
        A.h_ld = h->ld;
        if (dh) {
            A.dh = dh->data;
            A.dh_ld = dh->ld;
        }
        A.dx = dx->data;
        A.dx_ld = dx->ld;
        A.weight = weight;
        A.wdtype = weight_dtype;
        A.rstd = rstd;
        A.part = static_cast<float *>(workspace);
        A.rows = static_cast<int32_t>(h->rows);
        A.cols = static_cast<int32_t>(h->cols);
        A.workers = static_cast<int32_t>(workers);
        const bool wide = dy->dtype == DOPT_F32;
        if (h->dtype == DOPT_F32) launch_norm_grad<DOPT_F32, DOPT_F32>(A, stream);
        else if (h->dtype == DOPT_BF16 && wide) launch_norm_grad<DOPT_BF16, DOPT_F32>(A, stream);
        else if (h->dtype == DOPT_BF16) launch_norm_grad<DOPT_BF16, DOPT_BF16>(A, stream);
        else if (wide) launch_norm_grad<DOPT_F16, DOPT_F32>(A, stream);
        else launch_norm_grad<DOPT_F16, DOPT_F16>(A, stream);
        if (int rc = launched("dopt_rmsnorm_grad")) return rc;
    }
    if (workers == 0 && accumulate) return DOPT_OK;
    k_norm_weight<<<static_cast<unsigned>((h->cols + 31) / 32), kJoinThreads, 0, stream>>>(
        static_cast<const float *>(workspace), static_cast<int>(workers), static_cast<int>(h->cols), dweight, dweight_dtype, accumulate);
    return launched("dopt_rmsnorm_grad");
}
