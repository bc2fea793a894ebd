// The cast to block-scaled e4m3 (dopt_fp8_cast), and the checks that the 8-bit operators share.
#include <cstdio>
#include <string>

#include "fp8.h"

namespace dopt {

// ---- checks -----------------------------------------------------------------------

int check_dense(const char *name, const dopt_dense *x) {
    const std::string n(name);
    if (!x) return fail(DOPT_ERR_INVALID, n + ": null");
    if (!is_dtype(x->dtype)) return fail(DOPT_ERR_INVALID, n + ": bad dtype");
    if (x->rows < 0 || x->cols < 0 || x->rows > DOPT_FP8_MAX_ROWS || x->cols > DOPT_FP8_MAX_ROWS)
        return fail(DOPT_ERR_INVALID, n + ": bad size");
    if (x->rows == 0 || x->cols == 0) return DOPT_OK;
    if (x->ld < x->cols || x->ld >= (1 << 23)) return fail(DOPT_ERR_INVALID, n + ": bad distance between rows");
    if (!x->data) return fail(DOPT_ERR_INVALID, n + ": null device pointer");
    if (reinterpret_cast<uintptr_t>(x->data) % element_bytes(x->dtype))
        return fail(DOPT_ERR_INVALID, n + ": device pointer not aligned to its element");
    return DOPT_OK;
}

int check_fp8(const char *name, const dopt_fp8_matrix *x) {
    const std::string n(name);
    if (!x) return fail(DOPT_ERR_INVALID, n + ": null");
    if (x->kind != DOPT_FP8_ROW && x->kind != DOPT_FP8_TILE) return fail(DOPT_ERR_INVALID, n + ": bad kind");
    if (x->rows < 0 || x->cols < 0 || x->rows > DOPT_FP8_MAX_ROWS || x->cols > DOPT_FP8_MAX_COLS)
        return fail(DOPT_ERR_INVALID, n + ": bad size");
    if (x->rows == 0 || x->cols == 0) return DOPT_OK;
    const int64_t padded = (x->cols + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK * DOPT_FP8_BLOCK;
    if (x->ld < padded || x->ld % 16 || x->ld > DOPT_FP8_MAX_COLS)
        return fail(DOPT_ERR_INVALID, n + ": bad distance between rows of codes");
    const bool row = x->kind == DOPT_FP8_ROW;
    if (x->scale_ld < (row ? x->rows : (x->rows + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK) || (row && x->scale_ld % 4) ||
        x->scale_ld > (int64_t(1) << 31))
        return fail(DOPT_ERR_INVALID, n + ": bad distance between rows of scales");
    if (!x->codes || !x->scales) return fail(DOPT_ERR_INVALID, n + ": null device pointer");
    if (reinterpret_cast<uintptr_t>(x->codes) % 16) return fail(DOPT_ERR_INVALID, n + ": codes not 16-byte aligned");
    if (row && reinterpret_cast<uintptr_t>(x->scales) % 4) return fail(DOPT_ERR_INVALID, n + ": scales not 4-byte aligned");
    return DOPT_OK;
}

int check_vector(const char *name, const void *p, int64_t n, int32_t dtype) {
    if (!is_dtype(dtype)) return fail(DOPT_ERR_INVALID, std::string(name) + ": bad dtype");
    if (n == 0) return DOPT_OK;
    if (!p) return fail(DOPT_ERR_INVALID, std::string(name) + ": null device pointer");
    if (reinterpret_cast<uintptr_t>(p) % element_bytes(dtype))
        return fail(DOPT_ERR_INVALID, std::string(name) + ": device pointer not aligned to its element");
    return DOPT_OK;
}

Span dense_span(const char *name, const dopt_dense *x) {
    if (!x || x->rows == 0 || x->cols == 0) return span_of(name, nullptr, 0);
    const int es = element_bytes(x->dtype);
    return span_of(name, x->data, ((x->rows - 1) * x->ld + x->cols) * es, x->ld * es, x->cols * es);
}

Span codes_span(const char *name, const dopt_fp8_matrix *x) {
    if (!x || x->rows == 0 || x->cols == 0) return span_of(name, nullptr, 0);
    const int64_t padded = (x->cols + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK * DOPT_FP8_BLOCK;
    return span_of(name, x->codes, (x->rows - 1) * x->ld + padded, x->ld, padded);
}

Span scales_span(const char *name, const dopt_fp8_matrix *x) {
    if (!x || x->rows == 0 || x->cols == 0) return span_of(name, nullptr, 0);
    const int64_t groups = (x->cols + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK;
    const int64_t last = x->kind == DOPT_FP8_ROW ? x->rows : (x->rows + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK;
    return span_of(name, x->scales, (groups - 1) * x->scale_ld + last, x->scale_ld, last);
}

int check_apart(const Span *out, int n_out, const Span *in, int n_in) {
    const auto meet = [](const Span &a, const Span &b) {
        if (a.lo == a.hi || b.lo == b.hi || a.lo >= b.hi || b.lo >= a.hi) return false;
        if (a.pitch == 0 || a.pitch != b.pitch) return true;
        const uint64_t pitch = static_cast<uint64_t>(a.pitch);
        const uint64_t at = b.lo >= a.lo ? (b.lo - a.lo) % pitch : (pitch - (a.lo - b.lo) % pitch) % pitch;
        return at < static_cast<uint64_t>(a.width) || at + static_cast<uint64_t>(b.width) > pitch;
    };
    for (int i = 0; i < n_out; ++i) {
        for (int k = 0; k < i; ++k)
            if (meet(out[i], out[k])) return fail(DOPT_ERR_INVALID, std::string(out[i].name) + " overlaps " + out[k].name);
        for (int k = 0; k < n_in; ++k)
            if (meet(out[i], in[k])) return fail(DOPT_ERR_INVALID, std::string(out[i].name) + " overlaps " + in[k].name);
    }
    return DOPT_OK;
}

int launched(const char *what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(DOPT_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
    return DOPT_OK;
}

// ---- cast -------------------------------------------------------------------------

struct CastArgs {
    const void *x;
    const float *row;
    const void *col;
    uint8_t *codes, *scales, *t_codes, *t_scales;
    int64_t ld, codes_ld, scale_ld, t_codes_ld, t_scale_ld;
    int32_t rows, cols, col_dtype, col_tiles;
};

constexpr int kCastThreads = 256;

// One workgroup casts a tile of 128 x 128 elements both ways, so x is read
// once.  A thread holds 8 x 8 elements: 16 neighbouring lanes hold 8 rows of
// 128 elements, so a row's largest magnitude is a maximum over 16 lanes and
// its codes leave as 128 consecutive bytes.  Columns are joined over the
// threads through shared memory, and the transposed codes pass through it, so
// that they too leave as 128 consecutive bytes of a row.  What bounds it is memory: 8191 x 4096 bf16,
// both ways, 28.4 us (4.7 TB/s; a copy reaches 5.1), 14336 x 4096 weights 43.3 us (5.4 TB/s).
struct CastMem {
    uint32_t top[4][DOPT_FP8_BLOCK];
    alignas(16) uint8_t codes[DOPT_FP8_BLOCK * DOPT_FP8_BLOCK];
};

// STREAM: x is read around the caches, and weights' codes (TILE) are written
// around them: they are asked for when the other layers' weights have been cast, while a grad's or an
// activation's (ROW) are the next product's operands.  8192 x 4096 bf16, both ways, ROW: 30.8 us
// with ordinary reads, 28.6 around the caches, 24.8 with the codes too, but then the product of
// 4096 x 14336 behind it takes 10 us longer; 1024 x 4096: 8.2 and 8.5.  14336 x 4096, TILE: 47.8 and 43.6.  fp32, codes only, ROW
// and TILE: 4096 x 4096 15.0 and 14.9 us with ordinary reads, 19.6 and 17.7 around; 6000 x 4096 26.5 and 26.4, 26.6 and 25.2; 14336 x 4096
// 56.1 and 56.2, 55.3 and 52.8.
template <int T, bool TILE, bool WHOLE, bool STREAM>
__device__ __forceinline__ void cast_tile(const CastArgs &A, CastMem &mem, int row0, int col0) {
    auto &s_top = mem.top;
    auto &s_codes = mem.codes;
    const int t = threadIdx.x, cx = t % 16, ry = t / 16;
    const int r0 = row0 + 8 * ry, c0 = col0 + 8 * cx;
    const int n_cols = WHOLE || A.cols - c0 > 8 ? 8 : A.cols - c0 < 0 ? 0 : A.cols - c0;
    const auto inside = [&](int i) { return WHOLE || r0 + i < A.rows; };
    float x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        unpack8<T>(load8<T, STREAM>(A.x, static_cast<int64_t>(r0 + i) * A.ld + c0, WHOLE ? 8 : inside(i) ? n_cols : 0), x[i]);
    if (A.row) {
        float c[8];
        load_vector8(A.col, A.col_dtype, c0, n_cols, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = inside(i) ? A.row[r0 + i] : 0.0f;
            // what pads the tile stays 0 beside factors that are not finite
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = inside(i) && j < n_cols ? product3(x[i][j], r, c[j]) : 0.0f;
        }
    }

    uint32_t byte = 0;  // TILE: the tile's
    if constexpr (TILE) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, finite_bits(x[i][j]));
        top = max16(top);
        if (cx == 0) s_top[0][ry] = top;
        __syncthreads();
        top = s_top[0][cx];
        byte = scale_byte(max16(top));
        if (t == 0) {
            const int64_t i = row0 / DOPT_FP8_BLOCK, j = col0 / DOPT_FP8_BLOCK;
            if (A.codes) A.scales[j * A.scale_ld + i] = static_cast<uint8_t>(byte);
            if (A.t_codes) A.t_scales[i * A.t_scale_ld + j] = static_cast<uint8_t>(byte);
        }
    }

    u32x2 q[8];
    if (A.codes || TILE) {
        uint64_t bytes = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (!TILE) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, finite_bits(x[i][j]));
                byte = scale_byte(max16(top));
                bytes |= static_cast<uint64_t>(byte) << (8 * i);
            }
            q[i] = codes8(x[i], inverse_scale(byte));
        }
        if (A.codes) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (inside(i)) store_codes8<STREAM && TILE>(A.codes + static_cast<int64_t>(r0 + i) * A.codes_ld + c0, q[i]);
            if constexpr (!TILE)
                if (cx < 8 && (WHOLE || r0 + cx < A.rows))
                    A.scales[static_cast<int64_t>(col0 / DOPT_FP8_BLOCK) * A.scale_ld + r0 + cx] = static_cast<uint8_t>(bytes >> (8 * cx));
        }
    }
    if (!A.t_codes) return;

    // column j of the thread's 8 x 8 elements as 8 codes, at row c0 + j of the transposed tile
    if constexpr (!TILE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, finite_bits(x[i][j]));
            top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
            top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
            if (t % 64 < 16) s_top[t / 64][8 * cx + j] = top;
        }
        __syncthreads();
        if (t < DOPT_FP8_BLOCK) {
            byte = scale_byte(max(max(s_top[0][t], s_top[1][t]), max(s_top[2][t], s_top[3][t])));
            if (WHOLE || col0 + t < A.cols)
                A.t_scales[static_cast<int64_t>(row0 / DOPT_FP8_BLOCK) * A.t_scale_ld + col0 + t] = static_cast<uint8_t>(byte);
            s_top[0][t] = byte;
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        u32x2 w;
        if constexpr (TILE) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[h] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[h] |= ((q[4 * h + i][j / 4] >> (8 * (j % 4))) & 0xffu) << (8 * i);
            }
        } else {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i][j];
            w = codes8(y, inverse_scale(s_top[0][8 * cx + j]));
        }
        // 16 chunks of 8 bytes to a row; the XOR spreads the 16 lanes of one ry over all banks
        *reinterpret_cast<u32x2 *>(s_codes + (8 * cx + j) * DOPT_FP8_BLOCK + 8 * (ry ^ cx)) = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = ry + 16 * i;
        const u32x2 w = *reinterpret_cast<const u32x2 *>(s_codes + c * DOPT_FP8_BLOCK + 8 * (cx ^ (c / 8)));
        if (WHOLE || col0 + c < A.cols)
            store_codes8<STREAM && TILE>(A.t_codes + static_cast<int64_t>(col0 + c) * A.t_codes_ld + row0 + 8 * cx, w);
    }
}

// Tiles that are whole, which most are, take code without bounds.
template <int T, bool TILE, bool STREAM>
__global__ __launch_bounds__(kCastThreads) void k_cast(CastArgs A) {
    __shared__ CastMem mem;
    const int row0 = blockIdx.x / A.col_tiles * DOPT_FP8_BLOCK, col0 = blockIdx.x % A.col_tiles * DOPT_FP8_BLOCK;
    if (row0 + DOPT_FP8_BLOCK <= A.rows && col0 + DOPT_FP8_BLOCK <= A.cols) cast_tile<T, TILE, true, STREAM>(A, mem, row0, col0);
    else cast_tile<T, TILE, false, STREAM>(A, mem, row0, col0);
}

template <int T>
static void launch_cast(const CastArgs &A, bool tile, unsigned grid, hipStream_t stream) {
    const bool around = T == DOPT_F32 ? int64_t(A.rows) * A.cols * 4 > kStreamBytesF32 : int64_t(A.rows) * A.cols * 2 > kStreamBytes;
    if (tile && around) k_cast<T, true, true><<<grid, kCastThreads, 0, stream>>>(A);
    else if (tile) k_cast<T, true, false><<<grid, kCastThreads, 0, stream>>>(A);
    else if (around) k_cast<T, false, true><<<grid, kCastThreads, 0, stream>>>(A);
    else k_cast<T, false, false><<<grid, kCastThreads, 0, stream>>>(A);
}

}  // namespace dopt

using namespace dopt;

extern "C" int dopt_fp8_layout(int64_t rows, int64_t cols, int32_t kind, dopt_fp8_sizes *out) {
    if (!out) return fail(DOPT_ERR_INVALID, "null output");
    if (kind != DOPT_FP8_ROW && kind != DOPT_FP8_TILE) return fail(DOPT_ERR_INVALID, "bad kind");
    if (rows < 0 || cols < 0 || rows > DOPT_FP8_MAX_ROWS || cols > DOPT_FP8_MAX_COLS) return fail(DOPT_ERR_INVALID, "bad size");
    const int64_t groups = (cols + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK;
    out->ld = groups * DOPT_FP8_BLOCK;
    out->scale_ld = kind == DOPT_FP8_ROW ? (rows + 15) / 16 * 16 : (rows + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK;
    out->codes_bytes = rows * out->ld;
    out->scales_bytes = groups * out->scale_ld;
    return DOPT_OK;
}

extern "C" int dopt_fp8_cast(const dopt_dense *x, const float *row_factor, const void *col_factor, int32_t col_dtype,
                             const dopt_fp8_matrix *codes, const dopt_fp8_matrix *transposed, hipStream_t stream) {
    if (int rc = check_dense("x", x)) return rc;
    if (!codes && !transposed) return fail(DOPT_ERR_INVALID, "neither codes nor transposed is asked for");
    if (codes) {
        if (int rc = check_fp8("codes", codes)) return rc;
        if (codes->rows != x->rows || codes->cols != x->cols) return fail(DOPT_ERR_INVALID, "codes: not of x's size");
    }
    if (transposed) {
        if (int rc = check_fp8("transposed", transposed)) return rc;
        if (transposed->rows != x->cols || transposed->cols != x->rows)
            return fail(DOPT_ERR_INVALID, "transposed: not of the size of x's transpose");
    }
    if (codes && transposed && codes->kind != transposed->kind) return fail(DOPT_ERR_INVALID, "codes and transposed differ in kind");
    if (!row_factor != !col_factor && x->rows > 0 && x->cols > 0)
        return fail(DOPT_ERR_INVALID, "row and column factors come together");
    if (col_factor) {
        if (int rc = check_vector("row_factor", row_factor, x->rows, DOPT_F32)) return rc;
        if (int rc = check_vector("col_factor", col_factor, x->cols, col_dtype)) return rc;
    }
    if (x->rows == 0 || x->cols == 0) return DOPT_OK;
    const Span out[] = {codes_span("codes", codes), scales_span("codes' scales", codes),
                        codes_span("transposed", transposed), scales_span("transposed's scales", transposed)};
    const Span in[] = {dense_span("x", x), span_of("row_factor", row_factor, 4 * x->rows),
                       span_of("col_factor", col_factor, element_bytes(col_dtype) * x->cols)};
    if (int rc = check_apart(out, 4, in, 3)) return rc;

    CastArgs A{};
    A.x = x->data;
    A.row = row_factor;
    A.col = col_factor;
    A.ld = x->ld;
    A.rows = static_cast<int32_t>(x->rows);
    A.cols = static_cast<int32_t>(x->cols);
    A.col_dtype = col_dtype;
    if (codes) {
        A.codes = static_cast<uint8_t *>(codes->codes);
        A.scales = static_cast<uint8_t *>(codes->scales);
        A.codes_ld = codes->ld;
        A.scale_ld = codes->scale_ld;
    }
    if (transposed) {
        A.t_codes = static_cast<uint8_t *>(transposed->codes);
        A.t_scales = static_cast<uint8_t *>(transposed->scales);
        A.t_codes_ld = transposed->ld;
        A.t_scale_ld = transposed->scale_ld;
    }
    A.col_tiles = static_cast<int32_t>((x->cols + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK);
    const int64_t tiles = (x->rows + DOPT_FP8_BLOCK - 1) / DOPT_FP8_BLOCK * A.col_tiles;
    if (tiles * kCastThreads >= kMaxThreads) return fail(DOPT_ERR_INVALID, "x: too large");
    const bool tile = (codes ? codes : transposed)->kind == DOPT_FP8_TILE;
    const unsigned grid = static_cast<unsigned>(tiles);
    if (x->dtype == DOPT_F32) launch_cast<DOPT_F32>(A, tile, grid, stream);
    else if (x->dtype == DOPT_BF16) launch_cast<DOPT_BF16>(A, tile, grid, stream);
    else launch_cast<DOPT_F16>(A, tile, grid, stream);
    return launched("dopt_fp8_cast");
}
