// linear8_api.cu -- C ABI of the 8-bit linear layers: norm and activation with 8-bit output, and the
// product of 8-bit integers.  Argument validation only; the kernels live in row_quant.cuh and
// w8a8_*.cu.
#include <algorithm>
#include <cmath>

#include "linear8_internal.h"

using qgi::fail;

namespace {

constexpr int64_t MAX_COUNT = (int64_t(1) << 31) - 1;
constexpr int64_t MOST_ROUNDED = (int64_t(1) << 31) - 4096;     // sizes that the product's kernels round up to whole tiles

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

qgemm_status cuda_fail(cudaError_t e, const char *what) {
    return fail(QGEMM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

qgemm_status check_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative shape");
    if (rows > MAX_COUNT || cols > MAX_COUNT) return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "dimension >= 2^31");
    return QGEMM_OK;
}

// An input of rows of `item`-byte elements: rows may overlap or repeat (stride 0).  The stride of a
// single row is never stepped.
qgemm_status check_input(const void *p, int64_t ld, int64_t rows, int item, const char *what) {
    if (!p) return fail(QGEMM_ERR_INVALID_ARG, "%s is NULL", what);
    if (rows > 1 && ld < 0) return fail(QGEMM_ERR_INVALID_ARG, "%s: negative row stride", what);
    if (!aligned(p, item)) return fail(QGEMM_ERR_MISALIGNED, "%s must be %d-byte aligned", what, item);
    if (rows > 1 && ld > (int64_t(1) << 60) / rows) return fail(QGEMM_ERR_INVALID_ARG, "%s: row stride too large", what);
    return QGEMM_OK;
}

qgemm_status check_output(const void *p, int64_t ld, int64_t rows, int64_t cols, int item, const char *what) {
    if (!p) return fail(QGEMM_ERR_INVALID_ARG, "%s is NULL", what);
    if (rows > 1 && ld < cols)
        return fail(QGEMM_ERR_INVALID_ARG, "%s: row stride %lld < %lld elements", what, (long long)ld, (long long)cols);
    if (!aligned(p, item)) return fail(QGEMM_ERR_MISALIGNED, "%s must be %d-byte aligned", what, item);
    if (rows > 1 && ld > (int64_t(1) << 60) / rows) return fail(QGEMM_ERR_INVALID_ARG, "%s: row stride too large", what);
    return QGEMM_OK;
}

// Whether rows [p, ...) and [q, ...) of `rowp` and `rowq` elements share a byte (strides 0 where there is
// one row).  Rows of one stride in bytes may lie between each other's, as the halves of a fused buffer do; of two
// strides, extents that meet count as an overlap.
bool overlap(const void *p, int64_t ldp, int64_t rowp, int ip, const void *q, int64_t ldq, int64_t rowq, int iq,
             int64_t rows) {
    if (!p || !q) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    const uintptr_t ea = a + (uintptr_t)(((rows - 1) * ldp + rowp) * ip);
    const uintptr_t eb = b + (uintptr_t)(((rows - 1) * ldq + rowq) * iq);
    if (a >= eb || b >= ea) return false;
    const uintptr_t step = (uintptr_t)(ldp * ip);
    if (rows == 1 || step == 0 || step != (uintptr_t)(ldq * iq)) return true;
    const uintptr_t d = b >= a ? (b - a) % step : (step - (a - b) % step) % step;
    return d < (uintptr_t)(rowp * ip) || d + (uintptr_t)(rowq * iq) > step;
}

}  // namespace

#define QG_TRY(expr)                                \
    do {                                            \
        const qgemm_status st_ = (expr);            \
        if (st_ != QGEMM_OK) return st_;            \
    } while (0)

// What the two row quantisers share: types, shapes, the output and its scales.
static qgemm_status check_rows(qgi::RowQuantArgs &a, int64_t T, int64_t H) {
    if (a.dtype != QGEMM_F16 && a.dtype != QGEMM_BF16)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "activations are F16 or BF16 (got %d)", a.dtype);
    if (a.y_dtype != QGEMM_INT8 && a.y_dtype != QGEMM_E4M3 && a.y_dtype != a.dtype)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "Y is INT8, E4M3 or of the activations' type (got %d)", a.y_dtype);
    QG_TRY(check_shape(T, H));
    if (a.y_dtype == QGEMM_E4M3 && H % 32)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "E4M3: H %% 32 != 0 (H = %lld)", (long long)H);
    if (T == 0 || H == 0) return QGEMM_OK;
    const int item = a.y_dtype == a.dtype ? 2 : 1;
    QG_TRY(check_input(a.x, a.ldx, T, 2, "X"));
    QG_TRY(check_output(a.y, a.ldy, T, H, item, "Y"));
    if (a.y_dtype == QGEMM_INT8) {
        QG_TRY(check_output(a.scales, 1, T, 1, 4, "scales"));
    } else if (a.y_dtype == QGEMM_E4M3) {
        QG_TRY(check_output(a.scales, a.lds, T, H / 32, 1, "scales"));
    } else if (a.scales) {
        return fail(QGEMM_ERR_INVALID_ARG, "scales must be NULL for a 16-bit output");
    }
    if (T == 1) a.ldx = a.ld2 = a.ldso = a.ldy = a.lds = 0;      // never stepped
    a.T = (int)T;
    a.H = (int)H;
    return QGEMM_OK;
}

// An output may be an input where every element is written by the thread that has read it: same
// base, same stride.
static qgemm_status check_overlap(const void *out, int64_t ldo, int item, const void *in, int64_t ldi, int64_t T,
                                  int64_t H, const char *what) {
    if (!overlap(out, ldo, H, item, in, ldi, H, 2, T)) return QGEMM_OK;
    if (out == in && ldo == ldi && item == 2) return QGEMM_OK;
    return fail(QGEMM_ERR_INVALID_ARG, "%s overlap", what);
}

static qgemm_status w8a8_impl(const int8_t *A, int64_t lda, const float *sa, const int8_t *W, int64_t ldw,
                              const float *sw, const void *bias, void *C, int64_t ldc, int32_t c_dtype, int64_t M,
                              int64_t N, int64_t K, const qgemm_epilogue *ep, void *stream) {
    int epi = 0;
    if (ep) {
        if ((ep->accumulate != 0 && ep->accumulate != 1) || (ep->relu != 0 && ep->relu != 1))
            return fail(QGEMM_ERR_INVALID_ARG, "epilogue fields must be 0 or 1 (accumulate %d, relu %d)",
                        ep->accumulate, ep->relu);
        epi = (ep->accumulate ? qgi::EPI_ACCUMULATE : 0) | (ep->relu ? qgi::EPI_RELU : 0);
    }
    if (c_dtype != QGEMM_F16 && c_dtype != QGEMM_BF16)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "C is F16 or BF16 (got %d)", c_dtype);
    QG_TRY(check_shape(M, N));
    QG_TRY(check_shape(M, K));
    if (std::max({M, N, K}) > MOST_ROUNDED)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "dimension > %lld", (long long)MOST_ROUNDED);
    if (M == 0 || N == 0) return QGEMM_OK;
    QG_TRY(check_output(C, ldc, M, N, 2, "C"));
    if (bias) QG_TRY(check_input(bias, 0, 1, 2, "bias"));
    if (K > 0) {
        QG_TRY(check_input(A, lda, M, 16, "A"));
        QG_TRY(check_input(W, ldw, N, 16, "W"));
        QG_TRY(check_input(sa, 0, 1, 4, "a_scales"));
        QG_TRY(check_input(sw, 0, 1, 4, "w_scales"));
        if (M == 1) lda = (K + 15) / 16 * 16;                    // never stepped
        if (N == 1) ldw = (K + 15) / 16 * 16;
        if (lda < K || ldw < K)
            return fail(QGEMM_ERR_INVALID_ARG, "lda %lld or ldw %lld < K %lld", (long long)lda, (long long)ldw,
                        (long long)K);
        if (lda % 16 || ldw % 16) return fail(QGEMM_ERR_MISALIGNED, "row strides of A and W must be multiples of 16 bytes");
        // TMA strides are below 2^40 bytes
        if (lda >= (int64_t(1) << 40) || ldw >= (int64_t(1) << 40))
            return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "row stride >= 2^40 bytes");
    }
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    ctx.epi = epi;
    const qgi::W8A8Args a{A, W, lda, ldw, sa, sw, bias, C, M == 1 ? N : ldc, c_dtype == QGEMM_BF16, (int)M, (int)N, (int)K};
    if (K == 0) {
        const cudaError_t e = qgi::launch_w8a8_empty(a, ctx);
        return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_w8a8 launch");
    }
    bool enc = true;
    const cudaError_t e = qgi::launch_w8a8(a, ctx, &enc);
    if (!enc) return QGEMM_ERR_CUDA;
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_w8a8 launch");
}

extern "C" {

qgemm_status qgemm_norm_quant(const void *X, int64_t ldx, const void *residual, int64_t ldr, void *residual_out,
                              int64_t ldro, int32_t dtype, const void *weight, int32_t weight_dtype, double eps,
                              int64_t T, int64_t H, void *Y, int64_t ldy, int32_t y_dtype, void *scales, int64_t lds,
                              void *stream) {
    qgi::RowQuantArgs a{};
    a.x = X, a.ldx = ldx, a.second = residual, a.ld2 = ldr, a.sum_out = residual_out, a.ldso = ldro;
    a.weight = weight, a.weight_dtype = weight_dtype, a.y = Y, a.ldy = ldy, a.scales = scales, a.lds = lds;
    a.dtype = dtype, a.y_dtype = y_dtype, a.norm = 1, a.eps = (float)eps;
    if (!std::isfinite(eps) || !std::isfinite(a.eps) || eps < 0x1p-64)
        return fail(QGEMM_ERR_INVALID_ARG, "eps must be finite and at least 2^-64");
    if (weight && weight_dtype != QGEMM_F16 && weight_dtype != QGEMM_BF16 && weight_dtype != QGEMM_F32)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "weights are F16, BF16 or F32 (got %d)", weight_dtype);
    if (residual_out && !residual) return fail(QGEMM_ERR_INVALID_ARG, "residual_out without a residual");
    QG_TRY(check_rows(a, T, H));
    if (T == 0 || H == 0) return QGEMM_OK;
    if (weight) QG_TRY(check_input(weight, 0, 1, weight_dtype == QGEMM_F32 ? 4 : 2, "weight"));
    if (residual) QG_TRY(check_input(residual, ldr, T, 2, "residual"));
    const int yi = y_dtype == dtype ? 2 : 1;
    if (residual_out) {
        QG_TRY(check_output(residual_out, ldro, T, H, 2, "residual_out"));
        QG_TRY(check_overlap(residual_out, a.ldso, 2, X, a.ldx, T, H, "residual_out and X"));
        QG_TRY(check_overlap(residual_out, a.ldso, 2, residual, a.ld2, T, H, "residual_out and residual"));
        if (overlap(residual_out, a.ldso, H, 2, Y, a.ldy, H, yi, T))
            return fail(QGEMM_ERR_INVALID_ARG, "residual_out and Y overlap");
    }
    QG_TRY(check_overlap(Y, a.ldy, yi, X, a.ldx, T, H, "Y and X"));
    if (residual) QG_TRY(check_overlap(Y, a.ldy, yi, residual, a.ld2, T, H, "Y and residual"));
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_row_quant(a, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_norm_quant launch");
}

qgemm_status qgemm_act_quant(const void *X, int64_t ldx, const void *up, int64_t ldu, int32_t dtype,
                             int32_t activation, int64_t T, int64_t H, void *Y, int64_t ldy, int32_t y_dtype,
                             void *scales, int64_t lds, void *stream) {
    qgi::RowQuantArgs a{};
    a.x = X, a.ldx = ldx, a.second = up, a.ld2 = ldu, a.y = Y, a.ldy = ldy, a.scales = scales, a.lds = lds;
    a.dtype = dtype, a.y_dtype = y_dtype, a.activation = activation;
    if (activation < QGEMM_ACT_NONE || activation > QGEMM_ACT_GELU)
        return fail(QGEMM_ERR_INVALID_ARG, "unknown activation %d", activation);
    QG_TRY(check_rows(a, T, H));
    if (T == 0 || H == 0) return QGEMM_OK;
    const int yi = y_dtype == dtype ? 2 : 1;
    QG_TRY(check_overlap(Y, a.ldy, yi, X, a.ldx, T, H, "Y and X"));
    if (up) {
        QG_TRY(check_input(up, ldu, T, 2, "up"));
        QG_TRY(check_overlap(Y, a.ldy, yi, up, a.ld2, T, H, "Y and up"));
    }
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_row_quant(a, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_act_quant launch");
}

qgemm_status qgemm_w8a8(const int8_t *A, int64_t lda, const float *a_scales, const int8_t *W, int64_t ldw,
                        const float *w_scales, const void *bias, void *C, int64_t ldc, int32_t c_dtype, int64_t M,
                        int64_t N, int64_t K, void *stream) {
    return w8a8_impl(A, lda, a_scales, W, ldw, w_scales, bias, C, ldc, c_dtype, M, N, K, nullptr, stream);
}

qgemm_status qgemm_w8a8_ex(const int8_t *A, int64_t lda, const float *a_scales, const int8_t *W, int64_t ldw,
                           const float *w_scales, const void *bias, void *C, int64_t ldc, int32_t c_dtype, int64_t M,
                           int64_t N, int64_t K, const qgemm_epilogue *epilogue, void *stream) {
    return w8a8_impl(A, lda, a_scales, W, ldw, w_scales, bias, C, ldc, c_dtype, M, N, K, epilogue, stream);
}

}  // extern "C"
