// linear8_internal.h -- host-side internals of the 8-bit linear layers: arguments of the row
// quantisers and of the integer product, shared by the entry points and the kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "qgemm_internal.h"

namespace qgi {

// One call of a row quantiser (already validated).  Strides in elements, lds in bytes.
struct RowQuantArgs {
    const void *x;
    int64_t ldx;
    const void *second;       // residual or up; NULL: none
    int64_t ld2;
    void *sum_out;            // x + residual, rounded; NULL: not stored
    int64_t ldso;
    const void *weight;       // norm only; NULL: ones
    int32_t weight_dtype;
    void *y;
    int64_t ldy;
    void *scales;
    int64_t lds;
    int32_t dtype, y_dtype;
    int32_t norm;             // 1: norm, 0: activation
    int32_t activation;
    float eps;
    int T, H;
};
cudaError_t launch_row_quant(const RowQuantArgs &a, const LaunchCtx &ctx);

// One integer product (already validated; M, N, K > 0).
struct W8A8Args {
    const int8_t *A, *W;
    int64_t lda, ldw;         // bytes
    const float *sa, *sw;
    const void *bias;         // of C's type; NULL: none
    void *C;
    int64_t ldc;
    int32_t bf16;             // C's type
    int M, N, K;
};
cudaError_t launch_w8a8(const W8A8Args &a, const LaunchCtx &ctx, bool *encode_ok);
// At most 64 tokens: a weight stream (w8a8_decode.cu).
cudaError_t launch_w8a8_decode(const W8A8Args &a, const LaunchCtx &ctx, bool *encode_ok);
// On CTA pairs: any shape (w8a8_pair.cu).
cudaError_t launch_w8a8_pair(const W8A8Args &a, const LaunchCtx &ctx, bool *encode_ok);
// K = 0: C = relu?(bias [+ C_old]).
cudaError_t launch_w8a8_empty(const W8A8Args &a, const LaunchCtx &ctx);

}  // namespace qgi
