// row_quant_f16.cu -- the row quantisers' instances for fp16 activations, and the choice by type.
#include "row_quant.cuh"

namespace qgi {

cudaError_t launch_row_quant_bf16(const RowQuantArgs &a, const LaunchCtx &ctx);

cudaError_t launch_row_quant(const RowQuantArgs &a, const LaunchCtx &ctx) {
    return a.dtype == QGEMM_BF16 ? launch_row_quant_bf16(a, ctx) : launch_type<qg::TypeF16>(a, ctx);
}

}  // namespace qgi
