// row_quant_bf16.cu -- the row quantisers' instances for bfloat16 activations.
#include "row_quant.cuh"

namespace qgi {

cudaError_t launch_row_quant_bf16(const RowQuantArgs &a, const LaunchCtx &ctx) { return launch_type<qg::TypeBF16>(a, ctx); }

}  // namespace qgi
