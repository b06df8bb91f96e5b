// w8a8.cu -- the integer product's choice of kernel, and its form without products.
#include "w8a8_common.cuh"

namespace {

using namespace qg;

__global__ void __launch_bounds__(256) w8a8_empty_kernel(const __grid_constant__ qgi::W8A8Args a, int epi) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t total = static_cast<int64_t>(a.M) * a.N;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < total; i += gridDim.x * int64_t(256)) {
        const int64_t m = i / a.N, n = i - m * a.N;
        uint16_t *c = static_cast<uint16_t *>(a.C) + m * a.ldc + n;
        const float bias = a.bias ? load_16(a.bias, n, a.bf16) : 0.0f;
        *c = round_16(finish(0.0f, 0.0f, 0.0f, bias, epi & qgi::EPI_ACCUMULATE ? load_16(c, 0, a.bf16) : 0.0f, epi), a.bf16);
    }
}

}  // namespace

namespace qgi {

// Up to 16 tokens the weights' bytes bound the product and the weight stream is the fastest everywhere.  Up to 32 its
// products on mma.sync begin to: it is still ahead of the pairs' three launches on small matrices (32 tokens, 4096 x 4096: 11.1 us
// against 13.5, 5120 x 5120 14.2 against 15.0, 8192 x 4096 15.9 against 16.0; 8192 x 8192 24.4 against 20.9).
// Up to 64 where the launches are most of the time and few blocks of rows keep the tokens' rows from being read often (40
// tokens, 2048 x 2048: 7.7 us against 9.9, 1024 x 1024 5.2 against 7.6; 64 tokens 8.7 against 10.4, 7.2 against 7.7; 4096 x 1024 9.2
// against 8.2).  Of 13 matrices that the rule takes, at 33 to 64 tokens, the stream is ahead by 1 to 33 %, but for 1536 x 2560 at 56
// and 64 tokens (9.9 us against 9.7, 10.3 against 9.8) and 512 x 8192 at 64 (even); no bound on sizes tells them from their neighbours.
static bool few_tokens(const W8A8Args &a) {
    const int64_t weights = int64_t(a.N) * a.K;
    return a.M <= 16 || (a.M <= 32 && weights <= int64_t(1) << 25) ||
           (a.M <= 64 && a.N <= 2048 && weights <= int64_t(1) << 22);
}

cudaError_t launch_w8a8(const W8A8Args &a, const LaunchCtx &ctx, bool *encode_ok) {
    return few_tokens(a) ? launch_w8a8_decode(a, ctx, encode_ok) : launch_w8a8_pair(a, ctx, encode_ok);
}

cudaError_t launch_w8a8_empty(const W8A8Args &a, const LaunchCtx &ctx) {
    const int64_t total = static_cast<int64_t>(a.M) * a.N, blocks = (total + 255) / 256;
    const int64_t most = 16 * static_cast<int64_t>(ctx.num_sms);
    return qg::launch_dependent(w8a8_empty_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0,
                                ctx.stream, a, ctx.epi);
}

}  // namespace qgi
