// w8a8.cu -- product of 8-bit integers with a scale for each token and each channel.
//
//   C[m, n] = round( (sum_k A[m, k] W[n, k]) * sa[m] * sw[n] [+ bias[n]] [+ C_old] ), then ReLU.
//
// One thread an output, four products an instruction, sums in integers.
#include "kv_common.cuh"
#include "linear8_internal.h"

namespace {

using namespace qg;

template <class TY>
__device__ __forceinline__ void finish(const qgi::W8A8Args &a, int epi, int m, int n, float sum) {
    using T = typename TY::T;
    float x = a.K > 0 ? sum * a.sa[m] * a.sw[n] : 0.0f;
    if (a.bias) x += static_cast<float>(static_cast<const T *>(a.bias)[n]);
    T *c = static_cast<T *>(a.C) + m * a.ldc + n;
    if (epi & qgi::EPI_ACCUMULATE) x += static_cast<float>(*c);
    if (epi & qgi::EPI_RELU) x = fmaxf(x, 0.0f);
    *reinterpret_cast<uint16_t *>(c) = static_cast<uint16_t>(TY::pack(x, 0.0f));
}

template <class TY>
__global__ void __launch_bounds__(256) w8a8_simple_kernel(const __grid_constant__ qgi::W8A8Args a, int epi) {
    griddep_launch_dependents();
    griddep_wait();
    const int n = blockIdx.x * 16 + (threadIdx.x & 15), m = blockIdx.y * 16 + (threadIdx.x >> 4);
    if (n >= a.N || m >= a.M) return;
    const int8_t *pa = a.A + m * a.lda, *pw = a.W + n * a.ldw;
    float total = 0.0f;
    int k = 0;
    while (k < a.K) {
        const int end = min(a.K - a.K % 16, k + 65536);            // 2^16 products of at most 2^14 stay below 2^31
        int sum = 0;
        for (; k < end; k += 16) {
            const int4 x = __ldg(reinterpret_cast<const int4 *>(pa + k)), y = __ldg(reinterpret_cast<const int4 *>(pw + k));
            sum = __dp4a(x.x, y.x, __dp4a(x.y, y.y, __dp4a(x.z, y.z, __dp4a(x.w, y.w, sum))));
        }
        if (a.K - k < 16)
            for (; k < a.K; ++k) sum += int(pa[k]) * int(pw[k]);
        total += static_cast<float>(sum);
    }
    finish<TY>(a, epi, m, n, total);
}

}  // namespace

namespace qgi {

cudaError_t launch_w8a8(const W8A8Args &a, const LaunchCtx &ctx, bool *encode_ok) {
    *encode_ok = true;
    if (a.K < 0) return cudaErrorInvalidValue;
    const dim3 grid((a.N + 15) / 16, (a.M + 15) / 16);
    return qg::launch_dependent(a.bf16 ? w8a8_simple_kernel<qg::TypeBF16> : w8a8_simple_kernel<qg::TypeF16>, grid, 256,
                                0, ctx.stream, a, ctx.epi);
}

cudaError_t launch_w8a8_empty(const W8A8Args &a, const LaunchCtx &ctx) {
    bool ok;
    return launch_w8a8(a, ctx, &ok);
}

}  // namespace qgi
