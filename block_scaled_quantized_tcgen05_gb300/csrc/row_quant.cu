// row_quant.cu -- rows of a model's activations to 8 bits with scales, in one pass over the row: the
// root-mean-square norm (after the residual's addition) and the (gated) activation.
//
//   norm   h = x + r,  y = h / sqrt(mean h^2 + eps) * w
//   act    y = f(x) [* up]
//   INT8   q = rne(y * 127 / a), s = a / 127, a = max(max |y|, 2^-100)
//   E4M3   X = floor(log2(amax of 32)) - 8, q = e4m3_rn(y 2^-X) saturated, byte X + 127
//
// Bound by memory: a row is read once and written once.  All arithmetic is fp32; h and y are rounded
// only where they are stored.
#include <cfloat>

#include "kv_common.cuh"
#include "linear8_internal.h"

namespace {

using namespace qg;

constexpr float LEAST = 0x1p-100f;      // the least magnitude an INT8 row's scale is taken from
constexpr float SHRINK = 0x1p-80f;      // factor on h where the sum of squares passed fp32's range

enum Out { OUT_INT8, OUT_E4M3, OUT_16 };

// The larger of two magnitudes; NaN where either is (an INT8 row that holds one says so in its scale).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// f(x) = x / (1 + exp(-v)), v = x (SiLU) or 2 sqrt(2/pi) (x + 0.044715 x^3) (GELU: (1 + tanh u) / 2 is
// 1 / (1 + exp(-2 u))).  The exponential is taken of -|v|, so that it never overflows and results go down to the
// type's end.
__device__ __forceinline__ float activate(float x, int kind) {
    if (kind == QGEMM_ACT_NONE) return x;
    const float v = kind == QGEMM_ACT_SILU ? x : 1.5957691216057308f * (x + 0.044715f * x * x * x);
    const float t = __expf(-fabsf(v));
    return __fdividef(v < 0.0f ? x * t : x, 1.0f + t);
}

__device__ __forceinline__ float to_f32(const void *p, int64_t i, int32_t dtype) {
    if (dtype == QGEMM_F32) return static_cast<const float *>(p)[i];
    if (dtype == QGEMM_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// One INT8 code.  inv is 0 for a row with an infinity and NaN for one with a NaN: every code is then 0.
__device__ __forceinline__ int code_i8(float y, float inv) {
    return min(127, max(-127, __float2int_rn(y * inv)));
}

// UE8M0 byte of a block whose largest magnitude is amax, and 2^-X.
__device__ __forceinline__ uint32_t block_scale(float amax, float *inv) {
    // floor(log2) is the exponent field; fp32 subnormals (field 0) are below every X that is kept
    int X = int(__float_as_uint(amax) >> 23) - 127 - 8;
    X = amax > 0.0f ? max(X, -127) : 0;
    *inv = __uint_as_float(uint32_t(127 - X) << 23);               // X in [-127, 120]
    return uint32_t(X + 127);
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Sum of ss and maximum of amax over the block's warps; every thread gets both.
__device__ __forceinline__ void block_reduce(float &ss, float &amax, float2 *room) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (warps == 1) return;
    __syncthreads();                       // the last use of `room` has been read
    if (lane == 0) room[warp] = make_float2(ss, amax);
    __syncthreads();
    const float2 v = lane < warps ? room[lane] : make_float2(0.0f, 0.0f);
    ss = v.x;
    amax = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    }
}

// Any alignment, any H: one block a row, element by element, read a second time (from the caches) once
// the row's sum and maximum are known.  Every element is read and written by one thread, so an output
// may be an input.
template <class TY, int OUT>
__global__ void __launch_bounds__(256) row_quant_any_kernel(const __grid_constant__ qgi::RowQuantArgs a) {
    using T = typename TY::T;
    __shared__ float2 room[8];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        const T *second = static_cast<const T *>(a.second) + (a.second ? row * a.ld2 : 0);
        auto input = [&](int c) {          // h, or the activation's product
            float v = static_cast<float>(x[c]);
            if (a.norm) return a.second ? v + static_cast<float>(second[c]) : v;
            v = activate(v, a.activation);
            return a.second ? v * static_cast<float>(second[c]) : v;
        };
        auto weight = [&](int c) { return a.norm && a.weight ? to_f32(a.weight, c, a.weight_dtype) : 1.0f; };
        float f = 1.0f, r = 1.0f, ss = 0.0f, amax = 0.0f;
        if (a.norm || OUT == OUT_INT8) {
            for (int c = threadIdx.x; c < a.H; c += 256) {
                const float v = input(c);
                ss += v * v;
                amax = max_nan(amax, fabsf(v * weight(c)));
            }
            block_reduce(ss, amax, room);
            if (a.norm) {
                const bool wide = !(ss <= FLT_MAX);
                if (wide) {
                    f = SHRINK;
                    ss = 0.0f;
                    for (int c = threadIdx.x; c < a.H; c += 256) {
                        const float v = input(c) * f;
                        ss += v * v;
                    }
                    float unused = 0.0f;
                    block_reduce(ss, unused, room);
                }
                r = rsqrtf(ss / static_cast<float>(a.H) + (wide ? 0.0f : a.eps));
                if (OUT == OUT_INT8 && (wide || !(amax <= FLT_MAX))) {
                    amax = 0.0f;
                    for (int c = threadIdx.x; c < a.H; c += 256)
                        amax = max_nan(amax, fabsf(input(c) * f * r * weight(c)));
                    float unused = 0.0f;
                    block_reduce(unused, amax, room);
                } else {
                    amax *= r;
                }
            }
        }
        const float most = max_nan(amax, LEAST);
        const float inv8 = 127.0f / most;
        for (int c0 = threadIdx.x - lane; c0 < a.H; c0 += 256) {
            const int c = c0 + lane;
            const bool in = c < a.H;
            const float v = in ? input(c) : 0.0f;
            if (in && a.sum_out) {
                T *so = static_cast<T *>(a.sum_out) + row * a.ldso;
                const uint32_t p = TY::pack(v, 0.0f);
                reinterpret_cast<uint16_t *>(so)[c] = static_cast<uint16_t>(p);
            }
            const float y = in ? (a.norm ? v * f * r * weight(c) : v) : 0.0f;
            if constexpr (OUT == OUT_INT8) {
                if (in) (static_cast<int8_t *>(a.y) + row * a.ldy)[c] = static_cast<int8_t>(code_i8(y, inv8));
            } else if constexpr (OUT == OUT_E4M3) {
                float m = fabsf(y);        // a block of 32 is a warp's; fmaxf passes over NaN
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                float inv;
                const uint32_t byte = block_scale(fmaxf(m, 0.0f), &inv);
                if (in) (static_cast<uint8_t *>(a.y) + row * a.ldy)[c] = static_cast<uint8_t>(e4m3x2(y * inv, 0.0f));
                if (lane == 0) (static_cast<uint8_t *>(a.scales) + row * a.lds)[c / 32] = static_cast<uint8_t>(byte);
            } else {
                if (in) {
                    T *yo = static_cast<T *>(a.y) + row * a.ldy;
                    reinterpret_cast<uint16_t *>(yo)[c] = static_cast<uint16_t>(TY::pack(y, 0.0f));
                }
            }
        }
        if (OUT == OUT_INT8 && threadIdx.x == 0) static_cast<float *>(a.scales)[row] = most / 127.0f;
    }
}

template <class TY>
cudaError_t launch_type(const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    const dim3 grid(static_cast<unsigned>(a.T < 16 * ctx.num_sms ? a.T : 16 * ctx.num_sms));
    auto kern = a.y_dtype == QGEMM_INT8   ? row_quant_any_kernel<TY, OUT_INT8>
                : a.y_dtype == QGEMM_E4M3 ? row_quant_any_kernel<TY, OUT_E4M3>
                                          : row_quant_any_kernel<TY, OUT_16>;
    return launch_dependent(kern, grid, 256, 0, ctx.stream, a);
}

}  // namespace

namespace qgi {

cudaError_t launch_row_quant(const RowQuantArgs &a, const LaunchCtx &ctx) {
    return a.dtype == QGEMM_BF16 ? launch_type<qg::TypeBF16>(a, ctx) : launch_type<qg::TypeF16>(a, ctx);
}

}  // namespace qgi
