// row_quant.cuh -- rows of a model's activations to 8 bits with scales, in one pass over the row: the
// root-mean-square norm (after the residual's addition) and the (gated) activation.
//
//   norm   h = x + r,  y = h / sqrt(mean h^2 + eps) * w
//   act    y = f(x) [* up]
//   INT8   q = rne(y * 127 / a), s = a / 127, a = max(max |y|, 2^-100)
//   E4M3   X = floor(log2(amax of 32)) - 8, q = e4m3_rn(y 2^-X) saturated, byte X + 127
//
// Bound by memory: a row is read once and written once.  All arithmetic is fp32; h and y are rounded
// only where they are stored.
//
// An INT8 row's scale needs the maximum of |y| and y needs the row's sum of squares; y is h w times a
// factor of the row, so max |h w| is taken beside the sum and both travel through one exchange.
#pragma once

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

// The vector kernel's shape: a row held by a warp (WARP, eight rows a block) or by a block, 8 elements a
// thread and chunk, chunk i of thread t at element 8 (i nt + t).
template <class TY>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = TY::unpack(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

template <class TY>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(TY::pack(f[0], f[1]), TY::pack(f[2], f[3]), TY::pack(f[4], f[5]), TY::pack(f[6], f[7]));
}

__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void load_weight8(const qgi::RowQuantArgs &a, int e, float (&w)[8]) {
    if (!a.weight) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    } else if (a.weight_dtype == QGEMM_F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.weight) + e);
        const float4 u = __ldg(p), v = __ldg(p + 1);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
    } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.weight) + e));
        if (a.weight_dtype == QGEMM_F16) unpack8<TypeF16>(v, w);
        else unpack8<TypeBF16>(v, w);
    }
}

template <class TY, int OUT, bool NORM, bool SECOND, int C, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) row_quant_vec_kernel(const __grid_constant__ qgi::RowQuantArgs a) {
    __shared__ float2 room[32];
    griddep_launch_dependents();
    griddep_wait();
    const int nt = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = WARP ? blockIdx.x * int64_t(8) + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= a.T) return;                                // whole warps
    auto join = [&](float &ss, float &amax) {
        if constexpr (WARP) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            }
        } else {
            block_reduce(ss, amax, room);
        }
    };
    const uint16_t *px = static_cast<const uint16_t *>(a.x) + row * a.ldx;
    const uint16_t *p2 = static_cast<const uint16_t *>(a.second) + (SECOND ? row * a.ld2 : 0);
    uint4 xv[C], sv[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = 8 * (i * nt + t);
        const bool in = e < a.H;
        xv[i] = in ? load_once(px + e) : make_uint4(0, 0, 0, 0);
        if (SECOND) sv[i] = in ? load_once(p2 + e) : make_uint4(0, 0, 0, 0);
    }
    auto input = [&](int i, float (&v)[8]) {                       // h, or the activation's product
        unpack8<TY>(xv[i], v);
        float s[8];
        if (SECOND) unpack8<TY>(sv[i], s);
        if constexpr (NORM) {
            if (SECOND)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += s[j];
        } else {
            if (a.activation != QGEMM_ACT_NONE)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = activate(v[j], a.activation);
            if (SECOND)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= s[j];
        }
    };
    float f = 1.0f, r = 1.0f, ss = 0.0f, amax = 0.0f;
    float keep[NORM ? 1 : C][8];                                   // the activation is computed once
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = 8 * (i * nt + t);
            if (e >= a.H) continue;
            float v[8], w[8];
            input(i, v);
            load_weight8(a, e, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(v[j], v[j], ss);
                amax = max_nan(amax, fabsf(v[j] * w[j]));
            }
        }
        join(ss, amax);
        const bool wide = !(ss <= FLT_MAX);
        if (wide) {                                                // rare: the sum again of h * 2^-80
            f = SHRINK;
            ss = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float v[8];
                input(i, v);                                       // zeros past the row's end
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[j] * f, v[j] * f, ss);
            }
            float unused = 0.0f;
            join(ss, unused);
        }
        r = rsqrtf(ss / static_cast<float>(a.H) + (wide ? 0.0f : a.eps));
        if (OUT == OUT_INT8 && (wide || !(amax <= FLT_MAX))) {
            amax = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int e = 8 * (i * nt + t);
                if (e >= a.H) continue;
                float v[8], w[8];
                input(i, v);
                load_weight8(a, e, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(v[j] * f * r * w[j]));
            }
            float unused = 0.0f;
            join(unused, amax);
        } else {
            amax *= r;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            input(i, keep[i]);
            if (OUT == OUT_INT8)
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(keep[i][j]));
        }
        if (OUT == OUT_INT8) join(ss, amax);
    }
    const float most = max_nan(amax, LEAST);
    const float inv8 = 127.0f / most;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = 8 * (i * nt + t);
        if (8 * (i * nt + (t & ~31)) >= a.H) continue;             // whole warps
        const bool in = e < a.H;
        float y[8];
        if constexpr (NORM) {
            float w[8];
            input(i, y);
            if (SECOND && a.sum_out && in)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.sum_out) + row * a.ldso + e) = pack8<TY>(y);
            load_weight8(a, in ? e : 0, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = y[j] * f * r * w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = keep[i][j];
        }
        if constexpr (OUT == OUT_INT8) {
            uint32_t q[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int c[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) c[j] = code_i8(y[4 * h + j], inv8);
                q[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
            }
            if (in) *reinterpret_cast<uint2 *>(static_cast<int8_t *>(a.y) + row * a.ldy + e) = make_uint2(q[0], q[1]);
        } else if constexpr (OUT == OUT_E4M3) {
            float m = 0.0f;                                        // fmaxf passes over NaN
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            float inv;
            const uint32_t byte = block_scale(m, &inv);
            uint32_t q[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[h] = uint32_t(e4m3x2(y[4 * h] * inv, y[4 * h + 1] * inv)) |
                       uint32_t(e4m3x2(y[4 * h + 2] * inv, y[4 * h + 3] * inv)) << 16;
            if (in) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.y) + row * a.ldy + e) = make_uint2(q[0], q[1]);
                if ((t & 3) == 0) (static_cast<uint8_t *>(a.scales) + row * a.lds)[e / 32] = static_cast<uint8_t>(byte);
            }
        } else {
            if (in) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.y) + row * a.ldy + e) = pack8<TY>(y);
        }
    }
    if (OUT == OUT_INT8 && t == 0) static_cast<float *>(a.scales)[row] = most / 127.0f;
}

// 16-byte aligned rows of a multiple of 8 elements, 32768 at most (32 a thread).
inline bool vec_rows(const void *p, int64_t ld, int item) {
    return reinterpret_cast<uintptr_t>(p) % (8 * item) == 0 && ld % 8 == 0;
}

inline bool vec_eligible(const qgi::RowQuantArgs &a) {
    return a.H % 8 == 0 && a.H <= 32768 && vec_rows(a.x, a.ldx, 2) && vec_rows(a.second, a.ld2, 2) &&
           vec_rows(a.sum_out, a.ldso, 2) && vec_rows(a.y, a.ldy, a.y_dtype == a.dtype ? 2 : 1) &&
           reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
}

template <class TY, int OUT, bool NORM, bool SECOND>
cudaError_t launch_vec(const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    if (a.H <= 1024) {
        const dim3 grid(static_cast<unsigned>((int64_t(a.T) + 7) / 8));
        return a.H <= 512 ? launch_dependent(row_quant_vec_kernel<TY, OUT, NORM, SECOND, 2, true>, grid, 256, 0, ctx.stream, a)
                          : launch_dependent(row_quant_vec_kernel<TY, OUT, NORM, SECOND, 4, true>, grid, 256, 0, ctx.stream, a);
    }
    const dim3 grid(static_cast<unsigned>(a.T));
    auto threads = [&](int c) { return (a.H / 8 + 32 * c - 1) / (32 * c) * 32; };
    if (threads(2) <= 1024)
        return launch_dependent(row_quant_vec_kernel<TY, OUT, NORM, SECOND, 2, false>, grid, threads(2), 0, ctx.stream, a);
    return launch_dependent(row_quant_vec_kernel<TY, OUT, NORM, SECOND, 4, false>, grid, threads(4), 0, ctx.stream, a);
}

template <class TY, int OUT>
cudaError_t launch_out(const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    if (!vec_eligible(a)) {
        const dim3 grid(static_cast<unsigned>(a.T < 16 * ctx.num_sms ? a.T : 16 * ctx.num_sms));
        return launch_dependent(row_quant_any_kernel<TY, OUT>, grid, 256, 0, ctx.stream, a);
    }
    if (a.norm) return a.second ? launch_vec<TY, OUT, true, true>(a, ctx) : launch_vec<TY, OUT, true, false>(a, ctx);
    return a.second ? launch_vec<TY, OUT, false, true>(a, ctx) : launch_vec<TY, OUT, false, false>(a, ctx);
}

template <class TY>
cudaError_t launch_type(const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    return a.y_dtype == QGEMM_INT8   ? launch_out<TY, OUT_INT8>(a, ctx)
           : a.y_dtype == QGEMM_E4M3 ? launch_out<TY, OUT_E4M3>(a, ctx)
                                     : launch_out<TY, OUT_16>(a, ctx);
}

}  // namespace
