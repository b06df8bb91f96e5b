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
// factor of the row, so max |h w| is taken beside the sum and both travel through one exchange, and the codes are those of
// h w itself.
//
// Measured (GB300, whose copies reach 6.76 TB/s): norm with residual of 8192 x 8192 bf16 to E4M3 78.3 us, 6.03 TB/s; gated SiLU of
// 4096 x 14336 fp16 to E4M3 49.7 us, 5.95 TB/s.  Writes beside reads and the rows' exchanges cost what is left.  Without
// a residual the issue slots bound a norm to INT8: 5003 x 5112 22.7 us, 3.4 TB/s (about half of a row's instructions are its exchange's
// and its factor's, whatever its length); rows at any alignment, 5003 x 5111: 27.6 us, their shifts, and past 8192 elements, one
// block of 512 threads an SM, 5003 x 12289: 65 us, 2.8 TB/s.  16 x 14336: 3.0 to 3.4 us.
#pragma once

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "kv_common.cuh"
#include "linear8_internal.h"

namespace {

using namespace qg;

constexpr float LEAST = 0x1p-100f;      // the least magnitude an INT8 row's scale is taken from
constexpr float SHRINK = 0x1p-80f;      // factor on h where the sum of squares, or its mean and eps, passed fp32's range

constexpr int MAX_STAGES = 8;           // of a block's ring
constexpr int LONGEST = 1 << 15;        // elements of a row that a block's registers hold

enum Out { OUT_INT8, OUT_E4M3, OUT_16 };

// The larger of two magnitudes; NaN where either is (an INT8 row that holds one says so in its scale).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest of a magnitude and of two values' magnitudes; NaN where one is (max_nan) or passing over NaN (max_num).
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_num(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two products at once, each rounded as its scalar counterpart.
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// f(x) = x / (1 + exp(-v)), v = x (SiLU) or 2 sqrt(2/pi) (x + 0.044715 x^3) (GELU: (1 + tanh u) / 2 is
// 1 / (1 + exp(-2 u))).  The exponential is taken of -|v|, so that it never overflows, as the square of t = exp(-|v| / 2), so that
// it stays normal where f is: below 0 the numerator is x t t.  Two values at once.
__device__ __forceinline__ void activate2(float &x0, float &x1, int kind) {
    float v0 = x0, v1 = x1;
    if (kind == QGEMM_ACT_GELU) {
        float s0, s1;
        mul2(s0, s1, x0, x1, x0, x1);
        fma2(s0, s1, s0, s1, 0.0713548162726f, 0.0713548162726f, 1.5957691216057308f, 1.5957691216057308f);
        mul2(v0, v1, x0, x1, s0, s1);
    }
    float t0, t1, r0, r1, n0, n1, d0, d1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(fabsf(v0) * -0.7213475204444817f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(fabsf(v1) * -0.7213475204444817f));
    fma2(d0, d1, t0, t1, t0, t1, 1.0f, 1.0f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));          // of 1 .. 2
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
    mul2(n0, n1, x0, x1, t0, t1);
    mul2(n0, n1, n0, n1, t0, t1);
    mul2(x0, x1, v0 < 0.0f ? n0 : x0, v1 < 0.0f ? n1 : x1, r0, r1);
}

__device__ __forceinline__ float to_f32(const void *p, int64_t i, int32_t dtype) {
    if (dtype == QGEMM_F32) return static_cast<const float *>(p)[i];
    if (dtype == QGEMM_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// 127 / a as a pair: values half-way between codes are common (half of the row's largest is one, in a row as it is, in a norm's
// h w, in a product of two operands), and a factor rounded to 32 bits moves them to either side.  One part alone saves 4 to 8 %
// where issue slots are the bound (norm without residual, 5003 x 5112: 20.6 us against 22.1; gated SiLU, 4096 x 12288: 41.4 against
// 45.0) and 0 to 2 % elsewhere; it is taken for a gated SiLU or GELU only, whose values carry errors of their own.
struct Factor {
    float hi, lo;
    bool finite;                           // a row with an infinity or a NaN has no factor: every code is 0 there
    __device__ __forceinline__ explicit Factor(float a) : hi(127.0f / a), finite(a <= FLT_MAX) {
        lo = fmaf(-hi, a, 127.0f) * (hi * (1.0f / 127.0f));
    }
};

// Whether a norm's codes can be those of h w, whose largest magnitude is `most`: the row's factor r changes no code, and
// takes two roundings with it.  Not where the scale has its least value or none (y passes fp32's range), or h w may be below
// fp32's normal range (or NaN).
__device__ __forceinline__ bool codes_without_r(float most, float most_y) {
    return most <= FLT_MAX && most >= LEAST && most_y <= FLT_MAX && most_y >= LEAST;
}

// Four INT8 codes of y times the factor (PAIR: both parts of it), at most 127 in magnitude: 1.5 * 2^23 added leaves the
// nearest integer (ties to even) in the low bits.
template <bool PAIR>
__device__ __forceinline__ uint32_t codes_i8(const float *y, const Factor &f) {
    constexpr float HALF_WAY = 12582912.0f;
    float c[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        if constexpr (PAIR) {
            mul2(c[j], c[j + 1], y[j], y[j + 1], f.lo, f.lo);
            fma2(c[j], c[j + 1], y[j], y[j + 1], f.hi, f.hi, c[j], c[j + 1]);
            add2(c[j], c[j + 1], HALF_WAY, HALF_WAY);
        } else {
            fma2(c[j], c[j + 1], y[j], y[j + 1], f.hi, f.hi, HALF_WAY, HALF_WAY);
        }
    }
    const uint32_t q = __byte_perm(__byte_perm(__float_as_uint(c[0]), __float_as_uint(c[1]), 0x0040),
                                   __byte_perm(__float_as_uint(c[2]), __float_as_uint(c[3]), 0x0040), 0x5410);
    return f.finite ? q : 0u;
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

// The first n of 8 elements, the rest 0: a row's end, out of the common path.
__device__ __noinline__ uint4 first_of(uint4 v, int n) {
    uint32_t o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (2 * i + 1 >= n) o[i] = 2 * i >= n ? 0u : o[i] & 0xFFFFu;
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Elements 0 .. n - 1 of 16 bits from byte `off` of two 16-byte pieces on, the rest 0.
__device__ __forceinline__ uint4 shifted(const uint4 &lo, const uint4 &hi, uint32_t off, int n) {
    uint32_t w[5];
    switch (off >> 2) {
    case 0: w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x; break;
    case 1: w[0] = lo.y, w[1] = lo.z, w[2] = lo.w, w[3] = hi.x, w[4] = hi.y; break;
    case 2: w[0] = lo.z, w[1] = lo.w, w[2] = hi.x, w[3] = hi.y, w[4] = hi.z; break;
    default: w[0] = lo.w, w[1] = hi.x, w[2] = hi.y, w[3] = hi.z, w[4] = hi.w; break;
    }
    const uint32_t bits = 8 * (off & 2);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[i], w[i + 1], bits);
    const uint4 all = make_uint4(o[0], o[1], o[2], o[3]);
    return n < 8 ? first_of(all, n) : all;
}

// Elements 0 .. n - 1 of 16 bits at an address of any alignment, the rest 0: the aligned 16-byte pieces that hold
// them, shifted together.  No piece without one of the elements is read.  Pieces are read `off` bytes before the elements,
// the same for a whole row.
__device__ __forceinline__ uint4 load_any(const uint16_t *p, uint32_t off, int n) {
    const uint4 *piece = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(p) - off);
    if (off == 0 && n >= 8) return load_once(piece);
    const uint4 lo = load_once(piece);
    uint4 hi = make_uint4(0, 0, 0, 0);
    if (n > 8 - static_cast<int>(off) / 2) hi = load_once(piece + 1);        // (a row's bytes may pass 32 bits)
    return shifted(lo, hi, off, n);
}

// The same from a stage of the ring, `p` the element's place without the offset.
__device__ __forceinline__ uint4 shared_any(const uint8_t *p, uint32_t off, int n) {
    if (off == 0 && n >= 8) return *reinterpret_cast<const uint4 *>(p);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p + (off & 12));
    const uint32_t bits = 8 * (off & 2);
    const uint4 all = make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                                 __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    return n < 8 ? first_of(all, n) : all;
}

__device__ __forceinline__ uint32_t before_16(const void *p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15); }

// Debug build: n elements of `item` bytes at p, or fewer where n is more than the 8 of a thread, lie in the T rows of H elements at
// `base`.
__device__ __forceinline__ bool in_rows([[maybe_unused]] unsigned *err, const qgi::RowQuantArgs &a, const void *p, int n, int item,
                                        const void *base, int64_t ld) {
    return QG_IN_RANGE(err, p, min(n, 8) * item, base, ((a.T - 1) * ld + a.H) * item);
}

// Weights of elements e .. e + 7 (0 past the row's end).
template <bool ANY>
__device__ __forceinline__ void load_weight8(const qgi::RowQuantArgs &a, int e, float (&w)[8], unsigned *err) {
    if (!a.weight || !QG_IN_BOUNDS(err, e >= 0 && e < a.H && (ANY || a.H - e >= 8))) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    } else if (ANY && (a.H - e < 8 || before_16(a.weight) != 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < a.H - e ? to_f32(a.weight, int64_t(e) + i, a.weight_dtype) : 0.0f;
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

// Eight 16-bit or 8-bit elements, or the first n of them, at an address of any alignment.
__device__ __noinline__ void store_parts(uint16_t *p, uint4 v, int n) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
}
__device__ __noinline__ void store_parts(uint8_t *p, uint2 v, int n) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i & 3)));
}
__device__ __forceinline__ void store_any(uint16_t *p, const uint4 &v, int n) {
    if (n >= 8 && reinterpret_cast<uintptr_t>(p) % 16 == 0) *reinterpret_cast<uint4 *>(p) = v;
    else store_parts(p, v, n);
}
__device__ __forceinline__ void store_any(uint8_t *p, const uint2 &v, int n) {
    if (n >= 8 && reinterpret_cast<uintptr_t>(p) % 8 == 0) *reinterpret_cast<uint2 *>(p) = v;
    else store_parts(p, v, n);
}

// A warp's consecutive eights of 16-bit elements at an address of any alignment, n of them before the row's end (any number,
// 0 and less too; whole warps): each lane writes the aligned 16 bytes that its elements end with its neighbour's, the first
// and the last lane what is over at the ends.
__device__ __forceinline__ void store_warp(uint16_t *p, const uint4 &v, int n) {
    const uint32_t off = before_16(p);           // the same in all lanes
    const int lane = threadIdx.x & 31;
    if (off == 0) {
        if (n > 0) store_any(p, v, n);
        return;
    }
    uint4 before;
    before.x = __shfl_up_sync(0xFFFFFFFFu, v.x, 1);
    before.y = __shfl_up_sync(0xFFFFFFFFu, v.y, 1);
    before.z = __shfl_up_sync(0xFFFFFFFFu, v.z, 1);
    before.w = __shfl_up_sync(0xFFFFFFFFu, v.w, 1);
    const int over = static_cast<int>(off) / 2;  // elements of the neighbour's in this lane's 16 bytes
    if (lane == 0) {
        if (n > 0) store_parts(p, v, min(n, 8 - over));
    } else {
        const uint4 w = shifted(before, v, 16 - off, 8);
        if (n + over >= 8) *reinterpret_cast<uint4 *>(p - over) = w;
        else if (n + over > 0) store_parts(p - over, w, n + over);
    }
    if (lane == 31 && n > 8 - over) store_parts(p + 8 - over, shifted(v, v, 16 - off, 8), min(n, 8) - (8 - over));
}

// Elements e .. e + 7 of a row's y, or the n of them before its end (0 and less too), as the output has them; whole warps.
// PAIR: INT8 codes by both parts of the factor.
template <int OUT, bool ANY, class TY, bool PAIR>
__device__ __forceinline__ void store_row(const qgi::RowQuantArgs &a, int64_t row, uint32_t e, int n, const float (&v)[8],
                                          const Factor &factor, unsigned *err) {
    constexpr int ITEM = OUT == OUT_16 ? 2 : 1;
    if (n > 0 && !in_rows(err, a, static_cast<uint8_t *>(a.y) + (row * a.ldy + e) * ITEM, n, ITEM, a.y, a.ldy)) n = 0;
    if constexpr (OUT == OUT_INT8) {
        uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.ldy + e;
        const uint2 q = make_uint2(codes_i8<PAIR>(v, factor), codes_i8<PAIR>(v + 4, factor));
        if (n > 0) {
            if (ANY) store_any(y, q, n);
            else *reinterpret_cast<uint2 *>(y) = q;
        }
    } else if constexpr (OUT == OUT_E4M3) {
        float m = n > 0 ? 0.0f : 1.0f;         // (lanes past the row's end share no block with others)
        if (n > 0) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) m = max_num(m, v[j], v[j + 1]);
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        float inv;
        const uint32_t byte = block_scale(m, &inv);
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float u[4];
            mul2(u[0], u[1], v[4 * h], v[4 * h + 1], inv, inv);
            mul2(u[2], u[3], v[4 * h + 2], v[4 * h + 3], inv, inv);
            q[h] = uint32_t(e4m3x2(u[0], u[1])) | uint32_t(e4m3x2(u[2], u[3])) << 16;
        }
        if (n > 0) {
            uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.ldy + e;
            if (ANY) store_any(y, make_uint2(q[0], q[1]), n);
            else *reinterpret_cast<uint2 *>(y) = make_uint2(q[0], q[1]);
            if ((threadIdx.x & 3) == 0 && QG_IN_RANGE(err, static_cast<uint8_t *>(a.scales) + row * a.lds + e / 32, 1, a.scales,
                                                      (a.T - 1) * a.lds + a.H / 32))
                (static_cast<uint8_t *>(a.scales) + row * a.lds)[e / 32] = static_cast<uint8_t>(byte);
        }
    } else {
        uint16_t *y = static_cast<uint16_t *>(a.y) + row * a.ldy + e;
        if (ANY) store_warp(y, pack8<TY>(v), n);
        else if (n > 0) *reinterpret_cast<uint4 *>(y) = pack8<TY>(v);
    }
}

// Rows longer than a block holds in registers: one block a row, read a second time (from L2 mostly) once the row's sum and
// maximum are known.  Operands of any alignment.  Every element is read and written by one thread, so an output may be an
// input.  A thread's next pieces are on their way while it works on these.  Gated SiLU to INT8 of 1024 x 65536: 136 us, 16 x 53248:
// 15.3 - 16.8 us; with 512 threads, two blocks an SM, 147 and 18.4 (2048 x 53248: 228 against 212).  Norm with residual to INT8 of 1024 x
// 65536: 145 us.
template <class TY, int OUT>
__global__ void __launch_bounds__(1024) row_quant_long_kernel(const __grid_constant__ qgi::RowQuantArgs a, unsigned *err) {
    __shared__ float2 room[32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t H = a.H, first = 8 * threadIdx.x;               // elements of 32 bits without a sign: H ends near 2^31
    constexpr uint32_t STEP = 8 * 1024;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const uint16_t *x = static_cast<const uint16_t *>(a.x) + row * a.ldx;
        const uint16_t *second = static_cast<const uint16_t *>(a.second) + (a.second ? row * a.ld2 : 0);
        const uint32_t offx = before_16(x), off2 = before_16(second);
        struct Pieces {
            uint4 x, second;
        };
        auto fetch = [&](uint32_t e) {                             // elements e .. e + 7; 0 past the row's end
            Pieces p{};
            const int n = static_cast<int>(H - e);
            if (n > 0) {
                if (in_rows(err, a, x + e, n, 2, a.x, a.ldx)) p.x = load_any(x + e, offx, n);
                if (a.second && in_rows(err, a, second + e, n, 2, a.second, a.ld2)) p.second = load_any(second + e, off2, n);
            }
            return p;
        };
        auto input = [&](const Pieces &p, float (&v)[8]) {         // h, or the activation's product
            float s[8];
            unpack8<TY>(p.x, v);
            unpack8<TY>(p.second, s);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                if (!a.norm && a.activation != QGEMM_ACT_NONE) activate2(v[j], v[j + 1], a.activation);
                if (a.norm) add2(v[j], v[j + 1], s[j], s[j + 1]);
                else if (a.second) mul2(v[j], v[j + 1], v[j], v[j + 1], s[j], s[j + 1]);
            }
        };
        float f = 1.0f, r = 1.0f, ss = 0.0f, amax = 0.0f;
        // Sum of (h f)^2 and maximum of |y| / r, or of |y|
        auto measure = [&](bool scaled) {
            ss = amax = 0.0f;
            Pieces next = fetch(first);
            for (uint32_t e = first; e < H; e += STEP) {
                const Pieces here = next;
                next = fetch(e + STEP);
                float v[8];
                input(here, v);
                if (a.norm) {
                    float w[8], s2[2] = {0.0f, 0.0f};
                    if (OUT == OUT_INT8) load_weight8<true>(a, static_cast<int>(e), w, err);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        mul2(v[j], v[j + 1], v[j], v[j + 1], f, f);
                        fma2(s2[0], s2[1], v[j], v[j + 1], v[j], v[j + 1], s2[0], s2[1]);
                        if (scaled) mul2(v[j], v[j + 1], v[j], v[j + 1], r, r);
                        if (OUT == OUT_INT8) mul2(v[j], v[j + 1], v[j], v[j + 1], w[j], w[j + 1]);
                    }
                    ss += s2[0] + s2[1];
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2) amax = max_nan(amax, v[j], v[j + 1]);
            }
            block_reduce(ss, amax, room);
        };
        if (a.norm || OUT == OUT_INT8) {
            measure(false);
            if (a.norm) {
                const float count = static_cast<float>(a.H);
                const bool wide = !(ss / count + a.eps <= FLT_MAX);
                if (wide) {
                    f = SHRINK;
                    measure(false);
                }
                r = rsqrtf(ss / count + (wide ? a.eps * SHRINK * SHRINK : a.eps));
            }
        }
        float shown = amax * r;                                    // the largest |y|; amax that of what is turned into codes
        if (OUT == OUT_INT8) {
            if (a.norm && f == 1.0f && codes_without_r(amax, shown)) {
                r = 1.0f;
            } else {
                if (a.norm) measure(true);
                shown = amax = max_nan(amax, LEAST);
            }
        }
        const Factor factor(amax);
        Pieces next = fetch(first);
        for (uint32_t e0 = first - 8 * lane; e0 < H; e0 += STEP) {   // whole warps
            const uint32_t e = e0 + 8 * lane;
            const int n = static_cast<int>(H - e);
            const Pieces here = next;
            next = fetch(e + STEP);
            float v[8];
            input(here, v);
            if (a.sum_out) {
                uint16_t *sum = static_cast<uint16_t *>(a.sum_out) + row * a.ldso + e;
                store_warp(sum, pack8<TY>(v), n > 0 && !in_rows(err, a, sum, n, 2, a.sum_out, a.ldso) ? 0 : n);
            }
            if (a.norm && n > 0) {
                float w[8];
                load_weight8<true>(a, static_cast<int>(e), w, err);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    mul2(v[j], v[j + 1], v[j], v[j + 1], f, f);
                    mul2(v[j], v[j + 1], v[j], v[j + 1], r, r);
                    mul2(v[j], v[j + 1], v[j], v[j + 1], w[j], w[j + 1]);
                }
            }
            store_row<OUT, true, TY, true>(a, row, e, n, v, factor, err);
        }
        if (OUT == OUT_INT8 && threadIdx.x == 0 && QG_IN_BOUNDS(err, row < a.T)) static_cast<float *>(a.scales)[row] = shown / 127.0f;
    }
}

__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// The ring of a block in shared memory: rows, or parts of rows where few rows fit (`unit` chunks a stage).
struct Ring {
    int stages;
    uint32_t second_at, stage_bytes;         // where a stage's second operand begins; a stage
    int parts;                               // WARP: parts of a row, where an output needs nothing of the whole row
    int once;                                // the inputs pass through L2 (they do not fit beside what others left there)
};

// Chunks of a stage: a row's, whose place is free once its exchange has shown that all threads have read it; or one, free
// once its warps have said so, where a row of two operands takes half of shared memory and more (2048 x 28672 gated SiLU to INT8: 54 us
// against 70; shorter rows lose 5 to 15 % by the chunks' waits, and so does the long norm, which is short of registers).
template <bool NORM, bool SECOND, int C, bool BIG>
constexpr int unit_of = BIG && !NORM && SECOND ? 1 : C;

// Threads that a block of the ring kernel may have: its launch bound, and what the host chooses by.
constexpr int most_threads(int c, bool any, bool big) { return (c == 2 && !any) || big ? 1024 : 512; }

// A row held by L lanes of a warp (8, 16 or 32; loaded directly) or by a block (L = 0), 8 elements a thread and chunk, chunk i of
// thread t at element 8 (i nt + t).  A block walks its rows with the next ones on their way: bulk copies fill a ring in
// shared memory, so that loads go on through a row's sum, its exchange and its stores.  ANY: rows of any alignment and
// length.  BIG: 1024 threads, which leaves no registers for weights.
template <class TY, int OUT, bool NORM, bool SECOND, int C, int L, bool ANY, bool BIG>
__global__ void __launch_bounds__(L > 0 ? 256 : most_threads(C, ANY, BIG), L == 0 ? 1 : NORM ? 4 : 5)
row_quant_vec_kernel(const __grid_constant__ qgi::RowQuantArgs a, const Ring ring, unsigned *err, uint64_t timeout_ns) {
    constexpr bool WARP = L > 0, MANY = L == 8 || L == 16;         // MANY: rows of a warp side by side
    static_assert(!(MANY && ANY), "stores at any alignment are a warp's");
    __shared__ float2 room[2][32];
    constexpr int UNIT = unit_of<NORM, SECOND, C, BIG>;
    extern __shared__ uint8_t rows_smem[];
    griddep_launch_dependents();
    const int nt = WARP ? L : blockDim.x, t = WARP ? threadIdx.x & (L - 1) : threadIdx.x;
    [[maybe_unused]] const float per_h = 1.0f / static_cast<float>(a.H);
    int turn = 0;
    // Sum of ss and maximum of amax (not negative: its bits' order is its own, a NaN's the largest) over the row's threads; one
    // barrier, as the rooms alternate.  Only what the output needs.
    constexpr bool SUM = NORM, MOST = OUT == OUT_INT8;
    auto join = [&](float &ss, float &amax) {
        auto over = [&](int width) {
            if constexpr (SUM)
                for (int o = width / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            if constexpr (MOST && MANY)
                for (int o = width / 2; o > 0; o >>= 1)
                    amax = __uint_as_float(max(__float_as_uint(amax), __shfl_xor_sync(0xFFFFFFFFu, __float_as_uint(amax), o)));
            else if constexpr (MOST)
                amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax)));
        };
        over(WARP ? L : 32);
        if constexpr (!WARP) {
            const int warps = nt >> 5;
            if ((t & 31) == 0) room[turn][t >> 5] = make_float2(ss, amax);
            // Warps come here from two bodies of `process` at once where a row does not fill its block: the barrier by its number.
            asm volatile("barrier.sync 0;" ::: "memory");
            const float2 v = (t & 31) < warps ? room[turn][t & 31] : make_float2(0.0f, 0.0f);
            turn ^= 1;
            ss = v.x;
            amax = v.y;
            over(ANY ? warps > 16 ? 32 : warps > 8 ? 16 : warps > 4 ? 8 : 4 : 32);
            if constexpr (ANY && SUM) ss = __shfl_sync(0xFFFFFFFFu, ss, 0);
        }
    };
    // Whether any row of the warp takes a path that its lanes go together (a block's rows go alone).
    auto any_row = [](bool b) { return MANY ? __any_sync(0xFFFFFFFFu, b) != 0 : b; };
    auto put_sum = [&](int64_t row, int e, const uint4 &v, int n) {            // ANY: by whole warps
        uint16_t *p = static_cast<uint16_t *>(a.sum_out) + row * a.ldso + e;
        if (n > 0 && !in_rows(err, a, p, n, 2, a.sum_out, a.ldso)) n = 0;
        if constexpr (ANY) store_warp(p, v, n);
        else if (n > 0) *reinterpret_cast<uint4 *>(p) = v;
    };
    auto row_x = [&](int64_t row) { return static_cast<const uint16_t *>(a.x) + row * a.ldx; };
    auto row_2 = [&](int64_t row) { return static_cast<const uint16_t *>(a.second) + row * a.ld2; };

    // A row's weights, kept by the thread where its registers allow (a block's for all its rows).
    constexpr bool KEEP = NORM && !BIG;
    float wkept[KEEP ? C : 1][8];
    auto keep_weights = [&] {
        if constexpr (KEEP)
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (8 * (i * nt + t) < a.H) load_weight8<ANY>(a, 8 * (i * nt + t), wkept[i], err);
    };
    auto weights = [&](int i, int e, float (&w)[8]) {
        if constexpr (KEEP)
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = wkept[i][j];
        else
            load_weight8<ANY>(a, e, w, err);
    };

    // One row: load(i, e, n, xv, sv) gives chunk i's operands, read_done() says that all threads have theirs.  `in`: all of the warp's
    // elements are the row's, which saves the tests (n is the number of elements from e on that are, or at least 8).
    auto process = [&](auto in, int64_t row, int e0, auto &&load, auto &&read_done) {
        constexpr bool IN = decltype(in)::value;
        const int H = MANY && row >= a.T ? 0 : a.H;                // lanes without a row go along
        // h, or the activation's product; zeros past the row's end
        float v[C][8], amax = 0.0f;
        [[maybe_unused]] float shown = 0.0f;                       // the largest |y|; amax that of what is turned into codes
        [[maybe_unused]] float r = 1.0f, ss = 0.0f;
        {
            uint4 xv[C], sv[C];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int e = e0 + 8 * (i * nt + t);
                xv[i] = sv[i] = make_uint4(0, 0, 0, 0);
                load(i, e, IN ? 8 : H - e, xv[i], sv[i]);
            }
            if (!WARP && UNIT == C) fence_proxy_async_smem();      // read here, written next by the bulk copies
            float s2[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < C; ++i) {
                [[maybe_unused]] const int e = e0 + 8 * (i * nt + t);
                unpack8<TY>(xv[i], v[i]);
                float s[8];
                if (SECOND) unpack8<TY>(sv[i], s);
                if constexpr (NORM) {
                    if (SECOND)
#pragma unroll
                        for (int j = 0; j < 8; j += 2) add2(v[i][j], v[i][j + 1], s[j], s[j + 1]);
                    if (!IN && ANY && e - 8 * (t & 31) >= H) continue;  // whole warps
                    if (SECOND && a.sum_out && (IN || ANY || e < H))
                        put_sum(row, e, pack8<TY>(v[i]), IN ? 8 : H - e);
                    if (!IN && e >= H) continue;
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        fma2(s2[0], s2[1], v[i][j], v[i][j + 1], v[i][j], v[i][j + 1], s2[0], s2[1]);
                    if constexpr (OUT == OUT_INT8) {
                        float w[8];
                        weights(i, e, w);
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            float p[2];
                            mul2(p[0], p[1], v[i][j], v[i][j + 1], w[j], w[j + 1]);
                            amax = max_nan(amax, p[0], p[1]);
                        }
                    }
                } else {
                    if (a.activation != QGEMM_ACT_NONE)
#pragma unroll
                        for (int j = 0; j < 8; j += 2) activate2(v[i][j], v[i][j + 1], a.activation);
                    if (SECOND)
#pragma unroll
                        for (int j = 0; j < 8; j += 2) mul2(v[i][j], v[i][j + 1], v[i][j], v[i][j + 1], s[j], s[j + 1]);
                    if (OUT == OUT_INT8)
#pragma unroll
                        for (int j = 0; j < 8; j += 2) amax = max_nan(amax, v[i][j], v[i][j + 1]);
                }
            }
            ss = s2[0] + s2[1];
        }
        if constexpr (NORM) {
            join(ss, amax);
            read_done();
            const bool wide = !(fmaf(ss, per_h, a.eps) <= FLT_MAX);
            if (any_row(wide)) {                                   // rare: the sum again of h * 2^-80
                const float shrink = wide ? SHRINK : 1.0f;
                float again = 0.0f, unused = 0.0f;
#pragma unroll
                for (int i = 0; i < C; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[i][j] *= shrink;
                        again = fmaf(v[i][j], v[i][j], again);
                    }
                join(again, unused);
                if (wide) ss = again;
            }
            r = rsqrtf(fmaf(ss, per_h, wide ? a.eps * SHRINK * SHRINK : a.eps));
            if constexpr (OUT == OUT_INT8) {
                shown = amax * r;
                const bool slow = wide || !codes_without_r(amax, shown);
                if (any_row(slow)) {
                    const float times = slow ? r : 1.0f;
                    float most = 0.0f, unused = 0.0f;
#pragma unroll
                    for (int i = 0; i < C; ++i) {
                        const int e = e0 + 8 * (i * nt + t);
                        if (!IN && e >= H) continue;
                        float w[8];
                        weights(i, e, w);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[i][j] *= times;
#pragma unroll
                        for (int j = 0; j < 8; j += 2) most = max_nan(most, v[i][j] * w[j], v[i][j + 1] * w[j + 1]);
                    }
                    join(unused, most);
                    if (slow) shown = amax = max_nan(most, LEAST);
                }
            }
        } else if constexpr (OUT == OUT_INT8) {
            join(ss, amax);
            read_done();
            shown = amax = max_nan(amax, LEAST);
        } else {
            static_assert(WARP);                                   // nothing of the whole row is needed
        }
        [[maybe_unused]] const Factor factor(amax);
        auto store = [&](auto pair) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int e = e0 + 8 * (i * nt + t);
                if (!IN && e0 + 8 * (i * nt + (t & ~31)) >= a.H) continue;     // whole warps
                if constexpr (NORM) {
                    float w[8];
                    weights(i, IN || e < H ? e : 0, w);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        if (OUT != OUT_INT8) mul2(v[i][j], v[i][j + 1], v[i][j], v[i][j + 1], r, r);
                        mul2(v[i][j], v[i][j + 1], v[i][j], v[i][j + 1], w[j], w[j + 1]);
                    }
                }
                store_row<OUT, ANY, TY, decltype(pair)::value>(a, row, e, IN ? 8 : H - e, v[i], factor, err);
            }
        };
        if (NORM || !SECOND || OUT != OUT_INT8 || a.activation == QGEMM_ACT_NONE) store(std::true_type{});
        else store(std::false_type{});
        if (OUT == OUT_INT8 && t == 0 && (!MANY || H > 0) && QG_IN_BOUNDS(err, row >= 0 && row < a.T))
            static_cast<float *>(a.scales)[row] = shown / 127.0f;
    };

    if constexpr (WARP) {
        griddep_wait();
        const int64_t at = blockIdx.x * int64_t(256 / L) + threadIdx.x / L;
        const int64_t row = MANY || ring.parts == 1 ? at : at / ring.parts;
        const int e0 = MANY || ring.parts == 1 ? 0 : static_cast<int>(at - row * ring.parts) * 8 * L * C;
        if (row - (MANY ? (threadIdx.x & 31) / L : 0) >= a.T) return;                    // whole warps
        keep_weights();
        const uint16_t *px = row_x(row), *p2 = SECOND ? row_2(row) : nullptr;
        const uint32_t offx = ANY ? before_16(px) : 0, off2 = ANY && SECOND ? before_16(p2) : 0;
        auto load = [&](int, int e, int n, uint4 &xv, uint4 &sv) {
            if (n <= 0 || !in_rows(err, a, px + e, n, 2, a.x, a.ldx)) return;
            xv = ANY ? load_any(px + e, offx, n) : load_once(px + e);
            if (SECOND && in_rows(err, a, p2 + e, n, 2, a.second, a.ld2)) sv = ANY ? load_any(p2 + e, off2, n) : load_once(p2 + e);
        };
        const bool all_in = !ANY && a.H - e0 >= 8 * L * C && (!MANY || row + (31 - (threadIdx.x & 31)) / L < a.T);
        if (all_in) process(std::bool_constant<!ANY>{}, row, e0, load, [] {});
        else process(std::false_type{}, row, e0, load, [] {});
    } else {
        __shared__ uint64_t bars[UNIT == 1 ? 2 * MAX_STAGES : MAX_STAGES];
        const uint32_t sb = smem_u32(rows_smem), full0 = smem_u32(bars), empty0 = full0 + 8 * MAX_STAGES;
        if (t == 0) {
            for (int i = 0; i < ring.stages; ++i) {
                mbar_init(full0 + 8 * i, 1);
                if (UNIT == 1) mbar_init(empty0 + 8 * i, nt >> 5);
            }
            fence_barrier_init();
        }
        __syncthreads();
        griddep_wait();
        // By one thread: whole 16-byte pieces that hold a stage's part of a row.
        auto fetch = [&](int64_t row, int part, int stage) {
            const int first = 8 * UNIT * nt * part, n = UNIT == C ? a.H : min(8 * UNIT * nt, a.H - first);
            const uint16_t *px = row_x(row) + first;
            const uint32_t offx = ANY ? before_16(px) : 0, bytes = (2 * n + offx + 15) & ~15u;
            uint32_t off2 = 0, bytes2 = 0;
            const uint16_t *p2 = nullptr;
            if (SECOND) {
                p2 = row_2(row) + first;
                off2 = ANY ? before_16(p2) : 0;
                bytes2 = (2 * n + off2 + 15) & ~15u;
            }
            const uint32_t bar = full0 + 8 * stage, dst = sb + stage * ring.stage_bytes;
            // debug build: the part lies in its row, its pieces begin at 16 bytes and fit the stage
            if (!QG_IN_BOUNDS(err, row >= 0 && row < a.T && n > 0 && first + n <= a.H && stage < ring.stages &&
                                       (reinterpret_cast<uintptr_t>(px) - offx) % 16 == 0 &&
                                       bytes <= (SECOND ? ring.second_at : ring.stage_bytes)) ||
                (SECOND && !QG_IN_BOUNDS(err, (reinterpret_cast<uintptr_t>(p2) - off2) % 16 == 0 &&
                                                  ring.second_at + bytes2 <= ring.stage_bytes))) {
                mbar_arrive(bar);
                return;
            }
            mbar_arrive_expect_tx(bar, bytes + bytes2);
            const uint64_t policy = ring.once ? l2_policy_evict_first() : l2_policy_evict_normal();
            bulk_load_hint(dst, reinterpret_cast<const uint8_t *>(px) - offx, bytes, bar, policy);
            if (SECOND) bulk_load_hint(dst + ring.second_at, reinterpret_cast<const uint8_t *>(p2) - off2, bytes2, bar, policy);
        };
        const int64_t step = gridDim.x, ahead = step * ring.stages;
        int64_t f_row = blockIdx.x;              // UNIT == 1: the next part to fetch, and how many have been
        int f_part = 0, f_stage = 0, fetched = 0;
        auto fetch_next = [&] {
            if (f_row >= a.T) return;
            fetch(f_row, f_part, f_stage);
            ++fetched;
            if (++f_stage == ring.stages) f_stage = 0;
            if (++f_part == C) {
                f_part = 0;
                f_row += step;
            }
        };
        if (t == 0)
            for (int i = 0; i < ring.stages; ++i) {
                if (UNIT == 1) fetch_next();
                else if (blockIdx.x + i * step < a.T) fetch(blockIdx.x + i * step, 0, i);
            }
        keep_weights();
        int stage = 0, last = -1;                // UNIT == 1: the stage read last, and its phase
        uint32_t phase = 0, last_phase = 0;
        uint64_t limit = timeout_ns;             // UNIT == 1: a wait that gave up leaves the others no time; the lanes stay together
        int64_t row = blockIdx.x;
        const bool all_in = 8 * ((C - 1) * nt + (t | 31)) + 8 <= a.H;
        for (; row < a.T; row += step) {
            if (UNIT == C && !mbar_wait_warp(full0 + 8 * stage, phase, timeout_ns)) {
                limit = 0;
                break;
            }
            const uint8_t *st = rows_smem + stage * ring.stage_bytes, *st2 = st + ring.second_at;
            const uint32_t offx = ANY ? before_16(row_x(row)) : 0, off2 = ANY && SECOND ? before_16(row_2(row)) : 0;
            const int at = stage;
            auto load = [&](int, int e, int n, uint4 &xv, uint4 &sv) {
                    if constexpr (UNIT == C) {
                        if (n <= 0) return;
                        xv = ANY ? shared_any(st + 2 * e, offx, n) : *reinterpret_cast<const uint4 *>(st + 2 * e);
                        if (SECOND) sv = ANY ? shared_any(st2 + 2 * e, off2, n) : *reinterpret_cast<const uint4 *>(st2 + 2 * e);
                    } else {
                        if (!mbar_wait(full0 + 8 * stage, phase, limit)) limit = 0;
                        const uint8_t *p = rows_smem + stage * ring.stage_bytes + 16 * t, *p2 = p + ring.second_at;
                        if (n > 0) {
                            xv = ANY ? shared_any(p, offx, n) : *reinterpret_cast<const uint4 *>(p);
                            if (SECOND) sv = ANY ? shared_any(p2, off2, n) : *reinterpret_cast<const uint4 *>(p2);
                        }
                        fence_proxy_async_smem();                  // read here, written next by the bulk copies
                        __syncwarp();
                        if ((t & 31) == 0) mbar_arrive(empty0 + 8 * stage);
                        if (t == 0 && last >= 0) {                 // the stage before this one: every warp is at its end or past it
                            if (!mbar_wait(empty0 + 8 * last, last_phase, limit)) limit = 0;
                            else if (limit) fetch_next();
                        }
                        last = stage;
                        last_phase = phase;
                        if (++stage == ring.stages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                };
            auto read_done = [&] {
                if (UNIT == C && t == 0 && row + ahead < a.T) fetch(row + ahead, 0, at);
            };
            // (at any alignment a second body costs more than the tests: 5003 x 5111 29.0 us against 26.8)
            if (!ANY && all_in) process(std::bool_constant<!ANY>{}, row, 0, load, read_done);
            else process(std::false_type{}, row, 0, load, read_done);
            if (UNIT == C && ++stage == ring.stages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (limit == 0) {
            if ((t & 31) == 0) atomicOr(err, ERR_PRODUCER);
            // No copy may land after the block has left: those of the stages from here on.
            if (t == 0) {
                if (UNIT == C) fetched = static_cast<int>(min(int64_t(ring.stages), (a.T - row + step - 1) / step));
                for (int k = UNIT == C ? 0 : max(0, fetched - ring.stages); k < fetched; ++k) {
                    const int from = UNIT == C ? stage + k : k;
                    if (!mbar_wait(full0 + 8 * (from % ring.stages), (UNIT == C ? phase : 0) ^ (from / ring.stages & 1), timeout_ns))
                        atomicOr(err, ERR_DRAIN);
                }
            }
        }
    }
}

// Rows of a multiple of 8 elements, 16-byte aligned (8-byte in 8 bits): read and written as they are.
inline bool vec_rows(const void *p, int64_t ld, int item) {
    return reinterpret_cast<uintptr_t>(p) % (8 * item) == 0 && ld % 8 == 0;
}

inline bool vec_eligible(const qgi::RowQuantArgs &a) {
    return a.H % 8 == 0 && vec_rows(a.x, a.ldx, 2) && vec_rows(a.second, a.ld2, 2) && vec_rows(a.sum_out, a.ldso, 2) &&
           vec_rows(a.y, a.ldy, a.y_dtype == a.dtype ? 2 : 1) && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
}

// How rows go through blocks' rings: `c` chunks a thread, as many blocks as registers allow (1024 threads an SM at most), each
// with as many rows on their way as shared memory holds (8 at most).
struct RingPlan {
    Ring ring;
    int threads, blocks;
};

// A kernel's registers a thread, asked once a device (`known`: 0 until then; a query that failed is not kept).
template <class K>
int registers_of(K kern, std::atomic<int> &known) {
    int registers = known.load(std::memory_order_relaxed);
    if (registers == 0) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, kern) != cudaSuccess) {
            cudaGetLastError();              // the launch will say what is wrong
            return 128;
        }
        registers = (at.numRegs + 7) / 8 * 8;
        known.store(registers, std::memory_order_relaxed);
    }
    return registers;
}

constexpr int RING_ROOM = 220 * 1024;    // of an SM's shared memory for rings

inline RingPlan plan_ring(int registers, int c, int unit, int H, bool second, bool any) {
    RingPlan p;
    p.threads = ((H + 7) / 8 + 32 * c - 1) / (32 * c) * 32;
    p.ring.parts = 1;
    p.ring.second_at = (2 * std::min(H, 8 * unit * p.threads) + (any ? 30 : 0)) / 16 * 16;
    p.ring.stage_bytes = second ? 2 * p.ring.second_at : p.ring.second_at;
    p.blocks = std::max(1, std::min({16, 1024 / p.threads, 65536 / (registers * p.threads)}));
    while (p.blocks > 1 && 2 * c / unit * p.ring.stage_bytes > unsigned(RING_ROOM / p.blocks - 1536)) --p.blocks;
    p.ring.stages = std::min(MAX_STAGES, (RING_ROOM / p.blocks - 1536) / static_cast<int>(p.ring.stage_bytes));
    return p;
}

template <class K>
cudaError_t launch_ring(K kern, RingPlan p, int parts, const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    int64_t grid = int64_t(p.blocks) * ctx.num_sms;
    if (grid >= a.T) {           // one row a block
        grid = a.T;
        p.ring.stages = std::min(p.ring.stages, parts);
    }
    // Inputs of more than 64 MB (half of L2) leave it first: 8192 x 8192 with residual 79.0 us against 81.3, where 4096 x 4096, whose
    // inputs may still be there for the next call, would take 21.8 us against 21.2.
    p.ring.once = int64_t(a.T) * a.H * (a.second ? 4 : 2) > (int64_t(1) << 26);
    const int smem = p.ring.stages * static_cast<int>(p.ring.stage_bytes) + 32;   // a row's last pieces at any alignment are read whole
    if (smem > 40 * 1024) {
        // (one size, so that calls of two threads do not lower each other's)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_ROOM);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), p.threads, smem, ctx.stream, a, p.ring, ctx.err,
                            ctx.timeout_ns);
}

template <class TY, int OUT, bool NORM, bool SECOND, bool ANY>
cudaError_t launch_vec(const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    // Short rows a warp, or a part of one, each; and rows in parts of 512 elements where nothing of the whole row is needed.
    constexpr bool APART = !NORM && OUT != OUT_INT8;
    if (a.H <= 512 || APART) {
        auto kern = row_quant_vec_kernel<TY, OUT, NORM, SECOND, 2, 32, ANY, false>;
        int lanes = 32;
        // 16 elements a lane: 327680 heads of 128, norm to 16 bits, 32 us against 94 with a warp each, 30000 x 256 8.0 against 10.7.
        if constexpr (!ANY) {
            if (a.H <= 128) kern = row_quant_vec_kernel<TY, OUT, NORM, SECOND, 2, 8, ANY, false>, lanes = 8;
            else if (a.H <= 256) kern = row_quant_vec_kernel<TY, OUT, NORM, SECOND, 2, 16, ANY, false>, lanes = 16;
        }
        Ring ring{};
        ring.parts = (a.H + 511) / 512;
        const int64_t blocks = (int64_t(a.T) * ring.parts * lanes + 255) / 256;
        if (blocks < (int64_t(1) << 31))
            return launch_dependent(kern, dim3(static_cast<unsigned>(blocks)), 256, 0, ctx.stream, a, ring, ctx.err, ctx.timeout_ns);
    }
    if constexpr (APART) {
        return cudaErrorInvalidConfiguration;    // 2^43 elements
    } else {
        // 16 elements a thread while that leaves two blocks an SM, to alternate between loads and exchanges; else 32 (measured
        // at 4096 x 12288: norm to E4M3 56 us against 61) unless one block is all that fits either way and the first may have the threads;
        // past 16384 elements 32 in up to 1024 threads.
        auto k2 = row_quant_vec_kernel<TY, OUT, NORM, SECOND, 2, 0, ANY, false>;
        auto k4 = row_quant_vec_kernel<TY, OUT, NORM, SECOND, 4, 0, ANY, false>;
        auto big = row_quant_vec_kernel<TY, OUT, NORM, SECOND, 4, 0, ANY, true>;
        static_assert(32 * most_threads(4, ANY, false) >= 16384 && 32 * most_threads(4, ANY, true) >= LONGEST, "every row has a kernel");
        static std::atomic<int> known[qgi::MAX_DEVICES][3];
        std::atomic<int>(&r)[3] = known[ctx.device];
        constexpr int unit = unit_of<NORM, SECOND, 4, true>;
        if (a.H > 16384) return launch_ring(big, plan_ring(registers_of(big, r[2]), 4, unit, a.H, SECOND, ANY), 4 / unit, a, ctx);
        const RingPlan p2 = plan_ring(registers_of(k2, r[0]), 2, 2, a.H, SECOND, ANY);
        const bool two = p2.threads <= most_threads(2, ANY, false);
        if (two && p2.blocks >= 2) return launch_ring(k2, p2, 1, a, ctx);
        const RingPlan p4 = plan_ring(registers_of(k4, r[1]), 4, 4, a.H, SECOND, ANY);
        return p4.blocks >= 2 || !two ? launch_ring(k4, p4, 1, a, ctx) : launch_ring(k2, p2, 1, a, ctx);
    }
}

template <class TY, int OUT>
cudaError_t launch_out(const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    // Past what a block's registers hold; and past what 32 bits with a sign count, where nothing of the whole row is needed.
    if (a.H > (a.norm || OUT == OUT_INT8 ? LONGEST : 1 << 30)) {
        const dim3 grid(static_cast<unsigned>(a.T < ctx.num_sms ? a.T : ctx.num_sms));
        return launch_dependent(row_quant_long_kernel<TY, OUT>, grid, 1024, 0, ctx.stream, a, ctx.err);
    }
    const int kind = 4 * a.norm + 2 * (a.second != nullptr) + vec_eligible(a);
    switch (kind) {
    case 0: return launch_vec<TY, OUT, false, false, true>(a, ctx);
    case 1: return launch_vec<TY, OUT, false, false, false>(a, ctx);
    case 2: return launch_vec<TY, OUT, false, true, true>(a, ctx);
    case 3: return launch_vec<TY, OUT, false, true, false>(a, ctx);
    case 4: return launch_vec<TY, OUT, true, false, true>(a, ctx);
    case 5: return launch_vec<TY, OUT, true, false, false>(a, ctx);
    case 6: return launch_vec<TY, OUT, true, true, true>(a, ctx);
    default: return launch_vec<TY, OUT, true, true, false>(a, ctx);
    }
}

template <class TY>
cudaError_t launch_type(const qgi::RowQuantArgs &a, const qgi::LaunchCtx &ctx) {
    return a.y_dtype == QGEMM_INT8   ? launch_out<TY, OUT_INT8>(a, ctx)
           : a.y_dtype == QGEMM_E4M3 ? launch_out<TY, OUT_E4M3>(a, ctx)
                                     : launch_out<TY, OUT_16>(a, ctx);
}

}  // namespace
