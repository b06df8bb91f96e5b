// w8a8_common.cuh -- what the kernels of the integer product share: exact int8 -> fp16, and the
// output's arithmetic.
#pragma once

#include "kv_common.cuh"
#include "linear8_internal.h"

namespace qg {

// 4 int8 (one word) -> two fp16x2 of the same integers in order: q + 128 placed as a byte into the mantissa
// of 1024, less 1152 (both exact; a published integer-to-half technique, as in the int8 GEMV).
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140u);       // halves 0x64|b0, 0x64|b1
    const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342u);       // halves 0x64|b2, 0x64|b3
    const uint32_t bias = 0x64806480u;                             // 1152 = 1024 + 128
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(bias));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(bias));
}

__device__ __forceinline__ float load_16(const void *p, int64_t i, int bf16) {
    const uint16_t v = static_cast<const uint16_t *>(p)[i];
    return bf16 ? __uint_as_float(uint32_t(v) << 16) : __half2float(__ushort_as_half(v));
}

__device__ __forceinline__ uint16_t round_16(float x, int bf16) {
    return static_cast<uint16_t>(bf16 ? TypeBF16::pack(x, 0.0f) : TypeF16::pack(x, 0.0f));
}

// One output from its sum: the scales, the bias, the old value, ReLU.
__device__ __forceinline__ float finish(float sum, float sa, float sw, float bias, float old, int epi) {
    float x = sum * sa * sw + bias;
    if (epi & qgi::EPI_ACCUMULATE) x += old;
    return epi & qgi::EPI_RELU ? fmaxf(x, 0.0f) : x;
}

}  // namespace qg
