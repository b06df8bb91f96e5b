// w8a8_common.cuh -- what the kernels of the integer product share: the output's arithmetic, and the exact int8 -> fp16 of int8_f16.cuh.
#pragma once

#include "int8_f16.cuh"
#include "kv_common.cuh"
#include "linear8_internal.h"

namespace qg {

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
