// int8_f16.cuh -- 8-bit integers on the warp-level fp16 tensor path: the exact conversion and the instruction, shared by the int8 GEMV
// and the integer product.
#pragma once

#include <cstdint>

namespace qg {

// 4 int8 (one word) -> two fp16x2 of the same integers in order: q + 128 placed as a byte into the mantissa of 1024, less 1152 (both
// exact; a published integer-to-half technique).
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;                            // q + 128, as unsigned bytes
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140u);       // halves 0x64|b0, 0x64|b1
    const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342u);       // halves 0x64|b2, 0x64|b3
    const uint32_t bias = 0x64806480u;                             // 1152 = 1024 + 128
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(bias));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(bias));
}

// d = a b + c.  Not volatile: a pure function of its registers, so the compiler may interleave the MMAs of independent fragments.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

}  // namespace qg
