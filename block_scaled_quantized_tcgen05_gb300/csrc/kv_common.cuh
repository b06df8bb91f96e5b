// kv_common.cuh -- device helpers of the paged key-value cache kernels: 16-bit types, E4M3 codes
// with UE8M0 scales, and error reporting.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv_index.h"
#include "kv_internal.h"
#include "qgemm_debug.cuh"
#include "qgemm_ptx.cuh"

namespace qg {

// The two 16-bit activation types, by the conversions the kernels need.
struct TypeF16 {
    using T = __half;
    static constexpr bool BF16 = false;
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ uint32_t pack_down(float lo, float hi) {   // towards zero
        uint32_t r;
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
struct TypeBF16 {
    using T = __nv_bfloat16;
    static constexpr bool BF16 = true;
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ uint32_t pack_down(float lo, float hi) {   // towards zero
        uint32_t r;
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

// Launches a kernel as a programmatic dependent of the one before it on the stream: its blocks may be
// resident before that one ends, and wait for it (griddep_wait, first thing in every thread).
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A sequence number, position, length or page-table entry was out of range: what it named is
// skipped and the device error word says so.
__device__ __forceinline__ void report_index(unsigned *err) { atomicOr(err, qgi::ERR_INDEX); }

}  // namespace qg
