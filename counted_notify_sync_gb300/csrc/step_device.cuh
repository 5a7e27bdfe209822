// step_device.cuh -- what the device-wide steps (route.cu, gradclip.cu) share:
// element types, warp reductions, and the workspace's layout.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "cns.h"
#include "cns_device.cuh"

namespace cns {

// Workspace header (cns_step_workspace_init zeroes it), in 32-bit words.
constexpr uint32_t kStepStatusWord = CNS_SYNCALL_LINE_BYTES / 4;   // line 1: status, abort, round, CTA

constexpr unsigned kFullWarp = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFullWarp, v, d);
    return v;
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFullWarp, v, d);
    return v;
}

// One element of type `dtype` (cns_dtype_t) as a float, and back.
template <int D> struct Elem;
template <> struct Elem<CNS_DT_F32> {
    using type = float;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <> struct Elem<CNS_DT_BF16> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<CNS_DT_F16> {
    using type = __half;
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

}  // namespace cns
