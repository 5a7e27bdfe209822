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
constexpr uint32_t kStepEpochWord = 0;                             // line 0: calls done on this workspace
constexpr uint32_t kStepStatusWord = CNS_SYNCALL_LINE_BYTES / 4;   // line 1: status, abort, round, CTA
constexpr uint32_t kStepSlotWord = 512;                            // byte 2048: one 16-byte slot per CTA
constexpr uint32_t kStepMaxCtas = (CNS_STEP_WORKSPACE_HEADER_BYTES - 2048) / 16;

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

// ---------------------------------------------------------------------------
// The exchange: every CTA publishes one 64-bit value, every CTA gets them all
// ---------------------------------------------------------------------------
//
// A reduction that every CTA needs the result of is a barrier that carries a
// value.  Each CTA stores {value, tag} to its own 16-byte slot (one 128-bit
// access, so a tag never shows without its value) and polls all slots until
// each shows the call's tag.  The tag is the workspace's count of calls plus
// one: whatever grid sizes came before, no older slot carries it, and nothing
// has to be reset.  CTA 0 advances the count once it has seen every slot --
// every CTA had read the count by then.
//
// Against the soft SYNCALL barrier with the values stored beside it this saves
// the release fence, the atomic's round trip and the values' loads behind it.

struct Slot {
    uint64_t value, tag;
};

__device__ __forceinline__ void st_slot(uint32_t *header, uint32_t cta, uint64_t value, uint64_t tag)
{
    asm volatile("{\n\t.reg .b128 q;\n\tmov.b128 q, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], q;\n\t}" ::"l"(
                     header + kStepSlotWord + 4 * cta),
                 "l"(value), "l"(tag)
                 : "memory");
}

__device__ __forceinline__ Slot ld_slot(const uint32_t *header, uint32_t cta)
{
    Slot s;
    asm volatile("{\n\t.reg .b128 q;\n\tld.relaxed.gpu.global.b128 q, [%2];\n\tmov.b128 {%0, %1}, q;\n\t}"
                 : "=l"(s.value), "=l"(s.tag)
                 : "l"(header + kStepSlotWord + 4 * cta)
                 : "memory");
    return s;
}

// One warp waits for the slots of `ctas` CTAs and calls take(cta, value) for
// each, CTA c on lane c % 32, in rising order.  The slots of a batch are all
// in flight at once.  Bounded: true when the wait gave up (then the
// workspace's status is CNS_ERR_TIMEOUT).
template <class Take>
__device__ __forceinline__ bool wait_slots(uint32_t *header, uint32_t ctas, uint64_t tag, uint64_t timeout_ns, Take take)
{
    constexpr uint32_t kBatch = 5;   // 160 CTAs: the GPU's 152 SMs in one
    uint32_t *status = header + kStepStatusWord;
    const uint32_t lane = threadIdx.x & 31u;
    uint64_t deadline = 0;
    uint32_t spins = 0;
    for (uint32_t first = 0; first < ctas; first += 32 * kBatch) {
        Slot s[kBatch];
        for (;;) {
            bool all = true;
#pragma unroll
            for (uint32_t i = 0; i < kBatch; ++i) {
                const uint32_t c = first + 32 * i + lane;
                if (c < ctas)
                    s[i] = ld_slot(header, c);
            }
#pragma unroll
            for (uint32_t i = 0; i < kBatch; ++i)
                all &= first + 32 * i + lane >= ctas || s[i].tag == tag;
            if (__all_sync(kFullWarp, all))
                break;
            if ((++spins & 63u) == 0u) {
                // the warp decides together, by lane 0's view
                bool stop = false;
                if (lane == 0) {
                    const uint64_t now = globaltimer_ns();
                    if (ld_relaxed_gpu(status + 1) != 0u) {
                        stop = true;
                    } else if (deadline == 0) {
                        deadline = now + timeout_ns;
                    } else if (now > deadline) {
                        raise_timeout(status, 0u, blockIdx.x);
                        stop = true;
                    }
                }
                if (__any_sync(kFullWarp, stop))
                    return true;
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < kBatch; ++i)
            if (first + 32 * i + lane < ctas)
                take(first + 32 * i + lane, s[i].value);
    }
    return false;
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
