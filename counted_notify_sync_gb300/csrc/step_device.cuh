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
constexpr uint32_t kStepEpochWord = 0;                             // line 0: exchanges done on this workspace
constexpr uint32_t kStepPlanWord = 1;                              // CTAs of a plan that have the blocks' sums
constexpr uint32_t kStepTicketWord = 2;                            // CTAs that gather_last has seen
constexpr uint32_t kStepStatusWord = CNS_SYNCALL_LINE_BYTES / 4;   // line 1: status, abort, round, CTA
constexpr uint32_t kStepBoxWord = 2048;                            // byte 8192: the mailboxes
constexpr uint32_t kStepMaxCtas = 160;
constexpr uint32_t kStepBlockCtas = 16;                            // CTAs whose counts are summed together
constexpr uint32_t kStepSumWord = kStepBoxWord + 2 * kStepMaxCtas * kStepMaxCtas;   // [blocks][experts] of route.cu
constexpr uint32_t kStepSumWords = kStepMaxCtas / kStepBlockCtas * CNS_ROUTE_MAX_EXPERTS;
static_assert(4 * (kStepSumWord + kStepSumWords) == CNS_STEP_WORKSPACE_HEADER_BYTES, "header layout");

// Launches of CTAs that wait for one another: cooperative, so that all are on the GPU together.
inline cudaLaunchConfig_t together_launch(cudaLaunchAttribute *a)
{
    a->id = cudaLaunchAttributeCooperative;
    a->val.cooperative = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cfg;
}

// All other launches: the grid is set up while the one before it in the stream finishes, and waits for that one's
// results by grid_dependency_wait, which every thread calls before it touches memory.  In a stream of them a grid
// is scheduled 0.3-0.6 us after the last one's CTAs have left, where ordinary launches follow one another in steps
// of 2.05 us: calls of a routing gradient that queue behind other work take the GPU 1.8 us each at 509 x 64 against
// 4.1, at 16384 x 256 4.5 against 6.2.
inline cudaLaunchConfig_t early_launch(cudaLaunchAttribute *a)
{
    a->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cfg;
}

constexpr unsigned kFullWarp = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFullWarp, v, d);
    return v;
}

// ---------------------------------------------------------------------------
// The exchange: every CTA sends one 32-bit value, every CTA gets them all
// ---------------------------------------------------------------------------
//
// A reduction that every CTA needs the result of is a barrier that carries a
// value.  Each CTA has a row of mailboxes, one 64-bit word {tag, value} from
// each CTA; a CTA stores its word into every row and then polls its own until
// every box shows the call's tag.  The tag is the workspace's count of calls
// plus one: whatever grid sizes came before, no older word carries it, and
// nothing has to be reset.  CTA 0 advances the count once it has seen every
// box -- every CTA had read the count by then.
//
// Nobody polls a line that another SM polls.  (With one slot per CTA that all
// CTAs poll, 152 x 19 lines of requests met at the L2 slices of those 19
// lines, and the exchange took 2.0-2.8 us.)  Against the soft SYNCALL barrier
// with the values stored beside it, it saves the release fence, the atomic's
// round trip and the loads of the values behind the barrier.

__device__ __forceinline__ uint64_t *mailbox(uint32_t *header, uint32_t to, uint32_t from)
{
    return reinterpret_cast<uint64_t *>(header + kStepBoxWord) + to * kStepMaxCtas + from;
}

// The calling warp stores its CTA's value into the rows of `ctas` CTAs.
__device__ __forceinline__ void send_all(uint32_t *header, uint32_t ctas, uint32_t tag, uint32_t value)
{
    const uint64_t word = static_cast<uint64_t>(tag) << 32 | value;
#pragma unroll
    for (uint32_t c = 0; c < kStepMaxCtas; c += 32) {
        const uint32_t to = c + (threadIdx.x & 31u);
        if (to < ctas)
            st_relaxed_gpu_u64(mailbox(header, to, blockIdx.x), word);
    }
}

// The calling warp waits for its CTA's row: value[i] becomes the value of CTA
// 32 i + lane (0 beyond the last).  Bounded: true when the wait gave up (then
// the workspace's status is CNS_ERR_TIMEOUT).
template <class T>
__device__ __forceinline__ bool receive_all(uint32_t *header, uint32_t ctas, uint32_t tag, uint64_t timeout_ns, T *value)
{
    constexpr uint32_t kBatch = kStepMaxCtas / 32;
    static_assert(sizeof(T) == 4, "values are 32-bit words");
    uint32_t *status = header + kStepStatusWord;
    const uint32_t lane = threadIdx.x & 31u;
    const uint64_t *row = mailbox(header, blockIdx.x, lane);
    uint64_t deadline = 0;
    uint32_t spins = 0;
    uint64_t s[kBatch];
    for (;;) {
        bool all = true;
#pragma unroll
        for (uint32_t i = 0; i < kBatch; ++i)
            s[i] = 32 * i + lane < ctas ? ld_relaxed_gpu_u64(row + 32 * i) : static_cast<uint64_t>(tag) << 32;
#pragma unroll
        for (uint32_t i = 0; i < kBatch; ++i)
            all &= static_cast<uint32_t>(s[i] >> 32) == tag;
        if (__all_sync(kFullWarp, all))
            break;
        if ((++spins & 63u) == 0u) {
            bool stop = false;   // the warp decides together, by lane 0's view
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
    for (uint32_t i = 0; i < kBatch; ++i) {
        const uint32_t v = static_cast<uint32_t>(s[i]);
        value[i] = *reinterpret_cast<const T *>(&v);
    }
    return false;
}

// Where only the result leaves the GPU, nobody has to wait: every CTA leaves
// its value in the first row of mailboxes (under tag 0, which no call polls
// for) and the last one to do so gets them all.  The calling warp gets true in
// that CTA, with value[i] as receive_all fills it.
template <class T>
__device__ __forceinline__ bool gather_last(uint32_t *header, uint32_t ctas, uint32_t value, T *values)
{
    static_assert(sizeof(T) == 4, "values are 32-bit words");
    const uint32_t lane = threadIdx.x & 31u;
    uint32_t before = 0;
    if (lane == 0) {
        st_relaxed_gpu_u64(mailbox(header, 0, blockIdx.x), value);
        fence_release_gpu();
        before = atom_add_relaxed_gpu(header + kStepTicketWord, 1u);
        fence_acquire_gpu();
    }
    if (__shfl_sync(kFullWarp, before, 0) != ctas - 1u)
        return false;
    __syncwarp();
#pragma unroll
    for (uint32_t i = 0; i < kStepMaxCtas / 32; ++i) {
        const uint32_t v =
            32 * i + lane < ctas ? static_cast<uint32_t>(ld_relaxed_gpu_u64(mailbox(header, 0, 32 * i + lane))) : 0u;
        values[i] = *reinterpret_cast<const T *>(&v);
    }
    if (lane == 0)
        st_relaxed_gpu(header + kStepTicketWord, 0u);   // for the next call
    return true;
}

// e^x for what only ranks experts, and what an exact value settles where it leaves that open (the routing's near
// keys): off by a relative 2^-22 + 2^-23 |x|; tiny results are 0.
__device__ __forceinline__ float exp_near(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
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
