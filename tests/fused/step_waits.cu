// step_waits.cu -- one CTA of an exchange whose other CTAs never send, for tests of the bounded wait.
#include <cuda_runtime.h>

#include <cstdint>

#include "step_device.cuh"

namespace {

// out[0]: whether the wait gave up; out[1 + c]: the value of CTA c, when it did not.
__global__ void wait_kernel(uint32_t *header, uint32_t sent, uint32_t ctas, uint32_t tag, uint64_t timeout_ns,
                            uint32_t *out)
{
    float r[cns::kStepMaxCtas / 32];
    for (uint32_t from = threadIdx.x; from < sent; from += 32)
        cns::st_relaxed_gpu_u64(cns::mailbox(header, 0, from), static_cast<uint64_t>(tag) << 32 | (100u + from));
    __syncwarp();
    const bool stop = cns::receive_all(header, ctas, tag, timeout_ns, r);
    if (threadIdx.x == 0)
        out[0] = stop;
    for (uint32_t i = 0; !stop && i < cns::kStepMaxCtas / 32; ++i)
        if (32 * i + threadIdx.x < ctas)
            out[1 + 32 * i + threadIdx.x] = __float_as_uint(r[i]);
}

}  // namespace

// `sent` of the `ctas` CTAs have sent; returns a cudaError_t.
extern "C" int step_wait(uint32_t *header, uint32_t sent, uint32_t ctas, uint32_t tag, uint64_t timeout_ns,
                         uint32_t *out, cudaStream_t stream)
{
    if (ctas == 0 || ctas > cns::kStepMaxCtas || sent > ctas || timeout_ns > 1000000000ull)
        return cudaErrorInvalidValue;
    wait_kernel<<<1, 32, 0, stream>>>(header, sent, ctas, tag, timeout_ns, out);
    return cudaGetLastError();
}
