/* cudart_calls.c -- stands in for the CUDA runtime's calls that an entry point's host code makes, for tests
 * without a GPU: preloaded before libcns.so, it records them, reports a GB300, and lets one launch fail. */
#include <cuda_runtime_api.h>

enum { LAUNCH = 0, ATTRIBUTE = 1, MEMSET = 2, MOST = 4096 };

typedef struct {
    int kind;
    int failed;
    const void *what;      /* the kernel; for a memset, its address */
    unsigned long long n;  /* shared memory; the attribute's value; bytes */
    const void *stream;
} call_t;

static call_t calls[MOST];
static int made, launches, failing;

static void note(int kind, int failed, const void *what, unsigned long long n, const void *stream)
{
    if (made < MOST) {
        call_t c = {kind, failed, what, n, stream};
        calls[made++] = c;
    }
}

/* Forget the calls so far; launch number `fail` from here on (from 1; 0: none) returns an error. */
void fake_reset(int fail)
{
    made = launches = 0;
    failing = fail;
}

int fake_calls(call_t *out, int room)
{
    for (int i = 0; i < made && i < room; ++i)
        out[i] = calls[i];
    return made;
}

static cudaError_t launched(const void *kernel, size_t smem, cudaStream_t s)
{
    const int fails = ++launches == failing;
    note(LAUNCH, fails, kernel, smem, s);
    return fails ? cudaErrorLaunchOutOfResources : cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *cfg, const void *kernel, void **args)
{
    (void)args;
    return launched(kernel, cfg->dynamicSmemBytes, cfg->stream);
}

cudaError_t cudaLaunchKernel(const void *kernel, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t s)
{
    (void)grid, (void)block, (void)args;
    return launched(kernel, smem, s);
}

cudaError_t cudaFuncSetAttribute(const void *kernel, enum cudaFuncAttribute attr, int value)
{
    if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize)
        note(ATTRIBUTE, 0, kernel, value, 0);
    return cudaSuccess;
}

cudaError_t cudaMemsetAsync(void *at, int value, size_t n, cudaStream_t s)
{
    note(MEMSET, value != 0, at, n, s);
    return cudaSuccess;
}

cudaError_t cudaGetDevice(int *device)
{
    *device = 0;
    return cudaSuccess;
}

cudaError_t cudaDeviceGetAttribute(int *value, enum cudaDeviceAttr attr, int device)
{
    (void)device;
    *value = attr == cudaDevAttrMultiProcessorCount             ? 152
             : attr == cudaDevAttrMaxThreadsPerMultiProcessor   ? 2048
             : attr == cudaDevAttrComputeCapabilityMajor        ? 10
             : attr == cudaDevAttrComputeCapabilityMinor        ? 3
                                                                : 0;
    return cudaSuccess;
}

cudaError_t cudaGetLastError(void) { return cudaSuccess; }
