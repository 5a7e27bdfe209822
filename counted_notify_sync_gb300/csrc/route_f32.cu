// route_f32.cu -- the routing kernel for logits of type CNS_DT_F32.
#define CNS_ROUTE_KERNELS
#include "route_kernels.cuh"

namespace cns {

cudaError_t launch_route_f32(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    return launch_route<CNS_DT_F32>(p, ctas, warps, s);
}

}  // namespace cns
