// route_f32_logit.cu -- the routing kernel for logits of type CNS_DT_F32, chosen by logit.
#define CNS_ROUTE_KERNELS
#include "route_kernels.cuh"

namespace cns {

cudaError_t launch_route_f32_logit(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    return p.groups > p.top_groups ? launch_route<CNS_DT_F32, false, true>(p, ctas, warps, s)
                                   : launch_route<CNS_DT_F32, false, false>(p, ctas, warps, s);
}

}  // namespace cns
