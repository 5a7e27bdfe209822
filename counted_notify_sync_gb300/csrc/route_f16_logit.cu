// route_f16_logit.cu -- the routing kernel for logits of type CNS_DT_F16, chosen by logit.
#define CNS_ROUTE_KERNELS
#include "route_kernels.cuh"

namespace cns {

cudaError_t launch_route_f16_logit(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    return p.groups > p.top_groups ? launch_route<CNS_DT_F16, false, true>(p, ctas, warps, s)
                                   : launch_route<CNS_DT_F16, false, false>(p, ctas, warps, s);
}

}  // namespace cns
