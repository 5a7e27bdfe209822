// route_bf16_logit.cu -- the routing kernel for logits of type CNS_DT_BF16, chosen by logit.
#define CNS_ROUTE_KERNELS
#include "route_kernels.cuh"

namespace cns {

cudaError_t launch_route_bf16_logit(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    return p.groups > p.top_groups ? launch_route<CNS_DT_BF16, false, true>(p, ctas, warps, s)
                                   : launch_route<CNS_DT_BF16, false, false>(p, ctas, warps, s);
}

}  // namespace cns
