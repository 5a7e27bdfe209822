// route_f32_score.cu -- the routing kernel for logits of type CNS_DT_F32, chosen by score.
#define CNS_ROUTE_KERNELS
#include "route_kernels.cuh"

namespace cns {

cudaError_t launch_route_f32_score(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    return p.groups > p.top_groups ? launch_route<CNS_DT_F32, true, true>(p, ctas, warps, s)
                                   : launch_route<CNS_DT_F32, true, false>(p, ctas, warps, s);
}

}  // namespace cns
