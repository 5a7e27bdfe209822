// rms_norm_f16.cu -- the norm's kernels for rows in f16.
#include "rms_norm_kernels.cuh"

namespace cns {

cudaError_t launch_rms_norm_f16(const NormParams &p, bool wide, int sms, cudaStream_t s)
{
    return wide ? launch_forward<CNS_DT_F16, true>(p, sms, s) : launch_forward<CNS_DT_F16, false>(p, sms, s);
}

cudaError_t launch_rms_norm_backward_f16(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s)
{
    return wide ? launch_backward<CNS_DT_F16, true>(p, sms, parts, s) : launch_backward<CNS_DT_F16, false>(p, sms, parts, s);
}

}  // namespace cns
