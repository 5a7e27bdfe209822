// rms_norm_f32.cu -- the norm's kernels for rows in f32.
#include "rms_norm_kernels.cuh"

namespace cns {

cudaError_t launch_rms_norm_f32(const NormParams &p, bool wide, int sms, cudaStream_t s)
{
    return wide ? launch_forward<CNS_DT_F32, true>(p, sms, s) : launch_forward<CNS_DT_F32, false>(p, sms, s);
}

cudaError_t launch_rms_norm_backward_f32(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s)
{
    return wide ? launch_backward<CNS_DT_F32, true>(p, sms, parts, s) : launch_backward<CNS_DT_F32, false>(p, sms, parts, s);
}

}  // namespace cns
