// Group norm forward kernels, f32 tensors.
#include "gn_fwd.cuh"

namespace libnorm {

cudaError_t launch_gn_fwd_f32(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    return gn_dispatch_fwd<float>(p, a, act, B, s);
}

}  // namespace libnorm
