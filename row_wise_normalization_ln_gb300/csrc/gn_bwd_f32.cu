// Group norm backward kernels, f32 tensors.
#include "gn_bwd.cuh"

namespace libnorm {

cudaError_t launch_gn_bwd_f32(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    return gn_dispatch_bwd<float>(p, a, act, B, s);
}

}  // namespace libnorm
