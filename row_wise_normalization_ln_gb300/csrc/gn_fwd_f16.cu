// Group norm forward kernels, f16 tensors.
#include "gn_fwd.cuh"

namespace libnorm {

cudaError_t launch_gn_fwd_f16(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    return gn_dispatch_fwd<__half>(p, a, act, B, s);
}

}  // namespace libnorm
