// Group norm forward kernels, bf16 tensors.
#include "gn_fwd.cuh"

namespace libnorm {

cudaError_t launch_gn_fwd_bf16(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    return gn_dispatch_fwd<__nv_bfloat16>(p, a, act, B, s);
}

}  // namespace libnorm
