// Group norm backward kernels, bf16 tensors.
#include "gn_bwd.cuh"

namespace libnorm {

cudaError_t launch_gn_bwd_bf16(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    return gn_dispatch_bwd<__nv_bfloat16>(p, a, act, B, s);
}

}  // namespace libnorm
