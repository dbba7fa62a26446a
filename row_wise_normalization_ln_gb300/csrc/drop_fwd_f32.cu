// Dropout + add + norm forward kernels, fp32 rows.
#include "drop_fwd.cuh"

namespace libnorm {

cudaError_t launch_drop_fwd_f32(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return drop_dispatch_fwd<float>(p, a, ln, s);
}

}  // namespace libnorm
