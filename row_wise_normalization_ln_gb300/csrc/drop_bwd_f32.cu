// Dropout + add + norm backward kernels, fp32 rows.
#include "drop_bwd.cuh"

namespace libnorm {

cudaError_t launch_drop_bwd_f32(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return drop_dispatch_bwd<float>(p, a, ln, s);
}

}  // namespace libnorm
