// Dropout + add + norm backward kernels, bf16 rows.
#include "drop_bwd.cuh"

namespace libnorm {

cudaError_t launch_drop_bwd_bf16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return drop_dispatch_bwd<__nv_bfloat16>(p, a, ln, s);
}

}  // namespace libnorm
