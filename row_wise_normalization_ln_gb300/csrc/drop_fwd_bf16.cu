// Dropout + add + norm forward kernels, bf16 rows.
#include "drop_fwd.cuh"

namespace libnorm {

cudaError_t launch_drop_fwd_bf16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return drop_dispatch_fwd<__nv_bfloat16>(p, a, ln, s);
}

}  // namespace libnorm
