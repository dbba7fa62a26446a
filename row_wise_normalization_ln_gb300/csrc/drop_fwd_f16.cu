// Dropout + add + norm forward kernels, fp16 rows.
#include "drop_fwd.cuh"

namespace libnorm {

cudaError_t launch_drop_fwd_f16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return drop_dispatch_fwd<__half>(p, a, ln, s);
}

}  // namespace libnorm
