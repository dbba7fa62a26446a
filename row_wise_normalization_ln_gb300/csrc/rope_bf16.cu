// Head norm + rotation kernels, bf16 tensors.
#include "rope.cuh"

namespace libnorm {

cudaError_t launch_rope_bf16(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s) {
    return rope_dispatch<__nv_bfloat16>(p, a, interleaved, backward, s);
}

}  // namespace libnorm
