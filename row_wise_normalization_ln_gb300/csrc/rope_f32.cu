// Head norm + rotation kernels, fp32 tensors.
#include "rope.cuh"

namespace libnorm {

cudaError_t launch_rope_f32(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s) {
    return rope_dispatch<float>(p, a, interleaved, backward, s);
}

}  // namespace libnorm
