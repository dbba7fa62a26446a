// Head norm + rotation kernels, fp16 tensors.
#include "rope.cuh"

namespace libnorm {

cudaError_t launch_rope_f16(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s) {
    return rope_dispatch<__half>(p, a, interleaved, backward, s);
}

}  // namespace libnorm
