// Column sums of the dropout + add + norm backward's partial rows.
#include "drop_args.h"
#include "norm_bwd.cuh"

namespace libnorm {

cudaError_t launch_drop_colsum(const DropArgs& a, int64_t partials, bool ln, cudaStream_t s) {
    const float* ws = a.ws;
    int32_t N = a.N;
    float *o0 = a.dgamma, *o1 = ln ? a.dbeta : a.dgamma;
    void* args[] = {&ws, &partials, &N, &o0, &o1};
    const bool many = partials > 64;
    const void* fn = ln ? (many ? reinterpret_cast<const void*>(norm_bwd_colsum<2, 1, 32>) : reinterpret_cast<const void*>(norm_bwd_colsum<2, 1, 8>))
                        : (many ? reinterpret_cast<const void*>(norm_bwd_colsum<1, 1, 32>) : reinterpret_cast<const void*>(norm_bwd_colsum<1, 1, 8>));
    return launch_pdl(fn, dim3(static_cast<unsigned>((N + 31) / 32)), dim3(many ? 1024 : 256), 0, 1, s, args);
}

}  // namespace libnorm
