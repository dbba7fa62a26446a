// Column sums of the head norms' partial weight gradients.
#include "norm_device.cuh"
#include "rope_args.h"

namespace libnorm {

// dw of 8 neighbouring columns of a side per CTA: 32 threads share a column,
// each adds every 32nd partial row, and their sums meet in a tree in shared
// memory. D <= 512 columns and some hundreds of partial rows: the whole
// launch is latency, so its CTAs are many and their chains short.
constexpr int kRopeSumCols = 8, kRopeSumRows = 32;

static __global__ void __launch_bounds__(kRopeSumCols* kRopeSumRows) rope_colsum(const __grid_constant__ RopeArgs g) {
    __shared__ float sm[kRopeSumRows][kRopeSumCols + 1];
    grid_release();
    grid_wait();
    const int tiles = (g.D + kRopeSumCols - 1) / kRopeSumCols;
    const bool second = static_cast<int>(blockIdx.x) >= (g.side[0].heads > 0 ? tiles : 0);
    const RopeSide& sd = g.side[second];
    const int tile = static_cast<int>(blockIdx.x) - (second && g.side[0].heads > 0 ? tiles : 0);
    const int col = threadIdx.x % kRopeSumCols, row = threadIdx.x / kRopeSumCols;
    const int c = tile * kRopeSumCols + col;
    float t = 0.f;
    if (c < g.D)
#pragma unroll 4
        for (int p = row; p < sd.ctas; p += kRopeSumRows) t += sd.part[int64_t(p) * g.D + c];
    sm[row][col] = t;
    for (int half = kRopeSumRows / 2; half > 0; half >>= 1) {
        __syncthreads();
        if (row < half) sm[row][col] += sm[row + half][col];
    }
    if (row == 0 && c < g.D) sd.dw[c] = sm[0][col];
}

cudaError_t launch_rope_colsum(const RopeArgs& a, cudaStream_t s) {
    const int tiles = (a.D + kRopeSumCols - 1) / kRopeSumCols;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * ((a.side[0].heads > 0) + (a.side[1].heads > 0))));
    cfg.blockDim = dim3(kRopeSumCols * kRopeSumRows);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<RopeArgs*>(&a)};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(rope_colsum), args);
}

}  // namespace libnorm
