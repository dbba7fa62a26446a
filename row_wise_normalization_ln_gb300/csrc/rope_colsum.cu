// Column sums of the head norms' partial weight gradients.
#include "norm_device.cuh"
#include "rope_args.h"

namespace libnorm {

// dw of 8 neighbouring columns of a side per CTA: 128 threads share a column,
// each adds every 128th partial row, eight of them on the way at a time, then
// the threads' sums meet in a warp, in shared memory and in a warp again. D <=
// 512 columns and some hundreds of partial rows: the whole launch is latency,
// so its CTAs are many and their chains short.
constexpr int kRopeSumCols = 8, kRopeSumRows = 128, kRopeSumLoads = 8;
constexpr int kRopeSumWarps = kRopeSumCols * kRopeSumRows / 32;

static __global__ void __launch_bounds__(kRopeSumCols* kRopeSumRows) rope_colsum(const __grid_constant__ RopeArgs g) {
    __shared__ float sm[kRopeSumWarps][kRopeSumCols];
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
        for (int p0 = row; p0 < sd.ctas; p0 += kRopeSumLoads * kRopeSumRows) {
            float v[kRopeSumLoads];
#pragma unroll
            for (int k = 0; k < kRopeSumLoads; ++k) {
                const int p = p0 + k * kRopeSumRows;
                v[k] = p < sd.ctas ? sd.part[int64_t(p) * g.D + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kRopeSumLoads; ++k) t += v[k];
        }
    t += __shfl_xor_sync(kFullMask, t, 8);
    t += __shfl_xor_sync(kFullMask, t, 16);
    if ((threadIdx.x & 31) < kRopeSumCols) sm[threadIdx.x >> 5][col] = t;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    t = 0.f;
#pragma unroll
    for (int k = 0; k < kRopeSumWarps / 4; ++k) t += sm[row + 4 * k][col];
    t += __shfl_xor_sync(kFullMask, t, 8);
    t += __shfl_xor_sync(kFullMask, t, 16);
    if (row == 0 && c < g.D) sd.dw[c] = t;
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
