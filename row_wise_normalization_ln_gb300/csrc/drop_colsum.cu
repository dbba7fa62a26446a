// Column sums of the dropout + add + norm backward's partial rows.
#include <algorithm>

#include "drop_args.h"
#include "norm_device.cuh"

namespace libnorm {

// Partial rows of W values (dgamma, then dbeta) added up: a CTA of 8 warps has
// 32 x VEC columns, each warp every 8th of its CTA's partial rows; the CTAs of
// a cluster share the rows, and rank 0 adds their sums in rank order through
// distributed shared memory. The order depends on the numbers alone. The
// launch is latency, so the rows are shared out until a warp has few: 152
// partial rows of 16384 values 8.5 us with a CTA's 32 warps to a column, ..
constexpr int kSumWarps = 8;

template <int VEC>
__global__ void __launch_bounds__(kSumWarps * 32) drop_colsum(const float* ws, int64_t partials, int32_t W, int32_t N, float* out0, float* out1) {
    __shared__ float part[kSumWarps][32 * VEC];
    __shared__ float mine[32 * VEC];
    grid_release();
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int c = (blockIdx.x / C) * 32 * VEC + lane * VEC;
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = 0.f;
    if (c < W)
#pragma unroll 8
        for (int64_t p = rank * kSumWarps + warp; p < partials; p += C * kSumWarps) {
            const float* src = ws + p * W + c;
            if constexpr (VEC == 4) {
                const float4 v = *reinterpret_cast<const float4*>(src);
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            } else {
                s[0] += *src;
            }
        }
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[warp][lane * VEC + e] = s[e];
    __syncthreads();
    float t = 0.f;
    const int i = threadIdx.x;
    if (i < 32 * VEC) {
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) t += part[w][i];
        mine[i] = t;
    }
    if (C > 1) {
        cluster_barrier();
        if (rank == 0 && i < 32 * VEC)
            for (int k = 1; k < C; ++k) t += ld_peer_f32(peer_smem_addr(&mine[i], static_cast<uint32_t>(k)));
        cluster_barrier();  // no CTA leaves while its sums may be read
    }
    const int at = (blockIdx.x / C) * 32 * VEC + i;
    if (rank == 0 && i < 32 * VEC && at < W) (at < N ? out0[at] : out1[at - N]) = t;
}

cudaError_t launch_drop_colsum(const DropArgs& a, int64_t partials, bool ln, cudaStream_t s) {
    const float* ws = a.ws;
    int32_t N = a.N, W = ln ? 2 * N : N;
    float *o0 = a.dgamma, *o1 = a.dbeta;
    const int vec = W % 4 == 0 ? 4 : 1;
    // a warp has at most 8 partial rows, as far as clusters of 8 reach
    unsigned cluster = 1;
    while (cluster < 8 && partials > int64_t(cluster) * kSumWarps * 8) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((W + 32 * vec - 1) / (32 * vec)) * cluster);
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void* args[] = {&ws, &partials, &W, &N, &o0, &o1};
    return cudaLaunchKernelExC(&cfg, vec == 4 ? reinterpret_cast<const void*>(drop_colsum<4>) : reinterpret_cast<const void*>(drop_colsum<1>), args);
}

}  // namespace libnorm
