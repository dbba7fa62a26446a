// Column sums of the dropout + add + norm backward's partial rows.
#include "drop_args.h"
#include "norm_device.cuh"

namespace libnorm {

// Partial rows of W values (dgamma, then dbeta) at a pitch of whole 16 bytes,
// added up: a CTA has 128 columns, each of its 32 warps every 32nd partial row,
// then the warps' sums in order. The launch is latency, and 32 warps have every
// value of 256 partial rows on the way at once. (Clusters of CTAs of 8 warps
// that shared the rows and joined them through distributed shared memory: 515 x 768
// with 152 partial rows 8.0 us in all.)
constexpr int kSumWarps = 32, kSumLoads = 8;

__global__ void __launch_bounds__(kSumWarps * 32) drop_colsum(const float* ws, int64_t partials, int32_t W, int32_t pitch, int32_t N,
                                                              float* out0, float* out1) {
    __shared__ float part[kSumWarps][128];
    grid_release();
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 128 + lane * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < W) {
        const float* src = ws + c;
        for (int64_t p0 = warp; p0 < partials; p0 += kSumLoads * kSumWarps) {
            float4 v[kSumLoads];  // all on the way before the first is added
#pragma unroll
            for (int k = 0; k < kSumLoads; ++k) {
                const int64_t p = p0 + k * kSumWarps;
                v[k] = p < partials ? *reinterpret_cast<const float4*>(src + p * pitch) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kSumLoads; ++k) {
                s.x += v[k].x;
                s.y += v[k].y;
                s.z += v[k].z;
                s.w += v[k].w;
            }
        }
    }
    *reinterpret_cast<float4*>(&part[warp][lane * 4]) = s;
    __syncthreads();
    const int i = threadIdx.x, at = blockIdx.x * 128 + i;
    if (i < 128 && at < W) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) t += part[w][i];
        (at < N ? out0[at] : out1[at - N]) = t;
    }
}

cudaError_t launch_drop_colsum(const DropArgs& a, int64_t partials, bool ln, cudaStream_t s) {
    const float* ws = a.ws;
    int32_t N = a.N, W = ln ? 2 * N : N, pitch = drop_partial_pitch(W);
    float *o0 = a.dgamma, *o1 = a.dbeta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((W + 127) / 128));
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void* args[] = {&ws, &partials, &W, &pitch, &N, &o0, &o1};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(drop_colsum), args);
}

}  // namespace libnorm
