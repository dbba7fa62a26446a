// Argument block of the dropout + add + norm kernels and their launchers,
// shared by the host side (drop.cpp) and the kernels (drop_kernels.cuh).
#pragma once

#include <cstdint>

#include <cuda_runtime_api.h>

#include "libnorm_dropout.h"

namespace libnorm {

constexpr int kDropMaxThreads = 512;
constexpr int kDropMaxStages = 4;
constexpr int64_t kDropMaxSmem = 220 * 1024;  // dynamic, per CTA (beside the kernels' own few KB)
constexpr int kDropChain = 64;                // rows whose column terms are added one after the other

struct DropArgs {
    const void *x, *residual;       // forward
    const void *dy, *dh, *hin;      // backward
    const void *gamma, *beta;
    void *h, *y;                    // forward
    void *dx, *dres;                // backward; dx: null without dropout
    float *mean, *rstd;             // written by the forward, read by the backward (LayerNorm)
    float* ws;                      // backward: partial rows [partials][NA][N]
    float *dgamma, *dbeta;
    const uint64_t* rng;            // seed, offset in device memory, or null:
    uint64_t seed, offset;
    int64_t M;
    int32_t N;
    int32_t lanes;                  // lanes of a warp per row; 0: a CTA or a cluster
    int32_t cluster;
    int32_t stages;
    int32_t words_at, sums_at;      // where the masks' words and the column sums lie in shared memory
    uint32_t limit;                 // dropped where the word is below limit >> 16
    float scale, eps, invN;
};

// Elements per thread: 16 at most in the backward (its column sums stay in
// registers), 32 in the forward.
inline int drop_max_elems(bool backward) { return backward ? 16 : 32; }

// Dynamic shared memory of a launch: the ring of upcoming rows' accesses (of
// each thread its own; none where an access is one 16-bit element), the words
// of the mask where accesses are elements (16 bytes per group of 8 elements
// that a warp, or the lanes of a row, touch: two more than they have), and for
// rows that lanes share the backward's column sums.
inline int64_t drop_mask_bytes(int vec, int per_thread, int threads, int lanes) {
    const int unit = lanes > 0 ? lanes : 32;
    return vec == 1 ? 16 * int64_t(threads / unit) * ((unit * per_thread + 7) / 8 + 2) : 0;
}
inline int64_t drop_ring_bytes(int vec, int elem, int per_thread, int threads, int stages, int streams) {
    return vec * elem >= 4 ? int64_t(stages) * streams * per_thread * threads * vec * elem : 0;
}
inline int64_t drop_sums_bytes(bool ln, int vec, int per_thread, int threads) {
    return int64_t(ln ? 2 : 1) * vec * per_thread * threads * 4;
}

cudaError_t launch_drop_fwd_f32(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_fwd_bf16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_fwd_f16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_bwd_f32(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_bwd_bf16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_bwd_f16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);

// The sums of `partials` partial rows of columns: dgamma (and dbeta); zeros where there are none.
cudaError_t launch_drop_colsum(const DropArgs& a, int64_t partials, bool ln, cudaStream_t s);

}  // namespace libnorm
