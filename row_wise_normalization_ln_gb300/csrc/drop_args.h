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
constexpr int kDropChain = 64;                // rows whose column terms are added one after the other, at most

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
    int32_t pitch;                  // elements: bytes from one tensor's part of a row to the next
    int32_t words_at, sums_at;      // where the masks' words and the column sums lie in shared memory
    uint32_t limit;                 // dropped where the word is below limit >> 16
    float scale, eps, invN;
};

// The instances there are: accesses per thread V (of elements: pairs) and rows
// at a time R. A forward thread holds at most 32 values, a backward one the
// column sums of at most 16 columns.
inline bool drop_known(bool backward, bool group, int vec, int elem, int per_thread, int rows) {
    if (vec == 1) return !group && rows == 1 && (per_thread == 2 || per_thread == 8);
    if (vec * elem != 16) return false;
    if (group) return (per_thread == 1 && rows == 4) || (per_thread == 2 && rows == 2);
    if (per_thread == 1) return rows == 1 || rows == 4;
    if (elem == 4) return per_thread == 4 && (rows == 1 || rows == 2);
    return (per_thread == 2 && rows == 2) || (per_thread == 4 && !backward && rows == 1);
}

// Columns of a CTA's part of a row.
inline int64_t drop_cta_cols(int vec, int per_thread, int threads) { return int64_t(threads) * per_thread * (vec == 1 ? 2 : vec); }

// Shared memory of the stages: of each thread's own accesses, or of the CTA's
// part of a row of elements in whole 16-byte chunks at a pitch; of the masks'
// words of two rows of elements; and of the backward's column sums of rows
// that lanes share.
inline int64_t drop_pitch(int elem, int per_thread, int threads) { return (drop_cta_cols(1, per_thread, threads) * elem + 30) / 16 * 16; }
inline int64_t drop_ring_bytes(int vec, int elem, int per_thread, int threads, int rows, int stages, int streams) {
    return vec == 1 ? stages * streams * drop_pitch(elem, per_thread, threads)
                    : int64_t(stages) * streams * rows * per_thread * threads * 16;
}
inline int64_t drop_words_bytes(int vec, int per_thread, int threads) {
    return vec == 1 ? 2 * 16 * (drop_cta_cols(1, per_thread, threads) / 8 + 2) : 0;
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
