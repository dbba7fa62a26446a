// Argument block of the dropout + add + norm kernels and their launchers,
// shared by the host side (drop.cpp) and the kernels (drop_kernels.cuh).
#pragma once

#include <cstdint>

#include <cuda_runtime_api.h>

#include "libnorm_dropout.h"

namespace libnorm {

constexpr int kDropMaxThreads = 512;
constexpr int kDropNarrow = 128;              // threads of a forward CTA that keeps LayerNorm's parameters in registers
constexpr int kDropMaxStages = 4;
constexpr int64_t kDropMaxSmem = 225 * 1024;  // dynamic, per CTA (beside the kernels' own few KB)
constexpr int kDropChain = 64;                // rows whose column terms are added one after the other, at most

struct DropArgs {
    const void *x, *residual;       // forward
    const void *dy, *dh, *hin;      // backward
    const void *gamma, *beta;
    void *h, *y;                    // forward
    void *dx, *dres;                // backward; dx: null without dropout
    float *mean, *rstd;             // written by the forward, read by the backward (LayerNorm)
    float* ws;                      // backward: partial rows [partials][partial_pitch]
    float *dgamma, *dbeta;
    const uint64_t* rng;            // seed, offset in device memory, or null:
    uint64_t seed, offset;
    int64_t M;
    int32_t N;
    int32_t lanes;                  // lanes of a warp per row; 0: a team of warps or a cluster
    int32_t team;                   // threads of a team
    int32_t cluster;
    int32_t partial_pitch;
    int32_t phases;                 // rows after which one begins at the same place of a 16-byte vector
    int32_t stat_bytes;             // means and rstds of a warp's rows of a step
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
    if (vec == 1) return !group && rows == 1 && per_thread == 8;
    if (vec * elem != 16) return false;
    if (group) return per_thread == 2 && rows == 2;
    if (per_thread == 1) return rows == 4 || (rows == 1 && !backward);
    return elem == 2 && backward ? per_thread == 2 && rows == 2 : per_thread == 4 && rows == 1;
}

// Threads of a CTA, at most: what 32 values of a thread need in registers
// leaves room for half as many.
inline int drop_max_threads(int vec, int per_thread) { return vec * per_thread >= 32 ? 256 : kDropMaxThreads; }

// Rows after which one begins at the same place of a vector, and the vectors
// that a row touches at most.
inline int drop_phases(int64_t N, int vec) {
    int n = 1;
    while (vec > 1 && n * N % vec != 0) n *= 2;
    return n;
}
// CTAs (or clusters) whose teams are a multiple of the phases.
inline int drop_grid_unit(int phases, int teams) {
    int n = 1;
    while (int64_t(n) * teams % phases != 0) n *= 2;
    return n;
}
inline int64_t drop_vectors(int64_t N, int vec) {
    const int64_t most = vec - vec / drop_phases(N, vec);  // elements before the row
    return (most + N + vec - 1) / vec;
}

// Columns of a CTA's part of a row.
inline int64_t drop_cta_cols(int vec, int per_thread, int threads) { return int64_t(threads) * per_thread * (vec == 1 ? 2 : vec); }

// Shared memory of the stages: of each thread's own accesses (and, `stats`
// bytes a warp, the rows' statistics), or of the CTA's part of a row of
// elements in whole 16-byte chunks at a pitch; of the masks' words of two rows
// of elements; of parameters; and of the backward's column sums of a CTA of
// several teams.
inline int64_t drop_pitch(int elem, int per_thread, int threads) { return (drop_cta_cols(1, per_thread, threads) * elem + 30) / 16 * 16; }
inline int64_t drop_ring_bytes(int vec, int elem, int per_thread, int threads, int rows, int stages, int streams, int stats) {
    return vec == 1 ? stages * streams * drop_pitch(elem, per_thread, threads)
                    : int64_t(stages) * threads / 32 * (int64_t(streams) * rows * per_thread * 512 + stats);
}
inline int drop_stat_bytes(bool ln, bool bwd, int vec, int lanes, int rows) {
    return ln && bwd && vec > 1 ? (32 / (lanes > 0 ? lanes : 32) * rows * 8 + 15) / 16 * 16 : 0;
}
inline int64_t drop_words_bytes(int vec, int per_thread, int threads) {
    return vec == 1 ? 2 * 16 * (drop_cta_cols(1, per_thread, threads) / 8 + 2) : 0;
}
inline int64_t drop_param_bytes(bool ln, int vec, int per_thread, int threads) {  // forward
    return ln && vec > 1 && per_thread == 4 && threads > kDropNarrow ? int64_t(per_thread) * threads * 16 : 0;
}
inline int64_t drop_sums_bytes(bool ln, int vec, int per_thread, int threads) {
    return int64_t(ln ? 2 : 1) * vec * per_thread * threads * 4;
}

// Floats from one partial row of column sums to the next.
inline int32_t drop_partial_pitch(int32_t values) { return (values + 3) / 4 * 4; }

cudaError_t launch_drop_fwd_f32(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_fwd_bf16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_fwd_f16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_bwd_f32(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_bwd_bf16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);
cudaError_t launch_drop_bwd_f16(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s);

// The sums of `partials` partial rows of columns: dgamma (and dbeta); zeros where there are none.
cudaError_t launch_drop_colsum(const DropArgs& a, int64_t partials, bool ln, cudaStream_t s);

}  // namespace libnorm
