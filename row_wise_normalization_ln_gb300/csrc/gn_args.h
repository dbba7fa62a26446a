// Argument block of the group norm kernels and their launchers, shared by the
// host side (gn.cpp) and the kernels (gn_kernels.cuh).
#pragma once

#include <cstdint>

#include <cuda_runtime_api.h>

#include "libnorm_group.h"

namespace libnorm {

constexpr int kGnMaxThreads = 256;
// Channels of a tile whose accesses span groups (their sums are kept per
// channel): bounds the shared memory of the reductions.
constexpr int kGnMaxMixedChannels = 512;

// Division of n in [0, 2^31) by a fixed d >= 1: n / d = (mulhi(n, m) + n) >> s
// with s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1 (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994).
struct FastDiv {
    uint32_t m, s;
};
inline FastDiv fast_div(int64_t d) {
    uint32_t s = 0;
    while ((int64_t(1) << s) < d) ++s;
    const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << s) - static_cast<uint64_t>(d))) / static_cast<uint64_t>(d) + 1;
    return FastDiv{static_cast<uint32_t>(m), s};
}

struct GnArgs {
    const void* x;
    const void* dy;        // backward
    const void* gamma;
    const void* beta;
    void* y;               // forward: y; backward: dx
    float* mean;           // [B, G]: written by the forward, read by the backward
    float* rstd;
    float* shift;          // SPLIT forward: [B, G], the groups' first elements
    void* part;            // SPLIT: [B, G, tpg, chunks] group states of the row chunks (float4; backward float2)
    float* colg;           // backward: partial rows of dgamma and dbeta, [partials] rows of C values at a
    float* colb;           // pitch of col_pitch (dgamma and dbeta themselves where one partial row is all)
    int64_t S;
    int64_t xb, xr, dyb, dyr, yb, yr;  // pitches in elements
    int64_t col_pitch;
    int32_t C, G, D;
    int32_t ncols;         // accesses per row: C / VEC
    int32_t tile;          // accesses of a row per CTA
    int32_t tiles;         // tiles per row
    int32_t tpg;           // tiles a group may touch (1 when tiles are whole groups)
    int32_t segs;          // groups an access may touch
    int32_t par;           // rows a CTA works on at once: threads / tile
    int32_t cluster, cluster_bits;  // CHIP: CTAs per sample and tile
    int32_t join;          // CHIP backward: samples in one cluster (all of them), or 1
    int32_t chunks;        // row chunks summed per sample and tile
    int32_t out_chunks;    // row chunks written per sample and tile
    int64_t chunk_rows;    // rows per summed chunk (CHIP: per CTA of the cluster)
    int64_t out_rows;      // rows per written chunk
    int32_t partials;      // partial rows of the column gradients
    int32_t folds;         // rows they are added to first where they are many, otherwise 0
    float* fold;           // [folds, 2 C]
    int32_t ring_at;       // SPLIT: where the row stream's slots start in shared memory, in 16-byte units
    float *dgamma, *dbeta;
    FastDiv by_cluster;
    FastDiv by_tiles, by_tile, by_D, by_par, by_chunks, by_out_chunks;
    float eps;
};

// Dynamic shared memory of a kernel, from its plan: per group and warp that
// shares the group, a state (16 bytes, at most one per warp or per group); per
// group, 12 bytes of values; the per-thread states ([par][units]). (The
// column adders of the backward keep 8 bytes per thread.) `units`: states per
// row slot; tile * segs in the forward, tile * vec_elems in the backward,
// whose column sums are per channel. A multiple of
// 128 bytes, so that a warp's slots of the row stream (behind it) take whole
// wavefronts (on 16 bytes: gn_bwd bf16 4x65536x256 119 us instead of 104).
inline int64_t gn_smem_bytes(int par, int units, int groups, int threads) {
    const int64_t shared = groups > threads / 32 ? groups : threads / 32;
    const int64_t merge = int64_t(par) * units * 8 + shared * 16 + int64_t(groups) * 12 + 16;
    return ((merge > int64_t(threads) * 8 ? merge : int64_t(threads) * 8) + 127) / 128 * 128;
}

// Groups a tile of `channels` channels can touch.
inline int64_t gn_tile_groups(int64_t channels, int64_t D, bool whole) {
    return whole ? channels / D : (channels - 1 + D - 1) / D + 1;
}

cudaError_t launch_gn_fwd_f32(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s);
cudaError_t launch_gn_fwd_bf16(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s);
cudaError_t launch_gn_fwd_f16(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s);
cudaError_t launch_gn_bwd_f32(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s);
cudaError_t launch_gn_bwd_bf16(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s);
cudaError_t launch_gn_bwd_f16(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s);

}  // namespace libnorm
