// Argument block of the head norm + rotation kernels and their launchers,
// shared by the host side (rope.cpp) and the kernels (rope.cuh).
#pragma once

#include <cstdint>

#include <cuda_runtime_api.h>

#include "gn_args.h"
#include "libnorm_rope.h"

namespace libnorm {

constexpr int kRopeMaxD = 512;
constexpr int kRopeMaxWarps = 8;

struct RopeSide {
    norm_heads x, dy, y;
    const void* w;
    float* dw;
    float* part;      // backward: partial rows of dw, [ctas][D]
    int32_t heads;
    int32_t slots;    // groups of 32 / lanes heads
    int32_t chunks;   // warps a token's heads are shared by
    int32_t tasks;    // tokens * chunks
    int32_t ctas;
    FastDiv by_chunks;
};

struct RopeArgs {
    RopeSide side[2];  // queries, keys: CTAs [0, side[0].ctas) and those after
    const float *cos, *sin;
    const void* positions;
    int64_t table_pitch, P;
    int32_t pos_bytes;   // 8, 4, or 0: a token's position is its place in the sequence
    int32_t vec_table;   // table rows on 16-byte boundaries
    int32_t S, D, R;
    int32_t lanes_log;   // log2 of the lanes per head
    int32_t npairs;      // pairs of accesses per head
    int32_t rot_pairs;   // the first of them that rotate (R / (2 VEC); interleaved vectors: unused)
    int32_t chunk_slots; // slots per task
    float eps, invD;
    FastDiv by_S;
};

cudaError_t launch_rope_f32(const norm_rope_plan& p, const RopeArgs& a, bool interleaved, bool backward, cudaStream_t s);
cudaError_t launch_rope_bf16(const norm_rope_plan& p, const RopeArgs& a, bool interleaved, bool backward, cudaStream_t s);
cudaError_t launch_rope_f16(const norm_rope_plan& p, const RopeArgs& a, bool interleaved, bool backward, cudaStream_t s);

// Column sums of the partial rows: dw of both sides.
cudaError_t launch_rope_colsum(const RopeArgs& a, cudaStream_t s);

}  // namespace libnorm
