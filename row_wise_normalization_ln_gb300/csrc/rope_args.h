// Argument block of the head norm + rotation kernels and their launchers,
// shared by the host side (rope.cpp) and the kernels (rope.cuh).
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "gn_args.h"
#include "libnorm_rope.h"

namespace libnorm {

constexpr int kRopeMaxD = 512;
constexpr int kRopeMaxWarps = 8;

constexpr int kRopeRing = 4;  // heads of a warp in flight or being worked on; a power of two
constexpr int64_t kRopeMaxSmem = 225 * 1024;

// Dynamic shared memory of a launch: the backward's sums and the lanes' slots
// (asynchronous copies take 4 bytes or more).
inline int64_t rope_smem_bytes(int vec, int elem, int pairs, int warps, bool backward) {
    const int64_t sums = backward ? int64_t(pairs) * 2 * (vec == 1 ? 2 : vec) * 4 : 0;
    const int64_t slots = vec * elem >= 4 ? int64_t(backward ? 2 : 1) * kRopeRing * pairs * 2 * vec * elem : 0;
    return int64_t(warps) * 32 * (sums + slots);
}

struct RopeSide {
    norm_heads x, dy, y;
    const void* w;
    float* dw;
    float* part;      // backward: partial rows of dw, [ctas][D]
    int32_t heads;
    int32_t chunks;   // tasks a token's heads are cut into
    int32_t tasks;    // blocks of 32 / lanes tokens times chunks
    int32_t ctas;
    FastDiv by_chunks;
};

struct RopeArgs {
    RopeSide side[2];  // queries, keys: CTAs [0, side[0].ctas) and those after
    const float *cos, *sin;
    const void* positions;
    int64_t table_pitch, P;
    int32_t pos_bytes;   // 8, 4, or 0: a token's position is its place in the sequence
    int32_t vec_table;   // table rows of whole 16 bytes on 16-byte boundaries
    int32_t T, S, D, R;
    int32_t lanes_log;   // log2 of the lanes per head
    int32_t npairs;      // pairs of accesses per head
    int32_t rot_pairs;   // the first of them that rotate (R / (2 VEC); interleaved vectors: unused)
    int32_t chunk_heads; // heads per task
    float eps, invD;
    FastDiv by_S;
};

// The two sides' CTAs of a persistent launch of at most `ctas`, by their
// heads, and the places of their partial rows (side[0].part: the first).
inline void rope_share(RopeArgs* a, int64_t ctas) {
    const int64_t h0 = a->side[0].heads, h1 = a->side[1].heads;
    const int64_t n = std::min<int64_t>(std::max<int64_t>(ctas, 2), int64_t(a->side[0].ctas) + a->side[1].ctas);
    int64_t first = (n * h0 + (h0 + h1) / 2) / (h0 + h1);
    if (h0 > 0 && h1 > 0) first = std::max<int64_t>(1, std::min(first, n - 1));
    a->side[0].ctas = static_cast<int32_t>(std::min<int64_t>(a->side[0].ctas, first));
    a->side[1].ctas = static_cast<int32_t>(std::min<int64_t>(a->side[1].ctas, n - first));
    a->side[1].part = a->side[0].part + int64_t(a->side[0].ctas) * a->D;
}

// (A persistent launch takes no more CTAs than fit on the device at once:
// `a` then says how many it took.)
cudaError_t launch_rope_f32(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s);
cudaError_t launch_rope_bf16(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s);
cudaError_t launch_rope_f16(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s);

// Column sums of the partial rows: dw of both sides.
cudaError_t launch_rope_colsum(const RopeArgs& a, cudaStream_t s);

}  // namespace libnorm
