// Building blocks of the dropout + residual add + norm kernels, forward
// (drop_fwd.cuh) and backward (drop_bwd.cuh).
//
// Rows are walked by persistent CTAs. A row belongs to some lanes of a warp
// (short rows), a CTA, or a cluster of CTAs; a thread owns the same columns in
// every row it visits, so the parameters and, in the backward, the column sums
// stay in its registers. Upcoming rows travel through a ring of shared memory
// that every thread fills and reads for itself with asynchronous copies of its
// own accesses: no barrier and no registers while they travel. The mask is
// computed where it is used: one call of the generator for 8 elements, which
// are one access of a 16-bit row, half of the calls' outputs used on fp32
// rows; element accesses share the calls of a warp through shared memory.
#pragma once

#include "drop_args.h"
#include "gn_kernels.cuh"

namespace libnorm {

// ------------------------------------------------------------ the mask
// Philox4x32-7 (Salmon et al. 2011): 7 rounds of two 32 x 32 bit products, the
// key stepped by Weyl constants.
struct DropMask {
    uint32_t k0, k1, c2, c3, limit;
    __device__ __forceinline__ explicit DropMask(const DropArgs& a) {
        uint64_t seed = a.seed, offset = a.offset;
        if (a.rng) {
            seed = __ldg(reinterpret_cast<const unsigned long long*>(a.rng));
            offset = __ldg(reinterpret_cast<const unsigned long long*>(a.rng) + 1);
        }
        k0 = static_cast<uint32_t>(seed);
        k1 = static_cast<uint32_t>(seed >> 32);
        c2 = static_cast<uint32_t>(offset);
        c3 = static_cast<uint32_t>(offset >> 32);
        limit = a.limit;
    }
    __device__ __forceinline__ uint4 words(uint64_t group) const {
        uint32_t x0 = static_cast<uint32_t>(group), x1 = static_cast<uint32_t>(group >> 32), x2 = c2, x3 = c3;
        uint32_t a = k0, b = k1;
#pragma unroll
        for (int r = 0; r < 7; ++r) {
            const uint64_t p = static_cast<uint64_t>(x0) * 0xD2511F53u, q = static_cast<uint64_t>(x2) * 0xCD9E8D57u;
            x0 = static_cast<uint32_t>(q >> 32) ^ x1 ^ a;
            x2 = static_cast<uint32_t>(p >> 32) ^ x3 ^ b;
            x1 = static_cast<uint32_t>(q);
            x3 = static_cast<uint32_t>(p);
            a += 0x9E3779B9u;
            b += 0xBB67AE85u;
        }
        return make_uint4(x0, x1, x2, x3);
    }
    // The 16-bit words of a 32-bit one against the limit, which is in the high half.
    __device__ __forceinline__ bool low(uint32_t w) const { return (w << 16) >= limit; }
    __device__ __forceinline__ bool high(uint32_t w) const { return w >= limit; }
};

__device__ __forceinline__ uint32_t drop_word(const uint4& w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }

// ------------------------------------------------------------ a thread's place
struct DropPlace {
    int unit;        // lanes that share sums by butterflies: those of a row, or a warp
    int f0, step;    // first access within the row, from one to the next
    int nv;          // accesses that lie within the row
    int64_t row, rows_step;
    int64_t iters;   // rows the CTA's first team visits (the others' last may lie beyond M)
    bool first;      // writes the row's statistics
    int warps;       // warps of a CTA that share a row (1: a row's lanes lie in one warp)
    int rank, C;

    template <int VEC, int V>
    __device__ __forceinline__ void set(const DropArgs& a) {
        const int T = blockDim.x, tid = threadIdx.x;
        const int nacc = (a.N + VEC - 1) / VEC;
        C = a.cluster;
        rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
        int64_t first_row;
        if (a.lanes > 0) {
            unit = a.lanes;
            warps = 1;
            const int teams = T / unit;
            f0 = tid & (unit - 1);
            step = unit;
            first_row = static_cast<int64_t>(blockIdx.x) * teams;
            row = first_row + tid / unit;
            rows_step = static_cast<int64_t>(gridDim.x) * teams;
            first = f0 == 0;
        } else {
            unit = 32;
            warps = T >> 5;
            f0 = (rank * T + (tid >> 5 << 5)) * V + (tid & 31);
            step = 32;
            first_row = row = blockIdx.x / C;
            rows_step = gridDim.x / C;
            first = rank == 0 && tid == 0;
        }
        nv = f0 < nacc ? min(V, (nacc - f0 + step - 1) / step) : 0;
        iters = first_row < a.M ? (a.M - first_row + rows_step - 1) / rows_step : 0;
    }
};

// ------------------------------------------------------------ sums
// Two values per thread, over the row; every thread gets the same bits. One
// barrier of the CTA per call (and one of the cluster); slots alternate by
// `parity`, so that a slot is written again only after a barrier that every
// reader of its last value has passed.
struct DropSums {
    float2 warp[2][kDropMaxThreads / 32];
    float2 cta[2];
};

__device__ __forceinline__ float2 drop_peer(const float2* p, uint32_t rank) {
    float2 v;
    const uint32_t at = peer_smem_addr(p, rank);
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ int drop_pow2(int n) {
    int w = 1;
    while (w < n) w <<= 1;
    return w;
}

// Plain sums of both values.
__device__ __forceinline__ float2 drop_sum(DropSums& sm, const DropPlace& p, int parity, float2 v) {
    group_sum2(v.x, v.y, p.unit);
    if (p.warps > 1) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) sm.warp[parity][threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < p.warps ? sm.warp[parity][lane] : make_float2(0.f, 0.f);
        group_sum2(v.x, v.y, 16);  // (at most 16 warps: both halves have the sum of the first 16 lanes or of none)
        v.x = __shfl_sync(kFullMask, v.x, 0);
        v.y = __shfl_sync(kFullMask, v.y, 0);
    }
    if (p.C > 1) {
        const int lane = threadIdx.x & 31;
        if (threadIdx.x == 0) sm.cta[parity] = v;
        cluster_barrier();
        v = lane < p.C ? drop_peer(&sm.cta[parity], static_cast<uint32_t>(lane)) : make_float2(0.f, 0.f);
        group_sum2(v.x, v.y, 8);
        v.x = __shfl_sync(kFullMask, v.x, 0);
        v.y = __shfl_sync(kFullMask, v.y, 0);
    }
    return v;
}

// The merge of states (n, sum, M2 about the state's own mean) of the lanes
// [0, width), by the rule in its k-way form: mean = sum / n in all and
// M2 = sum (M2_i + n_i (mean_i - mean)^2). Returns (sum, M2) in every lane.
__device__ __forceinline__ float2 drop_merge(float n, float2 v, float inv_all, int width) {
    const float total = __shfl_sync(kFullMask, group_sum(v.x, width), 0);
    const float d = (n > 0.f ? v.x / n : 0.f) - total * inv_all;
    const float m2 = __shfl_sync(kFullMask, group_sum(fmaf(n * d, d, v.y), width), 0);
    return make_float2(total, m2);
}

// ------------------------------------------------------------ the ring
// NS tensors' accesses of upcoming rows, each thread its own.
template <class T, int VEC, int V, int NS>
struct DropRing {
    using X = GnVec<T, VEC>;
    using Raw = typename X::Raw;
    static constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
    static constexpr bool kAsync = kBytes >= 4;
    static constexpr int kAccess = 32 * kBytes;
    static constexpr int kStage = NS * V * kAccess;  // of a warp
    const T* p[NS];      // this thread's first access of the next row to send (null: a tensor that is not there)
    int64_t step;        // elements from one row to the next
    int64_t left;        // rows not yet sent, this thread's
    uint32_t base, at_send, at_read, end;
    int stages, nv, acc;  // acc: elements from one access to the next
    Raw next[kAsync ? 1 : NS][kAsync ? 1 : V];

    __device__ __forceinline__ DropRing(const DropArgs& a, const DropPlace& pl, void* smem, const void* const (&from)[NS])
        : stages(a.stages), nv(pl.nv), acc(pl.step * VEC) {
        step = pl.rows_step * a.N;
        left = pl.row < a.M ? (a.M - pl.row + pl.rows_step - 1) / pl.rows_step : 0;
#pragma unroll
        for (int n = 0; n < NS; ++n)
            p[n] = from[n] ? static_cast<const T*>(from[n]) + pl.row * a.N + static_cast<int64_t>(pl.f0) * VEC : nullptr;
        if constexpr (kAsync) {
            base = smem_addr(smem) + (threadIdx.x >> 5) * stages * kStage + (threadIdx.x & 31) * kBytes;
            end = base + stages * kStage;
            at_send = at_read = base;
            for (int i = 0; i < stages - 1; ++i) send();
        } else {
            send();
        }
    }
    // Sends (or loads) the next row; a group of copies is committed even when none is left.
    __device__ __forceinline__ void send() {
        if (left > 0) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (p[n]) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (j < nv) {
                            if constexpr (kAsync)
                                copy_async<kBytes>(at_send + (n * V + j) * kAccess, p[n] + j * acc);
                            else
                                next[n][j] = X::load(p[n] + j * acc);
                        }
                    p[n] += step;
                }
            --left;
        }
        if constexpr (kAsync) {
            copy_async_commit();
            at_send = at_send + kStage == end ? base : at_send + kStage;
        }
    }
    // Access j of tensor n of the row that was waited for.
    __device__ __forceinline__ Raw get(int n, int j) const {
        if constexpr (!kAsync) {
            return next[n][j];
        } else {
            Raw r;
            const uint32_t at = at_read + (n * V + j) * kAccess;
            if constexpr (kBytes == 16)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
            else
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
            return r;
        }
    }
    __device__ __forceinline__ void wait() const {
        if constexpr (kAsync) {
            if (stages == 2) copy_async_wait<0>();
            else if (stages == 3) copy_async_wait<1>();
            else copy_async_wait<2>();
        }
    }
    // On to the next row: its slot is the one that `send` fills next but one.
    __device__ __forceinline__ void advance() {
        if constexpr (kAsync) at_read = at_read + kStage == end ? base : at_read + kStage;
    }
};

// ------------------------------------------------------------ masks of a row
// keep(j, i): whether pair i of elements of access j is kept, both of it.
template <class T, int VEC, int V>
struct DropRowMask {
    const DropMask& m;
    const bool on;
    uint64_t group;   // VEC > 1: of the thread's first access; in halves for fp32 rows
    int acc;          // accesses from one to the next
    const unsigned short* words;  // VEC == 1: this thread's first element's word
    uint4 w;

    __device__ __forceinline__ DropRowMask(const DropMask& m_, bool on_, const DropArgs& a, const DropPlace& p, int64_t row, uint4* smem)
        : m(m_), on(on_), acc(p.step), words(nullptr) {
        if constexpr (VEC > 1) {
            group = static_cast<uint64_t>(row) * static_cast<uint32_t>(a.N / VEC) + static_cast<uint32_t>(p.f0);
        } else if (on) {
            // The words of the unit's columns, computed together: those of the
            // last row are no longer read, and those of this one complete
            // before they are.
            const int u = threadIdx.x & (p.unit - 1), per = (p.unit * V + 7) / 8 + 2;
            uint4* mine = smem + (threadIdx.x / p.unit) * per;
            const int64_t e = row * a.N + (p.f0 - u);
            const uint64_t g0 = static_cast<uint64_t>(e) >> 3;
            __syncwarp();
            for (int g = u; g < per; g += p.unit) mine[g] = m.words(g0 + g);
            __syncwarp();
            words = reinterpret_cast<const unsigned short*>(mine) + (e & 7) + u;
        }
    }
    __device__ __forceinline__ void access(int j) {
        if (!on) return;
        if constexpr (VEC == 8) w = m.words(group + j * acc);
        if constexpr (VEC == 4) {
            const uint64_t g = group + j * acc;
            const uint4 t = m.words(g >> 1);
            w.x = (g & 1) ? t.z : t.x;
            w.y = (g & 1) ? t.w : t.y;
        }
        if constexpr (VEC == 1) w.x = words[j * acc];
    }
    __device__ __forceinline__ bool lo(int i) const { return !on || m.low(drop_word(w, i)); }
    __device__ __forceinline__ bool hi(int i) const { return VEC > 1 && (!on || m.high(drop_word(w, i))); }
};

// ------------------------------------------------------------ launch
inline cudaError_t drop_resident(const void* fn, int threads, size_t smem, int cluster, int64_t* out) try {
    static std::mutex mu;
    static std::map<std::tuple<const void*, int, size_t, int, int>, int64_t> cache;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (smem > 16 * 1024) {
        e = gn_opt_in(fn);
        if (e != cudaSuccess) return e;
    }
    std::lock_guard<std::mutex> lock(mu);
    int64_t& n = cache[{fn, threads, smem, cluster, dev}];
    if (n == 0) {
        int per = 0;
        if (cluster > 1) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(cluster));
            cfg.blockDim = dim3(static_cast<unsigned>(threads));
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(cluster);
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&per, fn, &cfg);
            n = int64_t(per) * cluster;
        } else {
            int sms = 0;
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, threads, smem);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            n = int64_t(per) * sms;
        }
        if (e != cudaSuccess) {
            n = 0;
            return e;
        }
    }
    *out = n;
    return n > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
} catch (...) {  // (no exception leaves a C entry point)
    return cudaErrorMemoryAllocation;
}

inline cudaError_t drop_launch(const void* fn, int64_t grid, int threads, size_t smem, int cluster, cudaStream_t s, const DropArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    void* args[] = {const_cast<DropArgs*>(&a)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace libnorm
