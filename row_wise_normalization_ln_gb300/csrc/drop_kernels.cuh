// Building blocks of the dropout + residual add + norm kernels, forward
// (drop_fwd.cuh) and backward (drop_bwd.cuh).
//
// Rows are walked by persistent CTAs, R neighbouring ones at a time (the cost
// of a step, its barrier, sums and addresses, is that of many elements). A row
// belongs to some lanes of a warp (short rows), a CTA, or a cluster of CTAs; a
// thread owns the same columns in every row it visits, so the parameters and,
// in the backward, the column sums stay in its registers.
//
// Rows of whole 16-byte vectors: a thread's values come in accesses of 16
// bytes, through a ring of shared memory that it fills and reads for itself
// with asynchronous copies (DropRing): no barrier and no registers while they
// travel. Other rows (odd widths, any offset): the CTA copies the aligned 16
// bytes that hold its part of a row together (DropStage), and a thread takes
// its elements, every 32nd of its warp's, from there; what it stores goes out
// element by element.
//
// The mask is computed where it is used: one call of the generator for 8
// elements. On 16-bit rows that is an access, on fp32 rows half of the call is
// used, rows of elements share the calls of the CTA through shared memory.
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

// ------------------------------------------------------------ accesses
// What a thread takes at a time, as fp32 pairs: a 16-byte vector, or (VEC 1)
// two elements of its warp's run, 32 apart.
template <class T, int VEC>
struct DropVec : GnVec<T, VEC> {};
template <class T>
struct DropVec<T, 1> {
    using E = GnVec<T, 1>;
    struct Raw {
        uint32_t lo, hi;
    };
    static constexpr int H = 1;
    static __device__ __forceinline__ Raw zero() { return Raw{0, 0}; }
    static __device__ __forceinline__ float2 get(const Raw& r, int) { return make_float2(E::get(r.lo, 0).x, E::get(r.hi, 0).x); }
    static __device__ __forceinline__ void set(Raw& r, int, float2 v) {
        if constexpr (sizeof(T) == 4) {
            r.lo = __float_as_uint(v.x);
            r.hi = __float_as_uint(v.y);
        } else {
            const uint32_t w = Gn16<T>::Pair::pack(v.x, v.y);
            r.lo = w & 0xffff;
            r.hi = w >> 16;
        }
    }
};

// A thread's place: its columns, and how far its accesses lie apart.
template <int VEC, int V, bool GROUP>
struct DropPlace {
    static constexpr int kRun = VEC == 1 ? 64 * V : 32 * V * VEC;  // columns of a warp's run
    int unit;        // lanes that share sums by butterflies: those of a row, or a warp
    int col, step;   // first column; columns from one access to the next
    int nv;          // accesses that lie within the row; VEC 1: elements
    int warps;       // warps of a CTA that share a row
    int rank, C;
    int64_t block, blocks_step;  // blocks of R rows: the first, from one to the next
    bool first;                  // writes the row's statistics

    __device__ __forceinline__ explicit DropPlace(const DropArgs& a) {
        const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31;
        C = GROUP ? 1 : a.cluster;
        rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
        if constexpr (GROUP) {
            unit = a.lanes;
            warps = 1;
            col = (tid & (unit - 1)) * VEC;
            step = unit * VEC;
            const int teams = T / unit;
            block = static_cast<int64_t>(blockIdx.x) * teams + tid / unit;
            blocks_step = static_cast<int64_t>(gridDim.x) * teams;
            first = col == 0;
        } else {
            unit = 32;
            warps = T >> 5;
            col = (rank * warps + (tid >> 5)) * kRun + lane * VEC;
            step = 32 * VEC;
            block = blockIdx.x / C;
            blocks_step = gridDim.x / C;
            first = rank == 0 && tid == 0;
        }
        nv = col < a.N ? min(VEC == 1 ? 2 * V : V, (a.N - col + step - 1) / step) : 0;
    }
    __device__ __forceinline__ bool on(int j) const { return (VEC == 1 ? 2 * j : j) < nv; }
    // Columns from the first to access j (a constant but where lanes share rows).
    __device__ __forceinline__ int at(int j) const { return VEC == 1 ? 64 * j : GROUP ? j * step : 32 * VEC * j; }
    // Loads and stores of a row's access straight from memory; p: the first column's element.
    template <class T>
    __device__ __forceinline__ typename DropVec<T, VEC>::Raw load(const T* p, int j) const {
        if constexpr (VEC == 1) {
            using E = GnVec<T, 1>;
            typename DropVec<T, 1>::Raw r = DropVec<T, 1>::zero();
            if (2 * j < nv) r.lo = E::load(p + at(j));
            if (2 * j + 1 < nv) r.hi = E::load(p + at(j) + 32);
            return r;
        } else {
            return DropVec<T, VEC>::load(p + at(j));
        }
    }
    template <class T>
    __device__ __forceinline__ void store(T* p, int j, const typename DropVec<T, VEC>::Raw& r) const {
        if constexpr (VEC == 1) {
            using E = GnVec<T, 1>;
            if (2 * j < nv) E::store(p + at(j), r.lo);
            if (2 * j + 1 < nv) E::store(p + at(j) + 32, r.hi);
        } else {
            DropVec<T, VEC>::store(p + at(j), r);
        }
    }
    // Elements of warp w of CTA k of the cluster.
    static __device__ __forceinline__ float count(const DropArgs& a, int k, int w) {
        const int at = (k * static_cast<int>(blockDim.x >> 5) + w) * kRun;
        return static_cast<float>(max(0, min(a.N - at, kRun)));
    }
    static __device__ __forceinline__ float count_cta(const DropArgs& a, int k) {
        const int run = static_cast<int>(blockDim.x >> 5) * kRun;
        return static_cast<float>(max(0, min(a.N - k * run, run)));
    }
};

// ------------------------------------------------------------ sums
// Sums of K values (1, 2, 4 or 8) over a warp, transposed on the way: lane l
// ends with the sum of value l / (32 / K), the same in its whole block of
// lanes. log2 K steps that halve the values, then single butterflies: 6
// exchanges for 4 values instead of 20.
template <int K>
__device__ __forceinline__ float warp_sums(const float (&in)[K]) {
    float v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = in[k];
    int off = 16;
#pragma unroll
    for (int n = K; n > 1; n /= 2, off /= 2) {
        const bool up = (threadIdx.x & off) != 0;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float keep = up ? v[k + n / 2] : v[k], give = up ? v[k] : v[k + n / 2];
            v[k] = keep + __shfl_xor_sync(kFullMask, give, off);
        }
    }
#pragma unroll
    for (; off > 0; off /= 2) v[0] += __shfl_xor_sync(kFullMask, v[0], off);
    return v[0];
}

// K values of each warp of a CTA, and of each CTA of a cluster; slots
// alternate by parity, so that one is written again only after a barrier that
// every reader of its last values has passed.
template <int K>
struct DropSums {
    float warp[2][K][kDropMaxThreads / 32];  // those of warps that are not there stay 0
    float cta[2][K];
    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < 2 * K * (kDropMaxThreads / 32); i += blockDim.x) (&warp[0][0][0])[i] = 0.f;
        __syncthreads();
    }
};

__device__ __forceinline__ float drop_peer(const float* p, uint32_t rank) { return ld_peer_f32(peer_smem_addr(p, rank)); }

// How the lanes of a warp share the K x 16 values of the warps: LPI lanes per
// value, FPL of its warps each.
template <int K>
struct DropShare {
    static constexpr int kLanes = K == 1 ? 16 : 32 / K;
    static constexpr int kEach = (kDropMaxThreads / 32) / kLanes;
    int idx, w0;
    __device__ __forceinline__ DropShare() {
        const int lane = threadIdx.x & 31;
        idx = K == 1 ? 0 : lane / kLanes;
        w0 = (lane & (kLanes - 1)) * kEach;
    }
};

// Sums over the row of K values per thread; every thread gets all of them.
template <int K, class P>
__device__ __forceinline__ void drop_sum(DropSums<K>& sm, const P& p, int parity, float (&v)[K]) {
    constexpr int L = 32 / K;
    if (p.unit < 32) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = group_sum(v[k], p.unit);
        return;
    }
    const int lane = threadIdx.x & 31;
    float s = warp_sums<K>(v);
    int from = L;  // lanes between the values
    if (p.warps > 1) {
        if ((lane & (L - 1)) == 0) sm.warp[parity][lane / L][threadIdx.x >> 5] = s;
        __syncthreads();
        const DropShare<K> sh;
        const float* w = &sm.warp[parity][sh.idx][sh.w0];
        s = 0.f;
#pragma unroll
        for (int i = 0; i < DropShare<K>::kEach; ++i) s += w[i];
#pragma unroll
        for (int off = DropShare<K>::kLanes / 2; off > 0; off /= 2) s += __shfl_xor_sync(kFullMask, s, off);
        from = DropShare<K>::kLanes;
    }
    if (p.C > 1) {
        // value idx of this CTA, then the CTAs' in rank order
        if (threadIdx.x < 32 && (lane & (L - 1)) == 0) sm.cta[parity][lane / L] = s;
        cluster_barrier();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t = lane < p.C ? drop_peer(&sm.cta[parity][k], static_cast<uint32_t>(lane)) : 0.f;
            t = group_sum(t, 8);
            v[k] = __shfl_sync(kFullMask, t, 0);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(kFullMask, s, K == 1 ? 0 : k * from);
}

// ------------------------------------------------------------ the ring
// NS tensors' accesses of upcoming blocks of R rows, each thread its own.
template <class T, int VEC, int V, int R, int NS, class P>
struct DropRing {
    using Raw = typename DropVec<T, VEC>::Raw;
    static constexpr int kStage = R * NS * V * 32 * 16;  // of a warp
    const T* p[NS];      // this thread's first access of the next block to send (null: a tensor that is not there)
    int64_t step;        // elements from one block to the next
    int64_t rows;        // rows from the next block to send to the end
    int64_t rows_step;
    uint32_t base, at_send, at_read, end;
    int stages, N;

    __device__ __forceinline__ DropRing(const DropArgs& a, const P& pl, void* smem, const void* const (&from)[NS])
        : stages(a.stages), N(a.N) {
        rows_step = pl.blocks_step * R;
        step = rows_step * a.N;
        rows = a.M - pl.block * R;
#pragma unroll
        for (int n = 0; n < NS; ++n) p[n] = from[n] ? static_cast<const T*>(from[n]) + pl.block * R * a.N + pl.col : nullptr;
        base = smem_addr(smem) + (threadIdx.x >> 5) * stages * kStage + (threadIdx.x & 31) * 16;
        end = base + stages * kStage;
        at_send = at_read = base;
        for (int i = 0; i < stages - 1; ++i) send(pl);
    }
    // Sends the next block; a group of copies is committed even when none is left.
    __device__ __forceinline__ void send(const P& pl) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < rows) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    if (p[n]) {
                        const T* q = p[n] + r * N;
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (pl.on(j)) copy_async<16>(at_send + ((r * NS + n) * V + j) * 512, q + pl.at(j));
                    }
            }
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (p[n]) p[n] += step;
        rows -= rows_step;
        copy_async_commit();
        at_send = at_send + kStage == end ? base : at_send + kStage;
    }
    __device__ __forceinline__ void wait() const {
        if (stages == 2) copy_async_wait<0>();
        else if (stages == 3) copy_async_wait<1>();
        else copy_async_wait<2>();
    }
    // Access j of tensor n of row r of the block that was waited for.
    __device__ __forceinline__ Raw get(int r, int n, int j) const {
        Raw v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(at_read + ((r * NS + n) * V + j) * 512)
                     : "memory");
        return v;
    }
    __device__ __forceinline__ void advance() { at_read = at_read + kStage == end ? base : at_read + kStage; }
};

// Rows of any width and offset: the CTA's part of a row of NS tensors, as the
// aligned 16-byte chunks that hold it. A chunk starts no earlier than its
// allocation does (those start on larger boundaries), and bytes behind the
// part are not read. Rows are sent together, and read after a barrier that
// follows every thread's wait for its copies.
template <class T, int NS>
struct DropStage {
    static constexpr int kE = static_cast<int>(sizeof(T));
    const char* p[NS];  // the CTA's first element of the first row, or null
    int64_t rows_step, M, first;
    int N, cols, pitch, stages;
    uint32_t base;
    char* smem;

    __device__ __forceinline__ DropStage(const DropArgs& a, int64_t row, int64_t rows_step_, int c0, int cols_, char* smem_,
                                         const void* const (&from)[NS])
        : rows_step(rows_step_), M(a.M), first(row), N(a.N), cols(cols_), pitch(a.pitch), stages(a.stages), base(smem_addr(smem_)), smem(smem_) {
#pragma unroll
        for (int n = 0; n < NS; ++n) p[n] = from[n] ? static_cast<const char*>(from[n]) + static_cast<int64_t>(c0) * kE : nullptr;
    }
    __device__ __forceinline__ const char* row_of(int n, int64_t it) const { return p[n] + (first + it * rows_step) * N * kE; }
    __device__ __forceinline__ int slot(int64_t it) const { return static_cast<int>(it % stages) * (NS * pitch); }
    __device__ __forceinline__ void send(int64_t it) {
        if (first + it * rows_step < M && cols > 0) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (p[n]) {
                    const char* q = row_of(n, it);
                    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(q) & 15);
                    const int bytes = lead + cols * kE;
                    const uint32_t to = base + slot(it) + n * pitch;
                    for (int c = threadIdx.x * 16; c < bytes; c += blockDim.x * 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + c), "l"(q - lead + c), "r"(min(16, bytes - c)) : "memory");
                }
        }
        copy_async_commit();
    }
    // Where the CTA's first element of tensor n of a row lies in shared memory.
    __device__ __forceinline__ const T* row(int n, int64_t it) const {
        const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(row_of(n, it)) & 15);
        return reinterpret_cast<const T*>(smem + slot(it) + n * pitch + lead);
    }
    template <class P>
    static __device__ __forceinline__ typename DropVec<T, 1>::Raw get(const P& pl, const T* s, int j) {
        return pl.load(s, j);
    }
};

// ------------------------------------------------------------ masks of a row
// The words of access j of a row: `group` is the generator's group of the
// thread's first element (vectors of fp32: half groups).
template <int VEC>
struct DropWords {
    uint4 w;
    __device__ __forceinline__ void take(const DropMask& m, uint64_t group) {
        if constexpr (VEC == 8) w = m.words(group);
        if constexpr (VEC == 4) {
            const uint4 t = m.words(group >> 1);
            w.x = (group & 1) ? t.z : t.x;
            w.y = (group & 1) ? t.w : t.y;
        }
    }
    // VEC 1: two elements' words
    __device__ __forceinline__ void take(const unsigned short* s) { w.x = s[0] | static_cast<uint32_t>(s[32]) << 16; }
    __device__ __forceinline__ bool lo(const DropMask& m, int i) const { return m.low(drop_word(w, i)); }
    __device__ __forceinline__ bool hi(const DropMask& m, int i) const { return m.high(drop_word(w, i)); }
};

// The words of `cols` elements from flat element e on, by the CTA together;
// element e + i's is word (e & 7) + i.
__device__ __forceinline__ void drop_stage_words(const DropMask& m, uint64_t e, int cols, uint4* to) {
    const uint64_t g0 = e >> 3;
    const int n = static_cast<int>(((e + cols + 7) >> 3) - g0);
    for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = m.words(g0 + i);
}

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
