// Building blocks of the dropout + residual add + norm kernels, forward
// (drop_fwd.cuh) and backward (drop_bwd.cuh).
//
// Rows are walked by persistent CTAs, R neighbouring ones at a time (the cost
// of a step, its barrier, sums and addresses, is that of many elements). A row
// belongs to a team: some lanes of a warp (short rows), warps, or a cluster; a
// thread owns the same columns in every row it visits, so the parameters and,
// in the backward, the column sums stay in its registers.
//
// A thread's values come in accesses of 16 aligned bytes, through a ring of
// shared memory that it fills and reads for itself with asynchronous copies
// (DropRing): no barrier and no registers while they travel. Rows that are no
// whole number of vectors begin in the middle of one; where, depends on the
// row's number modulo a.phases (2, 4 or 8). A team takes rows of one phase
// alone, so that its threads own the same columns in all of them, shifted by
// `lead` elements, and only the warps that hold an end of the row look at
// single elements. (Before, such rows went through shared memory element by
// element: LayerNorm bf16 4096 x 5001 forward 75 us.) Pointers that
// are not 16-byte aligned still do: the CTA copies the aligned 16 bytes that
// hold its part of a row together (DropStage), and a thread takes its
// elements, every 32nd of its warp's, from there.
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
    // LEAN: the rounds' keys are formed for each call (two additions a round),
    // rather than kept in 14 registers, which LayerNorm's kernels lack (bf16
    // 4096 x 8192 forward 60 -> 48 us, backward 87 -> 73) and RMSNorm's do not
    // (forward 65536 x 2048 177 us with additions, 165 without).
    template <bool LEAN>
    __device__ __forceinline__ uint4 words(uint64_t group) const {
        uint32_t x0 = static_cast<uint32_t>(group), x1 = static_cast<uint32_t>(group >> 32), x2 = c2, x3 = c3;
        uint32_t a = k0, b = k1;
        if (LEAN) asm volatile("" : "+r"(a), "+r"(b));
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
// a b + c and a + c of 16-bit a and b in fp32: one instruction an element,
// without widening first (exact products; one rounding of the sum). LayerNorm
// backward bf16 4096 x 8192 73 us, with widened products 83.
template <class T>
__device__ __forceinline__ float mixed_fma(unsigned short a, unsigned short b, float c) {
    float d;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(a), "h"(b), "f"(c));
    else asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(a), "h"(b), "f"(c));
    return d;
}
template <class T>
__device__ __forceinline__ float mixed_add(unsigned short a, float c) {
    float d;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) asm("add.rn.f32.bf16 %0, %1, %2;" : "=f"(d) : "h"(a), "f"(c));
    else asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(a), "f"(c));
    return d;
}

// What a thread takes at a time, as fp32 pairs: a 16-byte vector, or (VEC 1)
// two elements of its warp's run, 32 apart.
template <class T, int VEC>
struct DropVec : GnVec<T, VEC> {
    using Raw = uint4;
    static constexpr int kPer = 4 / sizeof(T);  // elements of a 32-bit word
    // Pairs i of a and b: a b + c, a b, a + c (one c, or each its own).
    static __device__ __forceinline__ float2 fma(const Raw& a, const Raw& b, int i, float2 c) {
        if constexpr (kPer == 1) return __ffma2_rn(DropVec::get(a, i), DropVec::get(b, i), c);
        else return make_float2(mixed_fma<T>(half(a, 2 * i), half(b, 2 * i), c.x), mixed_fma<T>(half(a, 2 * i + 1), half(b, 2 * i + 1), c.y));
    }
    static __device__ __forceinline__ float2 mul(const Raw& a, const Raw& b, int i) { return fma(a, b, i, make_float2(-0.f, -0.f)); }
    static __device__ __forceinline__ float2 plus(const Raw& a, int i, float c) {
        if constexpr (kPer == 1) return __fadd2_rn(DropVec::get(a, i), f2_splat(c));
        else return make_float2(mixed_add<T>(half(a, 2 * i), c), mixed_add<T>(half(a, 2 * i + 1), c));
    }
    static __device__ __forceinline__ float2 sum(const Raw& a, int i, float2 c) {
        if constexpr (kPer == 1) return __fadd2_rn(DropVec::get(a, i), c);
        else return make_float2(mixed_add<T>(half(a, 2 * i), c.x), mixed_add<T>(half(a, 2 * i + 1), c.y));
    }
    static __device__ __forceinline__ unsigned short half(const Raw& r, int e) {
        return static_cast<unsigned short>(word(r, e / 2) >> (16 * (e % 2)));
    }
    static __device__ __forceinline__ uint32_t word(const Raw& r, int i) { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }
    // What lies in elements from lo on, zeros before.
    static __device__ __forceinline__ Raw keep(const Raw& r, int lo) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = word(r, i);
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (i * kPer + e < lo) w[i] &= kPer == 1 ? 0u : e == 0 ? 0xffff0000u : 0xffffu;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Elements [lo, hi) one by one, to and from the vector's place.
    static __device__ __forceinline__ void store_some(T* p, const Raw& r, int lo, int hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (i * kPer + e >= lo && i * kPer + e < hi) GnVec<T, 1>::store(p + i * kPer + e, word(r, i) >> (16 * e));
    }
    static __device__ __forceinline__ Raw load_some(const T* p, int lo, int hi) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (i * kPer + e >= lo && i * kPer + e < hi) w[i] |= GnVec<T, 1>::load(p + i * kPer + e) << (16 * e);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <class T>
struct DropVec<T, 1> {
    using E = GnVec<T, 1>;
    struct Raw {
        uint32_t lo, hi;
    };
    static constexpr int H = 1;
    static __device__ __forceinline__ float2 fma(const Raw& a, const Raw& b, int, float2 c) { return __ffma2_rn(get(a, 0), get(b, 0), c); }
    static __device__ __forceinline__ float2 mul(const Raw& a, const Raw& b, int) { return __fmul2_rn(get(a, 0), get(b, 0)); }
    static __device__ __forceinline__ float2 plus(const Raw& a, int, float c) { return __fadd2_rn(get(a, 0), f2_splat(c)); }
    static __device__ __forceinline__ float2 sum(const Raw& a, int, float2 c) { return __fadd2_rn(get(a, 0), c); }
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

// A thread's place: its columns, and how far its accesses lie apart. Of a
// step's R rows, a.phases rows lie from one to the next.
template <int VEC, int V, bool GROUP>
struct DropPlace {
    static constexpr bool kGroup = GROUP;
    static constexpr int kRun = VEC == 1 ? 64 * V : 32 * V * VEC;  // columns of a warp's run
    int unit;        // lanes that share sums by butterflies: those of a row, or a warp
    int lead;        // elements of the row's first vector before the row
    int col, step;   // first column (from -lead on); columns from one access to the next
    int N;
    int nv;          // accesses that touch the row; VEC 1: elements
    int warps;       // warps of a team: of a CTA that share a row
    int warp0, team; // the first of them; which team of the CTA
    int rank, C;
    int stride;             // rows from one row of a step to the next
    int64_t first_row, teams;  // of the first step; teams of the grid
    bool first;             // writes the row's statistics
    bool full;              // every access of the warp lies within the row
    int most;               // accesses of the warp's lane that has most
    bool straight;          // the warp has V accesses, each within the row or outside, none partly

    __device__ __forceinline__ explicit DropPlace(const DropArgs& a, int R) : N(a.N) {
        const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31;
        C = GROUP ? 1 : a.cluster;
        rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
        if constexpr (GROUP) {
            unit = a.lanes;
            warps = 1;
            warp0 = tid >> 5;
            team = tid / unit;
            col = (tid & (unit - 1)) * VEC;
            step = unit * VEC;
        } else {
            unit = 32;
            team = tid / a.team;
            warps = a.team >> 5;
            warp0 = team * warps;
            col = (rank * warps + (tid >> 5) - warp0) * kRun + lane * VEC;
            step = 32 * VEC;
        }
        const int each = T / (GROUP ? unit : a.team);
        teams = static_cast<int64_t>(gridDim.x / C) * each;
        const int64_t t = static_cast<int64_t>(blockIdx.x / C) * each + team;
        stride = VEC == 1 ? 1 : a.phases;
        const int phase = static_cast<int>(t) & (stride - 1);
        first_row = (t - phase) * R + phase;
        lead = lead_of(a, t);
        first = rank == 0 && col == 0;
        col -= lead;
        nv = col < N ? min(VEC == 1 ? 2 * V : V, (N - col + step - 1) / step) : 0;
        full = __all_sync(kFullMask, nv == (VEC == 1 ? 2 * V : V) && col >= 0 && (VEC == 1 || col + at(V - 1) + VEC <= N));
        most = VEC == 1 ? V : __reduce_max_sync(kFullMask, nv);
        straight = VEC == 1 ? full : most == V && __all_sync(kFullMask, nv == 0 || (col >= 0 && col + at(nv - 1) + VEC <= N));
    }
    // Elements between a vector's beginning and that of the rows of team t.
    static __device__ __forceinline__ int lead_of(const DropArgs& a, int64_t t) {
        return VEC == 1 ? 0 : ((static_cast<int>(t) & (a.phases - 1)) * a.N) & (VEC - 1);
    }
    __device__ __forceinline__ bool on(int j) const { return (VEC == 1 ? 2 * j : j) < nv; }
    // Whether the thread looks at access j (vectors: the warp does, and finds zeros where the row is not).
    __device__ __forceinline__ bool looks(int j) const { return VEC == 1 ? on(j) : j < most; }
    // The first column of access j, where single elements matter: formed anew
    // each time, as a row's comparisons kept from one step to the next would
    // take the registers of the warps that need none (LayerNorm bf16: 102 -> 128).
    __device__ __forceinline__ int from(int j) const {
        int c = col;
        asm volatile("" : "+r"(c));
        return c + at(j);
    }
    __device__ __forceinline__ int lo(int j) const { return -from(j); }  // elements [lo, hi) of access j lie in the row
    __device__ __forceinline__ int hi(int j) const { return N - from(j); }
    // Whether access j lies within the row as a whole.
    __device__ __forceinline__ bool whole(int j) const {
        const int l = lo(j);
        return VEC == 1 || (l <= 0 && l + N >= VEC);
    }
    // Element e of access j (VEC 1: its two elements).
    __device__ __forceinline__ bool valid(int j, int e) const {
        return VEC == 1 ? 2 * j + e < nv : static_cast<unsigned>(from(j) + e) < static_cast<unsigned>(N);
    }
    // A barrier of the team (0 is the CTA's).
    __device__ __forceinline__ void sync() const {
        if (warps == 1) __syncwarp();
        else if (warps * 32 == static_cast<int>(blockDim.x)) __syncthreads();
        else asm volatile("barrier.cta.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
    }
    // Columns from the first to access j (a constant but where lanes share rows).
    __device__ __forceinline__ int at(int j) const { return VEC == 1 ? 64 * j : GROUP ? j * step : 32 * VEC * j; }
    // Access j of a parameter; p: its first element.
    template <class T>
    __device__ __forceinline__ typename DropVec<T, VEC>::Raw param(const T* p, int j) const {
        p += col + at(j);
        if constexpr (VEC == 1) {
            using E = GnVec<T, 1>;
            typename DropVec<T, 1>::Raw r = DropVec<T, 1>::zero();
            if (2 * j < nv) r.lo = E::load(p);
            if (2 * j + 1 < nv) r.hi = E::load(p + 32);
            return r;
        } else {
            return stride > 1 ? DropVec<T, VEC>::load_some(p, lo(j), hi(j)) : DropVec<T, VEC>::load(p);
        }
    }
    // Access j of a row; p: the thread's first element there. FULL: where the warp is straight.
    template <bool FULL, class T>
    __device__ __forceinline__ void store(T* p, int j, const typename DropVec<T, VEC>::Raw& r) const {
        if constexpr (VEC == 1) {
            using E = GnVec<T, 1>;
            if (FULL || 2 * j < nv) E::store(p + at(j), r.lo);
            if (FULL || 2 * j + 1 < nv) E::store(p + at(j) + 32, r.hi);
        } else {
            if constexpr (FULL) {
                if (on(j)) DropVec<T, VEC>::store(p + at(j), r);
            } else {
                const int l = lo(j), h = l + N;
                if (l <= 0 && h >= VEC) DropVec<T, VEC>::store(p + at(j), r);
                else if (h > 0) DropVec<T, VEC>::store_some(p + at(j), r, l, h);
            }
        }
    }
    // Elements of warp w of CTA k of the cluster.
    __device__ __forceinline__ float count(const DropArgs& a, int k, int w) const {
        const int from = (k * (a.team >> 5) + w) * kRun - lead;
        return static_cast<float>(max(0, min(N, from + kRun) - max(0, from)));
    }
    __device__ __forceinline__ float count_cta(const DropArgs& a, int k) const {
        const int run = (a.team >> 5) * kRun, from = k * run - lead;
        return static_cast<float>(max(0, min(N, from + run) - max(0, from)));
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
    float warp[2][K][kDropMaxThreads / 32];
    float cta[2][K];
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

// Sums over the row of K values per thread, in two halves around a barrier of
// the team: drop_put leaves this warp's, drop_get gives every thread all of
// the row's. (Of rows that lanes of a warp share drop_put gives them.)
template <int K, class P>
__device__ __forceinline__ void drop_put(DropSums<K>& sm, const P& p, int parity, float (&v)[K]) {
    constexpr int L = 32 / K;
    if constexpr (P::kGroup) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = group_sum(v[k], p.unit);
        return;
    }
    const int lane = threadIdx.x & 31;
    const float s = warp_sums<K>(v);
    if ((lane & (L - 1)) == 0) sm.warp[parity][lane / L][threadIdx.x >> 5] = s;
}
template <int K, class P>
__device__ __forceinline__ void drop_get(DropSums<K>& sm, const P& p, int parity, float (&v)[K]) {
    constexpr int L = DropShare<K>::kLanes;
    const int lane = threadIdx.x & 31;
    const DropShare<K> sh;
    const float* w = &sm.warp[parity][sh.idx][p.warp0 + sh.w0];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < DropShare<K>::kEach; ++i) s += sh.w0 + i < p.warps ? w[i] : 0.f;
#pragma unroll
    for (int off = L / 2; off > 0; off /= 2) s += __shfl_xor_sync(kFullMask, s, off);
    if (p.C > 1) {
        // this CTA's value idx, then the CTAs' in rank order
        if (threadIdx.x < 32 && (lane & (32 / K - 1)) == 0) sm.cta[parity][lane / (32 / K)] = s;
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
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(kFullMask, s, K == 1 ? 0 : k * L);
}

// ------------------------------------------------------------ the ring
// NS tensors' accesses of upcoming steps of R rows, each thread its own; with
// STATS each row's mean and rstd too, which a row's lanes fetch together (read
// them after a __syncwarp that follows the wait).
template <class T, int VEC, int V, int R, int NS, bool STATS, class P>
struct DropRing {
    using Raw = typename DropVec<T, VEC>::Raw;
    static constexpr int kCopies = R * NS * V * 32 * 16;  // bytes of a warp's step
    uint32_t base, at_send, at_read, end;
    int stages, stage;

    __device__ __forceinline__ DropRing(const DropArgs& a, void* smem) : stages(a.stages) {
        stage = kCopies + (STATS ? a.stat_bytes : 0);
        base = smem_addr(smem) + (threadIdx.x >> 5) * stages * stage + (threadIdx.x & 31) * 16;
        end = base + stages * stage;
        at_send = at_read = base;
    }
    // Sends the step that begins at `row`; a group of copies is committed even behind the last.
    __device__ __forceinline__ void send(const DropArgs& a, const P& pl, const void* const (&from)[NS], int64_t row) {
        if constexpr (STATS) {
            const int lane = threadIdx.x & 31, i = lane & (pl.unit - 1);
            const uint32_t to = at_send - lane * 16 + kCopies + (lane - i) / pl.unit * (8 * R);
            for (int k = i; k < 2 * R; k += pl.unit) {
                const int64_t q = row + (k >> 1) * pl.stride;
                if (q < a.M) copy_async<4>(to + k * 4, (k & 1 ? a.rstd : a.mean) + q);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (row + r * pl.stride < a.M) {
                const int64_t at = (row + r * pl.stride) * a.N + pl.col;
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    if (from[n]) {
                        const T* const q = static_cast<const T*>(from[n]) + at;
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const uint32_t to = at_send + ((r * NS + n) * V + j) * 512;
                            if (pl.full) {
                                copy_async<16>(to, q + pl.at(j));
                            } else {  // zeros for what lies behind the row
                                const int bytes = max(0, min(16, pl.hi(j) * static_cast<int>(sizeof(T))));
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(bytes > 0 ? q + pl.at(j) : static_cast<const T*>(from[n])),
                                             "r"(bytes)
                                             : "memory");
                            }
                        }
                    }
            }
        copy_async_commit();
        at_send = at_send + stage == end ? base : at_send + stage;
    }
    __device__ __forceinline__ void wait() const {
        if (stages == 2) copy_async_wait<0>();
        else if (stages == 3) copy_async_wait<1>();
        else copy_async_wait<2>();
    }
    // A thread whose first vector begins before the row puts zeros there.
    __device__ __forceinline__ void clear_head(const P& pl) const {
        if (pl.col < 0) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    const Raw v = DropVec<T, VEC>::keep(get(r, n, 0), -pl.col);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at_read + (r * NS + n) * V * 512), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                }
        }
    }
    // Access j of tensor n of row r of the step that was waited for; zeros outside of the row.
    __device__ __forceinline__ Raw get(int r, int n, int j) const {
        Raw v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(at_read + ((r * NS + n) * V + j) * 512)
                     : "memory");
        return v;
    }
    // Mean and rstd of row r.
    __device__ __forceinline__ float2 stat(const P& pl, int r) const {
        const int lane = threadIdx.x & 31;
        float2 v;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(v.x), "=f"(v.y)
                     : "r"(at_read - lane * 16 + kCopies + (lane / pl.unit * R + r) * 8)
                     : "memory");
        return v;
    }
    __device__ __forceinline__ void advance() { at_read = at_read + stage == end ? base : at_read + stage; }
};

// Rows of any width and offset: the CTA's part of a row of NS tensors, as the
// aligned 16-byte chunks that hold it. A chunk starts no earlier than its
// allocation does (those start on larger boundaries), and bytes behind the
// part are not read. Rows are sent together, and read after a barrier that
// follows every thread's wait for its copies.
template <class T, int NS>
struct DropStage {
    static constexpr int kE = static_cast<int>(sizeof(T));
    const char* p[NS];      // the CTA's first element of the next row to send, or null
    uint32_t lead_read[NS];  // where that of the row being read lies in its chunk
    int64_t step, left;     // bytes from one row to the next; rows from the next to send on
    int64_t rows_step;
    int cols, pitch;
    uint32_t base, at_send, at_read, end;

    __device__ __forceinline__ DropStage(const DropArgs& a, int64_t row, int64_t rows_step_, int c0, int cols_, char* smem,
                                         const void* const (&from)[NS])
        : step(rows_step_ * a.N * kE), left(a.M - row), rows_step(rows_step_), cols(cols_), pitch(a.pitch), base(smem_addr(smem)) {
        at_send = at_read = base;
        end = base + a.stages * (NS * pitch);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            p[n] = from[n] ? static_cast<const char*>(from[n]) + (row * a.N + c0) * kE : nullptr;
            lead_read[n] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p[n])) & 15;
        }
    }
    __device__ __forceinline__ void next(uint32_t& at) const { at = at + NS * pitch == end ? base : at + NS * pitch; }
    __device__ __forceinline__ void send() {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (p[n]) {
                if (left > 0) {
                    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(p[n]) & 15);
                    const int bytes = cols > 0 ? lead + cols * kE : 0;
                    const char* const q = p[n] - lead;
                    const uint32_t to = at_send + n * pitch;
                    for (int c = threadIdx.x * 16; c < bytes; c += blockDim.x * 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + c), "l"(q + c), "r"(min(16, bytes - c)) : "memory");
                }
                p[n] += step;
            }
        left -= rows_step;
        copy_async_commit();
        next(at_send);
    }
    // The shared address of the CTA's first element of tensor n of the row being read.
    __device__ __forceinline__ uint32_t row(int n) const { return at_read + n * pitch + lead_read[n]; }
    __device__ __forceinline__ void advance() {
        next(at_read);
#pragma unroll
        for (int n = 0; n < NS; ++n) lead_read[n] = (lead_read[n] + static_cast<uint32_t>(step)) & 15;
    }
    static __device__ __forceinline__ uint32_t element(uint32_t at) {
        if constexpr (kE == 4) {
            uint32_t v;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
            return v;
        } else {
            unsigned short v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
            return v;
        }
    }
    // Access j of a thread whose first element lies at `at`; FULL: every element of the warp's run is there.
    template <bool FULL>
    static __device__ __forceinline__ typename DropVec<T, 1>::Raw get(uint32_t at, int j, int nv) {
        typename DropVec<T, 1>::Raw r = DropVec<T, 1>::zero();
        if (FULL || 2 * j < nv) r.lo = element(at + 64 * j * kE);
        if (FULL || 2 * j + 1 < nv) r.hi = element(at + (64 * j + 32) * kE);
        return r;
    }
};

// ------------------------------------------------------------ masks of a row
// The words of access j of a row: `group` is the generator's group of the
// thread's first element (vectors of fp32: half groups).
template <int VEC, bool LEAN>
struct DropWords {
    uint4 w = make_uint4(0, 0, 0, 0);  // kept, where nothing is dropped (the limit is 0)
    __device__ __forceinline__ void take(const DropMask& m, uint64_t group) {
        if constexpr (VEC == 8) w = m.words<LEAN>(group);
        if constexpr (VEC == 4) {
            const uint4 t = m.words<LEAN>(group >> 1);
            w.x = (group & 1) ? t.z : t.x;
            w.y = (group & 1) ? t.w : t.y;
        }
    }
    // VEC 1: two elements' words, from shared memory
    __device__ __forceinline__ void take(uint32_t at) {
        unsigned short x, y;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(y) : "r"(at + 64) : "memory");
        w.x = x | static_cast<uint32_t>(y) << 16;
    }
    __device__ __forceinline__ bool lo(const DropMask& m, int i) const { return m.low(drop_word(w, i)); }
    __device__ __forceinline__ bool hi(const DropMask& m, int i) const { return m.high(drop_word(w, i)); }
};

// The words of `cols` elements from flat element e on, by the CTA together;
// element e + i's is word (e & 7) + i.
__device__ __forceinline__ void drop_stage_words(const DropMask& m, uint64_t e, int cols, uint4* to) {
    const uint64_t g0 = e >> 3;
    const int n = static_cast<int>(((e + cols + 7) >> 3) - g0);
    for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = m.words<true>(g0 + i);
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

// As many CTAs as the device holds at a time, the teams a multiple of the phases.
inline cudaError_t drop_grid(const void* fn, const norm_plan& p, const DropArgs& a, size_t smem, int64_t* grid) {
    int64_t most = 0;
    const cudaError_t e = drop_resident(fn, p.threads, smem, p.cluster, &most);
    if (e != cudaSuccess) return e;
    const int unit = p.cluster * drop_grid_unit(a.phases, p.threads / (a.lanes > 0 ? a.lanes : a.team));
    *grid = std::min(p.grid, most) / unit * unit;
    return *grid > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
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
