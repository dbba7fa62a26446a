// Group norm over channels-last tensors [B, S, C], building blocks shared by
// the forward (gn_fwd.cuh) and the backward (gn_bwd.cuh).
//
// A thread keeps one access column (VEC neighbouring channels) of its CTA's
// tile and walks rows: channel parameters stay in registers, and `par` rows
// are in flight per step. Groups of D channels: when D is a multiple of VEC
// (ONE) an access lies within one group and a thread's state is one per
// access, otherwise it is one per channel while it runs and one per group that
// the access touches at the end. The states of a CTA meet in shared memory,
// some lanes or warps per group; those of a cluster in distributed shared
// memory; those of row chunks in the caller's workspace.
#pragma once

#include "gn_args.h"
#include "norm_device.cuh"
#include "norm_kernels.cuh"

namespace libnorm {

// ------------------------------------------------------------ accesses
// VEC elements: 16 bytes, a 32-bit pair of 16-bit values, or one element.
// Values are handed out as fp32 pairs (of a single element the second value
// of the pair is 0 and never counted).
template <class T>
struct Gn16 {
    using Pair = Bf16Pair;
};
template <>
struct Gn16<__half> {
    using Pair = F16Pair;
};

template <class T, int VEC>
struct GnVec {
    static_assert(sizeof(T) == 2 && VEC == 8, "16-byte access of a 16-bit type");
    using Raw = uint4;
    using P = typename Gn16<T>::Pair;
    static constexpr int H = 4;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ Raw load(const T* p) { return *reinterpret_cast<const uint4*>(p); }
    static __device__ __forceinline__ void store(T* p, const Raw& v) { *reinterpret_cast<uint4*>(p) = v; }
    static __device__ __forceinline__ float2 get(const Raw& r, int i) {
        return P::widen(i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w);
    }
    static __device__ __forceinline__ void set(Raw& r, int i, float2 v) {
        const uint32_t w = P::pack(v.x, v.y);
        if (i == 0) r.x = w;
        else if (i == 1) r.y = w;
        else if (i == 2) r.z = w;
        else r.w = w;
    }
};

template <>
struct GnVec<float, 4> {
    using Raw = uint4;
    static constexpr int H = 2;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ Raw load(const float* p) { return *reinterpret_cast<const uint4*>(p); }
    static __device__ __forceinline__ void store(float* p, const Raw& v) { *reinterpret_cast<uint4*>(p) = v; }
    static __device__ __forceinline__ float2 get(const Raw& r, int i) {
        return i == 0 ? make_float2(__uint_as_float(r.x), __uint_as_float(r.y))
                      : make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ void set(Raw& r, int i, float2 v) {
        if (i == 0) {
            r.x = __float_as_uint(v.x);
            r.y = __float_as_uint(v.y);
        } else {
            r.z = __float_as_uint(v.x);
            r.w = __float_as_uint(v.y);
        }
    }
};

template <>
struct GnVec<float, 1> {
    using Raw = uint32_t;
    static constexpr int H = 1;
    static __device__ __forceinline__ Raw zero() { return 0; }
    static __device__ __forceinline__ Raw load(const float* p) { return *reinterpret_cast<const uint32_t*>(p); }
    static __device__ __forceinline__ void store(float* p, Raw v) { *reinterpret_cast<uint32_t*>(p) = v; }
    static __device__ __forceinline__ float2 get(Raw r, int) { return make_float2(__uint_as_float(r), 0.f); }
    static __device__ __forceinline__ void set(Raw& r, int, float2 v) { r = __float_as_uint(v.x); }
};

template <class T>
struct GnVec<T, 2> {
    using Raw = uint32_t;
    using P = typename Gn16<T>::Pair;
    static constexpr int H = 1;
    static __device__ __forceinline__ Raw zero() { return 0; }
    static __device__ __forceinline__ Raw load(const T* p) { return *reinterpret_cast<const uint32_t*>(p); }
    static __device__ __forceinline__ void store(T* p, Raw v) { *reinterpret_cast<uint32_t*>(p) = v; }
    static __device__ __forceinline__ float2 get(Raw r, int) { return P::widen(r); }
    static __device__ __forceinline__ void set(Raw& r, int, float2 v) { r = P::pack(v.x, v.y); }
};

template <class T>
struct GnVec<T, 1> {
    using Raw = uint32_t;
    using P = typename Gn16<T>::Pair;
    static constexpr int H = 1;
    static __device__ __forceinline__ Raw zero() { return 0; }
    static __device__ __forceinline__ Raw load(const T* p) { return *reinterpret_cast<const unsigned short*>(p); }
    static __device__ __forceinline__ void store(T* p, Raw v) {
        *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(v);
    }
    static __device__ __forceinline__ float2 get(Raw r, int) { return P::widen(r); }
    static __device__ __forceinline__ void set(Raw& r, int, float2 v) { r = P::pack(v.x, 0.f); }
};

template <class T>
__device__ __forceinline__ float gn_elem(const T* p) {
    return GnVec<T, 1>::get(GnVec<T, 1>::load(p), 0).x;
}

__device__ __forceinline__ float2 f2_sub(float2 a, float2 b) {
    return __fadd2_rn(a, make_float2(-b.x, -b.y));
}
template <int VEC>
__device__ __forceinline__ float f2_sum(float2 v) {
    return VEC == 1 ? v.x : v.x + v.y;
}

// ------------------------------------------------------------ activations
// The logistic function 1 / (1 + 2^t), t = -z log2 e, of a pair, from the
// hardware's base-2 exponential and reciprocal: one instruction each, within a
// few ulp; an exponential beyond fp32 is infinity, whose reciprocal is 0. With
// the range handling of __expf and __fdividef the activation was more than
// half of the instructions of a forward pass. (One reciprocal of the product
// for both, with z held above -44 so that it stays in range, measured slower:
// gn_bwd f16 8x4096x320 23.2 -> 24.1 us.)
__device__ __forceinline__ float2 gn_logistic2(float2 z) {
    const float2 t = __fmul2_rn(z, f2_splat(-1.4426950408889634f));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    const float2 p = __fadd2_rn(e, f2_splat(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(p.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(p.y));
    return r;
}

// The normal distribution's tail of a pair: with m = min(|z|, 16), the limit
// beyond which the tail is below fp32, e = exp(-m^2 / 2) and
// tail = erfc(m / sqrt 2) / 2 = Q(t) e / 2, t = 1 / (1 + p m / sqrt 2). Q, of
// degree 8 without a constant, is this file's own fit of exp(x^2) erfc(x):
// erfc is within 2.1e-8 absolutely (relatively 4.5e-8 up to x = 2, 3.3e-7 up
// to 4, 1.1e-6 beyond; the form with 1 / (1 + p x) is that of
// Hastings, "Approximations for Digital Computers", 1955). In fp32 the tail is
// within 3 u of the exact one absolutely, relatively within 7 u for m up to 2
// and (52 + 1.5 m^2) u anywhere (m^2 / 2 is rounded before the exponential);
// gelu within u (|z| + 1). One pass for every z,
// and the slope's exp(-z^2 / 2) comes with it: with erff for each value, in two
// branches, gn_bwd bf16 4x65536x256 took 173 us for the 123, gn_fwd 96 for 79.
// (80 registers for gn_fwd_split_apply instead of 64 and a few spilled words:
// 99, since the two launches then do not fit side by side.)
struct GnTail {
    float2 m, e, tail;
};
__device__ __forceinline__ GnTail gn_tail2(float2 z) {
    GnTail r;
    asm("min.NaN.f32 %0, %1, 0f41800000;" : "=f"(r.m.x) : "f"(fabsf(z.x)));  // (NaN stays)
    asm("min.NaN.f32 %0, %1, 0f41800000;" : "=f"(r.m.y) : "f"(fabsf(z.y)));
    const float2 d = __ffma2_rn(r.m, f2_splat(0.42f * 0.70710678118654752f), f2_splat(1.f));
    const float2 u = __fmul2_rn(__fmul2_rn(r.m, r.m), f2_splat(-0.5f * 1.4426950408889634f));
    float2 t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(d.y));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.e.x) : "f"(u.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.e.y) : "f"(u.y));
    constexpr float q[8] = {0.23681276939172055f,  0.2398510887911381f,  0.1925742656963855f,   0.2772031931709584f,
                            -0.14858194757490237f, 0.46206568355798416f, -0.33348673756550784f, 0.07356170515362967f};
    float2 s = f2_splat(0.5f * q[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) s = __ffma2_rn(s, t, f2_splat(0.5f * q[i]));
    r.tail = __fmul2_rn(__fmul2_rn(s, t), r.e);
    return r;
}

template <int ACT>
__device__ __forceinline__ float2 gn_act2(float2 z) {
    if constexpr (ACT == NORM_ACT_SILU) {
        return __fmul2_rn(z, gn_logistic2(z));
    }
    if constexpr (ACT == NORM_ACT_GELU) {
        const GnTail k = gn_tail2(z);
        // max(z, 0) - |z| tail
        const float2 h = __fmul2_rn(z, f2_splat(0.5f));
        const float2 up = __fadd2_rn(h, make_float2(fabsf(h.x), fabsf(h.y)));
        return __ffma2_rn(make_float2(-k.m.x, -k.m.y), k.tail, up);
    }
    return z;
}

// act'(z): s (1 + z (1 - s)) with s = 1 / (1 + exp(-z)); Phi(z) + z phi(z).
template <int ACT>
__device__ __forceinline__ float2 gn_act_slope2(float2 z) {
    if constexpr (ACT == NORM_ACT_SILU) {
        const float2 s = gn_logistic2(z);
        const float2 zs = __fmul2_rn(z, s);               // s + z s (1 - s)
        return __fadd2_rn(s, __ffma2_rn(make_float2(-zs.x, -zs.y), s, zs));
    }
    if constexpr (ACT == NORM_ACT_GELU) {
        const GnTail k = gn_tail2(z);
        // for z >= 0, 1 - (tail - m phi), and below, tail - m phi; phi = e / sqrt(2 pi)
        const float2 v = __ffma2_rn(__fmul2_rn(k.m, f2_splat(-0.39894228040143268f)), k.e, k.tail);
        return make_float2(z.x < 0.f ? v.x : 1.f - v.x, z.y < 0.f ? v.y : 1.f - v.y);
    }
    return f2_splat(1.f);
}

// ------------------------------------------------------------ geometry
__device__ __forceinline__ int quot(int n, const FastDiv& d) {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), d.m) + static_cast<uint32_t>(n)) >> d.s);
}
// n / d of small numbers (both below 2^20): (n + 1/2) / d is at least
// 1 / (2 d) away from a whole number, far more than the division's error.
__device__ __forceinline__ int small_quot(int n, int d) {
    return static_cast<int>(__fdividef(static_cast<float>(n) + 0.5f, static_cast<float>(d)));
}

// The CTA's tile: which sample, which accesses of a row, which groups, and
// this thread's place in it.
struct GnTile {
    int64_t b;      // sample
    int t;          // tile of the row
    int c0, nc;     // first channel, channels
    int g0, ng;     // first group touched, groups touched
    int col, r;     // this thread's access column and row slot
    bool on;        // this thread has an access
};

template <int VEC>
__device__ __forceinline__ GnTile gn_tile(const GnArgs& a, int unit) {
    GnTile w;
    const int b = quot(unit, a.by_tiles);
    w.b = b;
    w.t = unit - b * a.tiles;
    const int k0 = w.t * a.tile;
    const int nk = min(a.tile, a.ncols - k0);
    w.c0 = k0 * VEC;
    w.nc = nk * VEC;
    w.g0 = quot(w.c0, a.by_D);
    w.ng = quot(w.c0 + w.nc - 1, a.by_D) - w.g0 + 1;
    w.r = quot(threadIdx.x, a.by_tile);
    w.col = static_cast<int>(threadIdx.x) - w.r * a.tile;
    w.on = w.r < a.par && w.col < nk;
    return w;
}

// Rows [first, first + n) of chunk k when every chunk has `per` rows.
__device__ __forceinline__ int64_t gn_chunk_len(int64_t S, int64_t per, int64_t k) {
    const int64_t left = S - k * per;
    return left < 0 ? 0 : left < per ? left : per;
}

// Rows each row slot visits of a chunk's `rows` rows walked `par` at a time:
// slots below `full` visit `most`, the others one fewer.
struct GnVisits {
    int most, full;
    __device__ __forceinline__ GnVisits(int rows, const GnArgs& a) {
        most = quot(rows + a.par - 1, a.by_par);
        full = rows - (most - 1) * a.par;
    }
    __device__ __forceinline__ int of(int r) const { return most == 0 ? 0 : most - (r < full ? 0 : 1); }
};

// The group of each of an access's channels, and where it changes: walks
// neighbouring channels with one division at the start.
struct GnWalk {
    int g, left;  // group of the current channel, channels left in it
    int D;
    __device__ __forceinline__ GnWalk(int c, const GnArgs& a) : D(a.D) {
        g = quot(c, a.by_D);
        left = (g + 1) * D - c;
    }
    __device__ __forceinline__ void next() {
        if (--left == 0) {
            ++g;
            left = D;
        }
    }
};

// How a CTA's threads share its groups in the merges: 2^bits lanes per group
// while there are more groups than warps, otherwise `wpg` whole warps.
struct GnShare {
    int lanes, bits, wpg;
    __device__ __forceinline__ explicit GnShare(int ng) {
        const int warps = blockDim.x >> 5;
        wpg = ng >= warps ? 1 : small_quot(warps, ng);
        bits = 5;
        while (bits > 0 && (ng << bits) > static_cast<int>(blockDim.x)) --bits;
        lanes = 1 << bits;
    }
};

// Sums of two values over aligned groups of `width` lanes, their butterflies
// side by side.
__device__ __forceinline__ void group_sum2(float& a, float& b, int width) {
    for (int off = width >> 1; off > 0; off >>= 1) {
        const float x = __shfl_xor_sync(kFullMask, a, off), y = __shfl_xor_sync(kFullMask, b, off);
        a += x;
        b += y;
    }
}

// A row of distributed shared memory: float2 at index i of cluster peer
// `rank`'s copy of `p`.
__device__ __forceinline__ float2 gn_peer(const float2* p, int i, uint32_t rank) {
    float2 v;
    const uint32_t at = peer_smem_addr(p + i, rank);
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// ------------------------------------------------------------ row streams
// Walks a thread's rows of N tensors with the next rows' accesses in flight:
// every thread copies its own accesses asynchronously into slots of shared
// memory of its own (no barrier: a thread waits for its own copies only),
// kStep * (kSteps - 1) rows ahead, which costs no registers while they travel.
// A slot is refilled one step after it was read. (Rings measured in us for
// gn_fwd bf16 1x262144x256 / gn_bwd f16 8x4096x320 / bf16 4x65536x256: 4 steps
// of 2 rows 69 / 22 / 104; 4 of 1 79 / 22 / 113; 8 of 1 69 / 23 / 107; 2 of 4
// 75 / 22 / 105; 4 of 4 76 / 33 / 115, when the second launch still read ahead of
// its wait: 0.6 us less of the second case. Of 4 bytes, gn_bwd f32 5x363654x25: 4 of
// 4 278, 4 of 2 310, 8 of 4 293, with two CTAs per SM.) Accesses of one 16-bit
// value, which asynchronous copies do not have, are loaded kBatch rows at a time
// instead (gn_bwd f16 5x363654x25, two CTAs per SM: 8 rows 220 us, 4 287; four:
// 8 rows 151, 16 190).
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

template <class T, int VEC, int N>
struct GnStream {
    using X = GnVec<T, VEC>;
    using Raw = typename X::Raw;
    static constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
    static constexpr bool kAsync = kBytes >= 4;
    // rows per step, steps in the ring
    static constexpr int kStep = kBytes == 16 ? 2 : 4, kSteps = 4;
    static constexpr int kBatch = 8;

    // Shared memory of the slots: those that `visits` rows per thread use.
    static size_t ring_bytes(int64_t visits, int threads) {
        const int64_t rows = (visits + kStep - 1) / kStep * kStep;
        return kAsync ? static_cast<size_t>(rows < kStep * kSteps ? rows : kStep * kSteps) * N * kBytes * threads : 0;
    }

    const T* p[N];      // the next row to copy (or load)
    int64_t step[N];    // to the row after it
    const int visits;
    uint32_t base, pitch;  // this thread's first slot, and from one slot to the next
    int sent = 0;          // rows whose copies have been issued

    // Row v of tensor n is at first[n] + v * step_[n]; the first copies are
    // issued at once, so that what is done until run() overlaps them.
    __device__ __forceinline__ GnStream(const T* const (&first)[N], const int64_t (&step_)[N], int visits_, void* ring)
        : visits(visits_), base(smem_addr(ring) + threadIdx.x * kBytes), pitch(blockDim.x * kBytes) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            p[n] = first[n];
            step[n] = step_[n];
        }
        if constexpr (kAsync) {
#pragma unroll
            for (int s = 0; s < kSteps - 1; ++s) send(s);
        }
    }
    __device__ __forceinline__ void send(int slot) {
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
            if (sent < visits) {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    copy_async<kBytes>(base + ((slot * kStep + u) * N + n) * pitch, p[n]);
                    p[n] += step[n];
                }
            }
            ++sent;
        }
        copy_async_commit();
    }
    // Calls f(v, raw) for rows v = 0 .. visits - 1 in order.
    template <class F>
    __device__ __forceinline__ void run(F f) {
        if constexpr (kAsync) {
            int slot = 0;
            for (int v = 0; v < visits; v += kStep) {
                copy_async_wait<kSteps - 2>();  // this step's copies have landed
                Raw raw[kStep][N];
#pragma unroll
                for (int u = 0; u < kStep; ++u)
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const uint32_t at = base + ((slot * kStep + u) * N + n) * pitch;
                        if constexpr (kBytes == 16)
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(raw[u][n].x), "=r"(raw[u][n].y), "=r"(raw[u][n].z), "=r"(raw[u][n].w)
                                         : "r"(at)
                                         : "memory");
                        else
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw[u][n]) : "r"(at) : "memory");
                    }
                // the slots read one step ago
                send((slot + kSteps - 1) & (kSteps - 1));
                slot = (slot + 1) & (kSteps - 1);
#pragma unroll
                for (int u = 0; u < kStep; ++u)
                    if (v + u < visits) f(v + u, raw[u]);
            }
        } else {
            for (int v = 0; v < visits; v += kBatch) {
                Raw raw[kBatch][N];
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
#pragma unroll
                    for (int n = 0; n < N; ++n) raw[u][n] = v + u < visits ? X::load(p[n] + u * step[n]) : X::zero();
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (v + u < visits) f(v + u, raw[u]);
#pragma unroll
                for (int n = 0; n < N; ++n) p[n] += kBatch * step[n];
            }
        }
    }
};

// ------------------------------------------------------------ launch
// Opts a kernel in to the device's largest dynamic shared memory per block
// (once per kernel and device; not a stream operation), and asks for the
// largest share of the SM's memory for it: CTAs of two launches then fit side
// by side (gn_bwd f32 3x1517x180 9.2 us instead of 11.2, larger calls alike).
inline cudaError_t gn_opt_in(const void* fn) try {
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, bool> done;
    int dev = 0, most = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({fn, dev})) return cudaSuccess;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, fn);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most - static_cast<int>(fa.sharedSizeBytes));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) done[{fn, dev}] = true;
    return e;
} catch (...) {  // (no exception leaves a C entry point)
    return cudaErrorMemoryAllocation;
}

// A kernel on `grid` CTAs in clusters of `cluster`, with programmatic stream
// serialization like every kernel of the library.
inline cudaError_t gn_launch(const void* fn, int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                             const GnArgs& a) {
    if (smem > 16 * 1024) {
        const cudaError_t e = gn_opt_in(fn);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
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
    void* args[] = {const_cast<GnArgs*>(&a)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace libnorm
