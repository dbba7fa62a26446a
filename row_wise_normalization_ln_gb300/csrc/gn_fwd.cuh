// Group norm forward kernels.
//
//   gn_fwd_chip   a CTA, or a cluster, holds all rows of a sample's tile in
//                 registers: statistics, activation and output from one read.
//   gn_fwd_split_sums,  for tiles that do not fit a cluster: row chunks are
//   gn_fwd_split_apply  summed into the workspace; the second launch merges
//                       them and writes y from a second read of x (from L2
//                       where x fits).
//
// Statistics: differences d = x - K from a shift K near the data, so that a
// group whose mean dwarfs its spread keeps its digits (x - K of nearby values
// is exact). Per-thread states (count, sum, M2 = sum (d - mean)^2) merge in
// the k-way form mean = sum s_t / n, M2 = sum M2_t + n_t (m_t - mean)^2,
// which is what any sequence of pairwise merges reaches; the variance is
// never formed as E[x^2] - E[x]^2 of unshifted values. All in fp32, the merged
// sums in pairs of fp32. Outputs are formed from x - mean, with what the
// rounding of the mean left added back.
//
// What bounds them (one GB300, copy bandwidth 6.8 TB/s, calls from a graph
// over inputs beyond L2):
//   gn_fwd_chip   launch and latency: a load, the merges, in a cluster two
//                 barriers, a store. bf16 1x64x1280 3.4 us, f32 3x1517x180
//                 (6.6 MB, clusters of 8) 7.4 us.
//   split         HBM, with x read twice where it exceeds L2: bf16
//                 1x262144x256 69 us, 5.8 TB/s of its 403 MB (sums 26 us at
//                 5.2 TB/s, apply 44 at 5.6). Small calls are two launches of
//                 about 4 us, and the second's first rows, which it may not
//                 read before its wait: bf16 2x4096x320 9.6 us.
// One persistent kernel that works in bands of rows that stay in L2, and bands
// in launches of their own, were measured and were slower (the persistent one
// 91 us for the 69).
#pragma once

#include "gn_kernels.cuh"

namespace libnorm {

// Collapses the per-channel states (sum s, M2 m2 of `visits` values each) of
// an access to one per group it touches: (sum, M2) of visits * channels
// values, in this thread's slots st[0 .. segs).
template <int VEC>
__device__ __forceinline__ void gn_collapse(const float2* s, const float2* m2, float visits, int c, const GnArgs& a,
                                            float2* st) {
    constexpr int H = (VEC + 1) / 2;
    GnWalk k(c, a);
    const float inv = visits > 0.f ? __fdividef(1.f, visits) : 0.f;
    int seg = 0, first = 0;
    float t = 0.f;
    // the channels of one group end where the walk steps to the next
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        t += (j & 1) ? s[j / 2].y : s[j / 2].x;
        const int g = k.g;
        k.next();
        if (j == VEC - 1 || k.g != g) {
            const float mean = __fdividef(t, static_cast<float>(j + 1 - first)) * inv;
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 d = __ffma2_rn(s[i], f2_splat(inv), f2_splat(-mean));
                const float2 e = __ffma2_rn(__fmul2_rn(d, f2_splat(visits)), d, m2[i]);
                if (2 * i >= first && 2 * i <= j) q += e.x;
                if (2 * i + 1 >= first && 2 * i + 1 <= j) q += e.y;
            }
            st[seg++] = make_float2(t, q);
            t = 0.f;
            first = j + 1;
        }
    }
}

// A merged state: the sum of the differences from the group's first element
// as an unevaluated pair (x + y, |y| within half an ulp of x), M2 in z, the
// count in w. The pair keeps the mean's last bits where it is small against
// the spread: one rounding of a sum of that size would be a large error of
// such a mean.
__device__ __forceinline__ void ff_add(float& hi, float& lo, float a, float b) {
    const float s = hi + a, t = s - hi;  // Knuth's two-sum
    lo += ((hi - (s - t)) + (a - t)) + b;
    hi = s;
}

// Merges the states that walk(f) hands to f one by one over aligned groups of
// `lanes` lanes (every lane of the warp calls it).
template <class Walk>
__device__ __forceinline__ float4 gn_merge(Walk walk, int lanes) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    walk([&](const float4& e) {
        ff_add(t.x, t.y, e.x, e.y);
        t.w += e.w;
    });
    for (int off = lanes >> 1; off > 0; off >>= 1) {
        const float x = __shfl_xor_sync(kFullMask, t.x, off), y = __shfl_xor_sync(kFullMask, t.y, off);
        t.w += __shfl_xor_sync(kFullMask, t.w, off);
        ff_add(t.x, t.y, x, y);
    }
    const float mean = t.w > 0.f ? __fdividef(t.x, t.w) : 0.f;
    walk([&](const float4& e) {
        const float d = __fdividef(e.x, e.w) - mean;
        if (e.w > 0.f) t.z += fmaf(e.w * d, d, e.z);
    });
    t.z = group_sum(t.z, lanes);
    return t;
}

// Merges the CTA's thread states into states gs[g * wpg + part]. The states
// (sum, M2) of row slot r and access column u start at st[(r * tile + u) *
// segs], one per group the access touches. Lanes side by side over the
// group's accesses, then row slots. Every thread of the CTA calls it, after a
// barrier.
template <int VEC>
__device__ __forceinline__ void gn_merge_threads(const GnArgs& a, const GnTile& w, const float2* st, int segs,
                                                 const GnVisits& vis, const GnShare& sh, float4* gs) {
    const int lanes = sh.lanes, lane = threadIdx.x & (lanes - 1);
    const int jobs = w.ng * sh.wpg;
    for (int base = 0; base < jobs << sh.bits; base += blockDim.x) {
        // (every lane of a warp takes part in the butterflies, with or without a job)
        const int j = (base + static_cast<int>(threadIdx.x)) >> sh.bits;
        const bool on = j < jobs;
        const int g = !on ? 0 : sh.wpg == 1 ? j : small_quot(j, sh.wpg), part = on ? j - g * sh.wpg : 0;
        const int lo = max((w.g0 + g) * a.D, w.c0), hi = min((w.g0 + g + 1) * a.D, w.c0 + w.nc);
        const int u0 = (lo - w.c0) / VEC, n = (hi - 1 - w.c0) / VEC - u0 + 1;
        const int across = min(n, lanes), deep = small_quot(lanes, across);
        const int r0 = small_quot(lane, across), uf = lane - r0 * across;
        const float4 t = gn_merge([&](auto f) {
            if (on && r0 < deep)
                for (int u = uf; u < n; u += lanes) {
                    const int ch = w.c0 + (u0 + u) * VEC;  // the access's first channel
                    const int len = min(hi, ch + VEC) - max(lo, ch);
                    const int seg = segs == 1 ? 0 : w.g0 + g - quot(ch, a.by_D);
                    for (int r = part + sh.wpg * r0; r < a.par; r += sh.wpg * deep) {
                        const float2 e = st[(r * a.tile + u0 + u) * segs + seg];
                        f(make_float4(e.x, 0.f, e.y, static_cast<float>(vis.of(r) * len)));
                    }
                }
        }, lanes);
        if (on && lane == 0) gs[j] = t;
    }
}

// The groups' states from their `wpg` states in each of the `cs` CTAs of the
// cluster: calls done(group, state) once for each of the tile's groups. The
// lanes of a group take one state each where there are enough.
template <class F>
__device__ __forceinline__ void gn_merge_cluster(const float4* gs, int ng, int wpg, int cs, F done) {
    const int n = cs * wpg;
    if (n == 1) {
        for (int g = threadIdx.x; g < ng; g += blockDim.x) done(g, gs[g]);
        return;
    }
    int bits = 0;
    while (bits < 5 && (1 << bits) < n) ++bits;
    const int lanes = 1 << bits, lane = threadIdx.x & (lanes - 1);
    for (int base = 0; base < ng << bits; base += blockDim.x) {
        const int g = (base + static_cast<int>(threadIdx.x)) >> bits;
        const bool on = g < ng;
        const float4 t = gn_merge([&](auto f) {
            if (on)
                for (int i = lane; i < n; i += lanes) {
                    const int k = wpg == 1 ? i : small_quot(i, wpg), at = g * wpg + (i - k * wpg);
                    f(cs > 1 ? ld_peer_f32x4(peer_smem_addr(gs + at, k)) : gs[at]);
                }
        }, lanes);
        if (on && lane == 0) done(g, t);
    }
}

// The mean of a group from its first element K and its merged state, rounded
// once, and what the rounding left.
__device__ __forceinline__ float2 gn_mean(float K, const float4& t) {
    const float q = __fdiv_rn(t.x, t.w);
    const float rest = __fdividef(fmaf(-q, t.w, t.x) + t.y, t.w);  // what the quotient leaves
    float hi = K, lo = 0.f;
    ff_add(hi, lo, q, rest);
    const float mean = hi + lo;
    return make_float2(mean, (hi - mean) + lo);
}

// The square root and the division are the correctly rounded ones: there is
// one per group, and rsqrtf's two ulps would scale every output.
__device__ __forceinline__ float gn_rstd(float m2, float count, float eps) {
    return __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(m2, count) + eps));
}

// y = act(d * s + o) per channel: s = rstd * gamma, o = beta - rest * s, with
// K the group's rounded mean, rest what the rounding left, and d = x - K.
template <class T, int VEC, bool ONE, int ACT>
struct GnOut {
    using X = GnVec<T, VEC>;
    static constexpr int HG = ONE ? 1 : X::H;
    float2 K[HG], s[X::H], o[X::H];

    // fin(g): float2 (rest, rstd) of group g.
    template <class Fin>
    __device__ __forceinline__ void init(const typename X::Raw& rg, const typename X::Raw& rb, int c, const GnArgs& a,
                                         Fin fin) {
        GnWalk k(c, a);
        float2 fa = fin(k.g);
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            float2 fb = fa;
            if constexpr (!ONE) {
                if (i > 0) fa = fin(k.g);
                k.next();
                fb = fin(k.g);
                k.next();
            }
            const float2 gm = X::get(rg, i), be = X::get(rb, i);
            s[i] = make_float2(fa.y * gm.x, fb.y * gm.y);
            o[i] = make_float2(fmaf(-fa.x, s[i].x, be.x), fmaf(-fb.x, s[i].y, be.y));
        }
    }
    __device__ __forceinline__ typename X::Raw apply(const typename X::Raw& r) const {
        typename X::Raw out = X::zero();
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            const float2 z = __ffma2_rn(f2_sub(X::get(r, i), K[ONE ? 0 : i]), s[i], o[i]);
            X::set(out, i, gn_act2<ACT>(z));
        }
        return out;
    }
};

// A value per channel of an access from one per group: v(g).
template <class T, int VEC, bool ONE, class F>
__device__ __forceinline__ void gn_per_group(float2* K, int c, const GnArgs& a, F v) {
    using X = GnVec<T, VEC>;
    GnWalk k(c, a);
    float last = v(k.g);
    if constexpr (ONE) {
        K[0] = make_float2(last, VEC == 1 ? 0.f : last);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (j & 1) K[j / 2].y = last;
            else K[j / 2].x = last;
            const int g = k.g;
            k.next();
            if (j + 1 < VEC && k.g != g) last = v(k.g);
        }
    }
}

template <class T, int VEC, bool ONE, int ACT, int V>
__global__ void __launch_bounds__(kGnMaxThreads) gn_fwd_chip(const GnArgs a) {
    using X = GnVec<T, VEC>;
    constexpr int HG = ONE ? 1 : X::H;
    extern __shared__ __align__(16) float2 sm[];
    grid_release();
    const int cs = a.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const GnTile w = gn_tile<VEC>(a, static_cast<int>(blockIdx.x) >> a.cluster_bits);
    const int segs = ONE ? 1 : a.segs;
    const GnShare sh(w.ng);
    float4* gs = reinterpret_cast<float4*>(sm);  // (16-byte aligned: first)
    float2* fin = reinterpret_cast<float2*>(gs + w.ng * sh.wpg);
    float2* st = fin + w.ng;
    float* mid = reinterpret_cast<float*>(st + a.par * a.tile * segs);  // the first element of each group, then its mean

    const int64_t row0 = int64_t(rank) * a.chunk_rows;
    const int rows = static_cast<int>(gn_chunk_len(a.S, a.chunk_rows, rank));
    const GnVisits vis(rows, a);
    const int visits = w.on ? vis.of(w.r) : 0;
    const int c = w.c0 + w.col * VEC;
    const T* xs = static_cast<const T*>(a.x) + w.b * a.xb;
    const T* xp = xs + (row0 + w.r) * a.xr + c;
    grid_wait();
    typename X::Raw raw[V], rg, rb;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < visits) raw[v] = X::load(xp + int64_t(v) * a.par * a.xr);
    // the shift of a group: its first element in the sample's first row
    GnOut<T, VEC, ONE, ACT> out;
    if (w.on) {
        gn_per_group<T, VEC, ONE>(out.K, c, a, [&](int g) { return gn_elem(xs + int64_t(g) * a.D); });
        rg = X::load(static_cast<const T*>(a.gamma) + c);
        rb = X::load(static_cast<const T*>(a.beta) + c);
    }
    // The thread's states by two passes over its registers. An access within
    // one group has one state for its channels.
    if (w.on) {
        float2 s[HG], q[HG];
#pragma unroll
        for (int i = 0; i < HG; ++i) s[i] = q[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < visits) {
#pragma unroll
                for (int i = 0; i < X::H; ++i) {
                    const int j = ONE ? 0 : i;
                    s[j] = __fadd2_rn(s[j], f2_sub(X::get(raw[v], i), out.K[j]));
                }
            }
        const float inv = visits > 0 ? __fdividef(1.f, static_cast<float>(visits)) : 0.f;
        float2 m[HG];  // the means
        if constexpr (ONE) {
            s[0].x = f2_sum<VEC>(s[0]);
            m[0] = f2_splat(s[0].x * inv * (1.f / VEC));
        } else {
#pragma unroll
            for (int i = 0; i < HG; ++i) m[i] = __fmul2_rn(s[i], f2_splat(inv));
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < visits) {
#pragma unroll
                for (int i = 0; i < X::H; ++i) {
                    const int j = ONE ? 0 : i;
                    const float2 d = f2_sub(f2_sub(X::get(raw[v], i), out.K[j]), m[j]);
                    q[j] = __ffma2_rn(d, d, q[j]);
                }
            }
        float2* mine = st + (w.r * a.tile + w.col) * segs;
        if constexpr (ONE)
            mine[0] = make_float2(s[0].x, f2_sum<VEC>(q[0]));
        else
            gn_collapse<VEC>(s, q, static_cast<float>(visits), c, a, mine);
    }
    // (before the cluster's barrier: in place, row 0 is overwritten after it)
    for (int g = threadIdx.x; g < w.ng; g += blockDim.x) mid[g] = gn_elem(xs + int64_t(w.g0 + g) * a.D);
    __syncthreads();
    gn_merge_threads<VEC>(a, w, st, segs, vis, sh, gs);
    if (cs > 1)
        cluster_barrier();
    else
        __syncthreads();
    gn_merge_cluster(gs, w.ng, sh.wpg, cs, [&](int g, const float4& t) {
        const float rstd = gn_rstd(t.z, t.w, a.eps);
        const float2 m = gn_mean(mid[g], t);
        fin[g] = make_float2(m.y, rstd);
        mid[g] = m.x;
        if (rank == 0) {
            const int64_t at = w.b * a.G + w.g0 + g;
            if (a.mean) a.mean[at] = m.x;
            if (a.rstd) a.rstd[at] = rstd;
        }
    });
    __syncthreads();
    if (cs > 1) cluster_arrive();  // this CTA has read its peers' states
    if (w.on) {
        gn_per_group<T, VEC, ONE>(out.K, c, a, [&](int g) { return mid[min(g - w.g0, w.ng - 1)]; });
        out.init(rg, rb, c, a, [&](int g) { return fin[min(g - w.g0, w.ng - 1)]; });
        T* yp = static_cast<T*>(a.y) + w.b * a.yb + (row0 + w.r) * a.yr + c;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < visits) X::store(yp + int64_t(v) * a.par * a.yr, out.apply(raw[v]));
    }
    if (cs > 1) cluster_wait();
}

// Rows a thread adds with one shift before it merges them into its running
// state. The shift may lie far from the other rows, and a long chain of fp32
// additions of squares is biased (each add rounds to a multiple of the sum's
// ulp, and more squares lie below half of it than above): 512 in a row lose
// 2e-6 of the sum, 64 2e-7.
constexpr int kGnShiftRows = 32;

// The pairwise merge (S, m2) of n values += k values with sum s and sum of
// squares q about K, with `to` = K - the reference of S.
__device__ __forceinline__ void gn_pair_merge(float& S, float& m2, float n, float s, float q, float k, float to) {
    const float m = __fdividef(s, k), b2 = fmaf(-s, m, q);
    const float d = n > 0.f ? (to + m) - __fdividef(S, n) : 0.f;
    m2 += fmaf(d * d, __fdividef(n * k, n + k), b2 < 0.f ? 0.f : b2);  // (the subtraction can round below 0; NaN stays)
    S += fmaf(to, k, s);
}

// Row chunk k of a tile: its groups' states into the workspace.
template <class T, int VEC, bool ONE>
__device__ __forceinline__ void gn_fwd_sums(const GnArgs& a, const GnTile& w, int k, float2* sm, void* ring) {
    using X = GnVec<T, VEC>;
    constexpr int HG = ONE ? 1 : X::H;
    const int segs = ONE ? 1 : a.segs;
    const GnShare sh(w.ng);
    float4* gs = reinterpret_cast<float4*>(sm);
    float2* st = reinterpret_cast<float2*>(gs + w.ng * sh.wpg);

    const int rows = static_cast<int>(gn_chunk_len(a.S, a.chunk_rows, k));
    const GnVisits vis(rows, a);
    const int c = w.c0 + w.col * VEC;
    const T* xs = static_cast<const T*>(a.x) + w.b * a.xb;
    const int visits = w.on ? vis.of(w.r) : 0;
    const T* const p[1] = {xs + (k * a.chunk_rows + w.r) * a.xr + c};
    const int64_t step[1] = {int64_t(a.par) * a.xr};
    grid_wait();
    grid_release();
    GnStream<T, VEC, 1> rows_in(p, step, visits, ring);
    if (w.on) {
        // Blocks of kGnShiftRows rows, shifted by the block's first value:
        // per channel, or for an access within a group in two chains over its
        // channels. A full block goes into the running state (S, m2), whose
        // sum is relative to the group's first element.
        constexpr int HS = ONE ? (X::H < 2 ? X::H : 2) : X::H;
        float2 S[HG], m2[HG], K[HG], s[HS], q[HS];
#pragma unroll
        for (int i = 0; i < HG; ++i) S[i] = m2[i] = K[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < HS; ++i) s[i] = q[i] = make_float2(0.f, 0.f);
        auto merge = [&](int first, int stop) {
            const float n = static_cast<float>(first), kk = static_cast<float>(stop - first);
            float2 G0[HG];
            gn_per_group<T, VEC, ONE>(G0, c, a, [&](int g) { return gn_elem(xs + int64_t(g) * a.D); });
            if constexpr (ONE) {
                float ts = f2_sum<VEC>(s[0]), tq = f2_sum<VEC>(q[0]);
                if constexpr (HS > 1) {
                    ts += f2_sum<VEC>(s[HS - 1]);
                    tq += f2_sum<VEC>(q[HS - 1]);
                }
                gn_pair_merge(S[0].x, m2[0].x, n * VEC, ts, tq, kk * VEC, K[0].x - G0[0].x);
            } else {
#pragma unroll
                for (int i = 0; i < HG; ++i) {
                    gn_pair_merge(S[i].x, m2[i].x, n, s[i].x, q[i].x, kk, K[i].x - G0[i].x);
                    gn_pair_merge(S[i].y, m2[i].y, n, s[i].y, q[i].y, kk, K[i].y - G0[i].y);
                }
            }
        };
        rows_in.run([&](int v, const auto& raw) {
            if ((v & (kGnShiftRows - 1)) == 0) {
                if (v > 0) merge(v - kGnShiftRows, v);
#pragma unroll
                for (int i = 0; i < HG; ++i) {
                    K[i] = X::get(raw[0], i);
                    if (ONE && VEC > 1) K[i].y = K[i].x;
                }
#pragma unroll
                for (int i = 0; i < HS; ++i) s[i] = q[i] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                const int j = ONE ? i & (HS - 1) : i;
                const float2 d = f2_sub(X::get(raw[0], i), K[ONE ? 0 : i]);
                s[j] = __fadd2_rn(s[j], d);
                q[j] = __ffma2_rn(d, d, q[j]);
            }
        });
        if (visits > 0) merge((visits - 1) & ~(kGnShiftRows - 1), visits);
        float2* mine = st + (w.r * a.tile + w.col) * segs;
        if constexpr (ONE)
            mine[0] = make_float2(S[0].x, m2[0].x);
        else
            gn_collapse<VEC>(S, m2, static_cast<float>(visits), c, a, mine);
    }
    __syncthreads();
    gn_merge_threads<VEC>(a, w, st, segs, vis, sh, gs);
    __syncthreads();
    gn_merge_cluster(gs, w.ng, sh.wpg, 1, [&](int g, const float4& t) {
        const int gg = w.g0 + g;
        const int64_t bg = w.b * a.G + gg;
        const int ti = a.tpg == 1 ? 0 : w.t - quot(gg * a.D / VEC, a.by_tile);
        reinterpret_cast<float4*>(a.part)[(bg * a.tpg + ti) * a.chunks + k] = t;
        if (k == 0 && ti == 0) a.shift[bg] = gn_elem(xs + int64_t(gg) * a.D);
    });
}

// Output row chunk k of a tile.
template <class T, int VEC, bool ONE, int ACT>
__device__ __forceinline__ void gn_fwd_apply(const GnArgs& a, const GnTile& w, int k, float2* sm, void* ring) {
    using X = GnVec<T, VEC>;
    float2* fin = sm;  // (rest of the mean, rstd) per group of the tile
    float* mid = reinterpret_cast<float*>(sm + w.ng);  // its mean
    const int c = w.c0 + w.col * VEC;
    const int visits = w.on ? GnVisits(static_cast<int>(gn_chunk_len(a.S, a.out_rows, k)), a).of(w.r) : 0;
    // last rows first: what was summed last is the likeliest in L2
    const int64_t row = k * a.out_rows + w.r + int64_t(visits - 1) * a.par;
    const T* const p[1] = {static_cast<const T*>(a.x) + w.b * a.xb + row * a.xr + c};
    const int64_t step[1] = {-int64_t(a.par) * a.xr};
    // Nothing is read before this launch's own wait, x and the parameters
    // neither: the sums' wait orders what wrote them before this launch, but
    // only a wait of its own makes those writes visible to it.
    grid_wait();
    // (the rows and parameters travel while the states are merged)
    GnStream<T, VEC, 1> rows_in(p, step, visits, ring);
    typename X::Raw rg = X::zero(), rb = X::zero();
    if (w.on) {
        rg = X::load(static_cast<const T*>(a.gamma) + c);
        rb = X::load(static_cast<const T*>(a.beta) + c);
    }
    // The groups' states from every tile and chunk, lanes side by side.
    const GnShare sh(w.ng);
    const int lanes = sh.lanes, lane = threadIdx.x & (lanes - 1);
    for (int base = 0; base < w.ng << sh.bits; base += blockDim.x) {
        const int g = (base + static_cast<int>(threadIdx.x)) >> sh.bits;
        const bool on = g < w.ng;
        const int gg = w.g0 + (on ? g : 0);
        const int64_t bg = w.b * a.G + gg;
        const float4* src = reinterpret_cast<const float4*>(a.part) + bg * a.tpg * a.chunks;
        const int t0 = a.tpg == 1 ? w.t : quot(gg * a.D / VEC, a.by_tile);
        const int t1 = a.tpg == 1 ? w.t : quot(((gg + 1) * a.D - 1) / VEC, a.by_tile);
        const int n = (t1 - t0 + 1) * a.chunks;
        const float K = a.shift[bg];
        const float4 t = gn_merge([&](auto f) {
            if (on)
#pragma unroll 4
                for (int i = lane; i < n; i += lanes) f(src[i]);
        }, lanes);
        if (on && lane == 0) {
            const float rstd = gn_rstd(t.z, t.w, a.eps);
            const float2 m = gn_mean(K, t);
            fin[g] = make_float2(m.y, rstd);
            mid[g] = m.x;
            if (k == 0 && t0 == w.t) {
                if (a.mean) a.mean[bg] = m.x;
                if (a.rstd) a.rstd[bg] = rstd;
            }
        }
    }
    __syncthreads();
    if (!w.on) return;
    GnOut<T, VEC, ONE, ACT> out;
    gn_per_group<T, VEC, ONE>(out.K, c, a, [&](int g) { return mid[min(g - w.g0, w.ng - 1)]; });
    out.init(rg, rb, c, a, [&](int g) { return fin[min(g - w.g0, w.ng - 1)]; });
    T* yp = static_cast<T*>(a.y) + w.b * a.yb + row * a.yr + c;
    const int64_t ystep = -int64_t(a.par) * a.yr;
    rows_in.run([&](int, const auto& raw) {
        X::store(yp, out.apply(raw[0]));
        yp += ystep;
    });
}

// The split path's two launches, one CTA per tile and chunk.
template <class T, int VEC, bool ONE>
__global__ void __launch_bounds__(kGnMaxThreads, ONE ? 4 : 3) gn_fwd_split_sums(const GnArgs a) {
    extern __shared__ __align__(16) float2 states[];  // the merges' states, then the row stream's slots
    const int unit = quot(blockIdx.x, a.by_chunks);
    gn_fwd_sums<T, VEC, ONE>(a, gn_tile<VEC>(a, unit), static_cast<int>(blockIdx.x) - unit * a.chunks,
                             states, states + 2 * a.ring_at);
}

template <class T, int VEC, bool ONE, int ACT>
__global__ void __launch_bounds__(kGnMaxThreads, ONE ? 4 : 3) gn_fwd_split_apply(const GnArgs a) {
    extern __shared__ __align__(16) float2 states[];
    grid_release();
    const int unit = quot(blockIdx.x, a.by_out_chunks);
    gn_fwd_apply<T, VEC, ONE, ACT>(a, gn_tile<VEC>(a, unit), static_cast<int>(blockIdx.x) - unit * a.out_chunks,
                                   states, states + 2 * a.ring_at);
}

// ------------------------------------------------------------ launch
using GnKernel = void (*)(const GnArgs);

template <class T, int VEC, bool ONE, int ACT>
GnKernel gn_pick_chip(int V) {
    switch (V) {
        case 1: return gn_fwd_chip<T, VEC, ONE, ACT, 1>;
        case 2: return gn_fwd_chip<T, VEC, ONE, ACT, 2>;
        case 4: return gn_fwd_chip<T, VEC, ONE, ACT, 4>;
        case 8: return gn_fwd_chip<T, VEC, ONE, ACT, 8>;
        default: return nullptr;
    }
}

template <class T, int VEC, bool ONE>
cudaError_t gn_launch_fwd(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    const int64_t units = B * a.tiles;
    const int channels = a.tile * VEC;
    const int groups = static_cast<int>(gn_tile_groups(channels, a.D, false));
    const size_t smem = static_cast<size_t>(gn_smem_bytes(a.par, a.tile * (ONE ? 1 : a.segs), groups, p.threads));
    if (p.path == GN_PATH_CHIP) {
        const GnKernel k = act == NORM_ACT_SILU   ? gn_pick_chip<T, VEC, ONE, NORM_ACT_SILU>(p.per_thread)
                           : act == NORM_ACT_GELU ? gn_pick_chip<T, VEC, ONE, NORM_ACT_GELU>(p.per_thread)
                                                  : gn_pick_chip<T, VEC, ONE, NORM_ACT_NONE>(p.per_thread);
        if (k == nullptr) return cudaErrorInvalidValue;
        return gn_launch(reinterpret_cast<const void*>(k), units * a.cluster, p.threads, smem, a.cluster, s, a);
    }
    const auto all = [&](int64_t rows) {
        return smem + GnStream<T, VEC, 1>::ring_bytes((rows + a.par - 1) / a.par, p.threads);
    };
    const cudaError_t e = gn_launch(reinterpret_cast<const void*>(gn_fwd_split_sums<T, VEC, ONE>), units * a.chunks,
                                    p.threads, all(a.chunk_rows), 1, s, a);
    if (e != cudaSuccess) return e;
    const GnKernel k = act == NORM_ACT_SILU   ? gn_fwd_split_apply<T, VEC, ONE, NORM_ACT_SILU>
                       : act == NORM_ACT_GELU ? gn_fwd_split_apply<T, VEC, ONE, NORM_ACT_GELU>
                                              : gn_fwd_split_apply<T, VEC, ONE, NORM_ACT_NONE>;
    return gn_launch(reinterpret_cast<const void*>(k), units * a.out_chunks, p.threads, all(a.out_rows), 1, s, a);
}

template <class T>
cudaError_t gn_dispatch_fwd(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    const bool one = a.D % p.vec_elems == 0;
    if (p.vec_elems == full)
        return one ? gn_launch_fwd<T, full, true>(p, a, act, B, s) : gn_launch_fwd<T, full, false>(p, a, act, B, s);
    if constexpr (sizeof(T) == 2) {
        if (p.vec_elems == 2)
            return one ? gn_launch_fwd<T, 2, true>(p, a, act, B, s) : gn_launch_fwd<T, 2, false>(p, a, act, B, s);
    }
    return gn_launch_fwd<T, 1, true>(p, a, act, B, s);
}

}  // namespace libnorm
