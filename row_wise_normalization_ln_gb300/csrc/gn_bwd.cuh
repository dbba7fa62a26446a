// Group norm backward kernels.
//
//   gn_bwd_chip   a CTA, or a cluster, holds all rows of a sample's tile (x
//                 and dy) in registers: the sums and dx from one read.
//   gn_bwd_sums,  for tiles that do not fit a cluster: the first kernel sums
//   gn_bwd_apply  row chunks into the workspace, the second merges the chunks
//                 and writes dx from a second read of x and dy.
//
// With d = x - mean, A = rstd gamma, z = d A + beta, dz = dy act'(z), the two
// sums S1 = sum dz and S2 = sum dz d per channel give everything: dbeta = S1,
// dgamma = rstd S2, and per group m1 = sum_c gamma S1 / n,
// m2 = sum_c gamma S2 / n (n = S D), from which
//     dx = A dz - rstd m1 - d rstd^3 m2.
// Per-thread sums in fp32 over at most kGnSumRows rows, then blocks of them.
#pragma once

#include "gn_kernels.cuh"
#include "norm_bwd.cuh"  // the fixed-order column sum of partial rows

namespace libnorm {

constexpr int kGnSumRows = 128;

// A thread's channels: d and dz of an access.
template <class T, int VEC, bool ONE, int ACT>
struct GnBwdCh {
    using X = GnVec<T, VEC>;
    static constexpr int HG = ONE ? 1 : X::H;
    float2 mu[HG], A[X::H], be[X::H];

    __device__ __forceinline__ void init(const GnArgs& a, int64_t b, int c) {
        const auto rg = X::load(static_cast<const T*>(a.gamma) + c);
        const auto rb = X::load(static_cast<const T*>(a.beta) + c);
        const float* mean = a.mean + b * a.G;
        const float* rstd = a.rstd + b * a.G;
        GnWalk k(c, a.D);
        float2 m = f2_splat(mean[k.g]), r = f2_splat(rstd[k.g]);
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            if constexpr (!ONE) {
                m.x = mean[k.g];
                r.x = rstd[k.g];
                k.next();
                m.y = mean[min(k.g, a.G - 1)];
                r.y = rstd[min(k.g, a.G - 1)];
                k.next();
                k.g = min(k.g, a.G - 1);
            }
            if (i < HG) mu[i] = m;
            A[i] = __fmul2_rn(r, X::get(rg, i));
            be[i] = X::get(rb, i);
        }
    }
    __device__ __forceinline__ float2 diff(const typename X::Raw& x, int i) const {
        return f2_sub(X::get(x, i), mu[ONE ? 0 : i]);
    }
    __device__ __forceinline__ float2 dz(const typename X::Raw& dy, float2 d, int i) const {
        const float2 v = X::get(dy, i);
        if constexpr (ACT == NORM_ACT_NONE) return v;
        const float2 z = __ffma2_rn(d, A[i], be[i]);
        return __fmul2_rn(v, gn_act_slope2<ACT>(z));
    }
};

// dx = A dz - u - d v with u = rstd m1, v = rstd^3 m2 of the channel's group.
template <class T, int VEC, bool ONE>
struct GnBwdOut {
    using X = GnVec<T, VEC>;
    static constexpr int HG = ONE ? 1 : X::H;
    float2 u[HG], v[HG];

    template <class Fin>
    __device__ __forceinline__ void init(const GnArgs& a, int c, Fin fin) {
        GnWalk k(c, a.D);
#pragma unroll
        for (int i = 0; i < HG; ++i) {
            const float2 fa = fin(k.g);
            float2 fb = fa;
            if constexpr (!ONE) {
                k.next();
                fb = fin(k.g);
                k.next();
            }
            u[i] = make_float2(fa.x, fb.x);
            v[i] = make_float2(fa.y, fb.y);
        }
    }
    template <int ACT>
    __device__ __forceinline__ typename X::Raw apply(const GnBwdCh<T, VEC, ONE, ACT>& ch, const typename X::Raw& x,
                                                     const typename X::Raw& dy) const {
        typename X::Raw out = X::zero();
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            const int j = ONE ? 0 : i;
            const float2 d = ch.diff(x, i);
            const float2 g = __ffma2_rn(ch.A[i], ch.dz(dy, d, i), make_float2(-u[j].x, -u[j].y));
            X::set(out, i, __ffma2_rn(make_float2(-d.x, -d.y), v[j], g));
        }
        return out;
    }
};

// A thread's column sums (S1, S2) into its row slot's states. The state of a
// tile's channel is at gn_at(channel): the channels of an access lie `tile`
// states apart, so that the lanes of a warp write side by side.
template <int VEC>
__device__ __forceinline__ int gn_at(int ch, int tile) {
    return VEC == 1 ? ch : (ch % VEC) * tile + ch / VEC;
}
template <int VEC>
__device__ __forceinline__ void gn_bwd_put(float2* st, int tile, int col, const float2* s1, const float2* s2) {
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i) {
        st[2 * i * tile + col] = make_float2(s1[i].x, s2[i].x);
        if (VEC > 1) st[(2 * i + 1) * tile + col] = make_float2(s1[i].y, s2[i].y);
    }
}

// The CTA's column sums from its row slots' states (st[r * stride + i]), left
// in row 0 of st, and the groups' gamma-weighted sums of them in gs. Every
// thread of the CTA calls it, after a barrier. Order of the additions: fixed
// by the CTA's shape.
template <class T, int VEC>
__device__ __forceinline__ void gn_bwd_merge_threads(const GnArgs& a, const GnTile& w, float2* st, int stride,
                                                     float2* gs) {
    // `deep` threads per state add every deep-th row slot, then one adds theirs
    const int deep = min(a.par, max(1, static_cast<int>(blockDim.x) / stride));
    if (deep > 1) {
        const int d = static_cast<int>(threadIdx.x) / stride, i = static_cast<int>(threadIdx.x) - d * stride;
        if (d < deep) {
            float2 t = st[d * stride + i];
#pragma unroll 4
            for (int r = d + deep; r < a.par; r += deep) t = __fadd2_rn(t, st[r * stride + i]);
            st[d * stride + i] = t;
        }
        __syncthreads();
    }
    const int left = deep > 1 ? deep : a.par;
    if (left > 1) {
        for (int i = threadIdx.x; i < stride; i += blockDim.x) {
            float2 t = st[i];
#pragma unroll 4
            for (int r = 1; r < left; ++r) t = __fadd2_rn(t, st[r * stride + i]);
            st[i] = t;
        }
        __syncthreads();
    }
    const T* gamma = static_cast<const T*>(a.gamma) + w.c0;
    int lanes = 32;
    while (lanes > 1 && lanes * w.ng > static_cast<int>(blockDim.x)) lanes >>= 1;
    const int lane = threadIdx.x & (lanes - 1);
    const int rounds = (w.ng * lanes + blockDim.x - 1) / blockDim.x;
    for (int it = 0; it < rounds; ++it) {
        const int g = (static_cast<int>(threadIdx.x) + it * static_cast<int>(blockDim.x)) / lanes;
        float2 t = make_float2(0.f, 0.f);
        if (g < w.ng) {
            const int lo = max((w.g0 + g) * a.D - w.c0, 0);
            const int hi = min((w.g0 + g + 1) * a.D - w.c0, w.nc);
            for (int ch = lo + lane; ch < hi; ch += lanes)
                t = __ffma2_rn(f2_splat(gn_elem(gamma + ch)), st[gn_at<VEC>(ch, a.tile)], t);
        }
        t.x = group_sum(t.x, lanes);
        t.y = group_sum(t.y, lanes);
        if (g < w.ng && lane == 0) gs[g] = t;
    }
}

// The cluster's column sums, channels shared out over its CTAs, into partial
// row `row` of the column gradients (dgamma = rstd S2, dbeta = S1).
template <int VEC>
__device__ __forceinline__ void gn_bwd_write_cols(const GnArgs& a, const GnTile& w, const float2* st, int rank,
                                                  int cs, int64_t row) {
    const int per = (w.nc + cs - 1) / cs;
    const int hi = min(w.nc, (rank + 1) * per);
    for (int ch = rank * per + static_cast<int>(threadIdx.x); ch < hi; ch += blockDim.x) {
        float2 t;
        if (cs > 1) {
            t = gn_peer(st, gn_at<VEC>(ch, a.tile), 0);
            for (int k = 1; k < cs; ++k) t = __fadd2_rn(t, gn_peer(st, gn_at<VEC>(ch, a.tile), k));
        } else {
            t = st[gn_at<VEC>(ch, a.tile)];
        }
        const int c = w.c0 + ch;
        a.colg[row * a.col_pitch + c] = t.y * a.rstd[w.b * a.G + c / a.D];
        a.colb[row * a.col_pitch + c] = t.x;
    }
}

// (u, v) of a group from its sums (m1 n, m2 n).
__device__ __forceinline__ float2 gn_bwd_fin(const GnArgs& a, float2 t, int64_t bg) {
    const float inv = 1.f / (static_cast<float>(a.S) * static_cast<float>(a.D));
    const float r = a.rstd[bg];
    return make_float2(r * (t.x * inv), r * (r * (r * (t.y * inv))));
}

template <class T, int VEC, bool ONE, int ACT, int V>
__global__ void __launch_bounds__(kGnMaxThreads) gn_bwd_chip(const GnArgs a) {
    using X = GnVec<T, VEC>;
    extern __shared__ float2 sm[];
    grid_release();
    grid_wait();
    const int cs = a.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const GnTile w = gn_tile<VEC>(a, blockIdx.x / cs);
    const int stride = a.tile * VEC;
    float2* st = sm;
    float2* gs = st + a.par * stride;
    float2* fin = gs + (a.tile * VEC - 1 + a.D - 1) / a.D + 1;

    const int64_t row0 = int64_t(rank) * a.chunk_rows;
    const int rows = static_cast<int>(gn_chunk_len(a.S, a.chunk_rows, rank));
    const int c = w.c0 + w.col * VEC;
    const int visits = w.on ? GnVisits(rows, a.par).of(w.r) : 0;
    const T* xp = static_cast<const T*>(a.x) + w.b * a.xb + (row0 + w.r) * a.xr + c;
    const T* dyp = static_cast<const T*>(a.dy) + w.b * a.dyb + (row0 + w.r) * a.dyr + c;
    typename X::Raw rx[V], rdy[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < visits) {
            rx[v] = X::load(xp + int64_t(v) * a.par * a.xr);
            rdy[v] = X::load(dyp + int64_t(v) * a.par * a.dyr);
        }
    GnBwdCh<T, VEC, ONE, ACT> ch;
    if (w.on) {
        ch.init(a, w.b, c);
        float2 s1[X::H], s2[X::H];
#pragma unroll
        for (int i = 0; i < X::H; ++i) s1[i] = s2[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < visits) {
#pragma unroll
                for (int i = 0; i < X::H; ++i) {
                    const float2 d = ch.diff(rx[v], i);
                    const float2 dz = ch.dz(rdy[v], d, i);
                    s1[i] = __fadd2_rn(s1[i], dz);
                    s2[i] = __ffma2_rn(dz, d, s2[i]);
                }
            }
        gn_bwd_put<VEC>(st + w.r * stride, a.tile, w.col, s1, s2);
    }
    __syncthreads();
    gn_bwd_merge_threads<T, VEC>(a, w, st, stride, gs);
    if (cs > 1)
        cluster_barrier();
    else
        __syncthreads();
    for (int g = threadIdx.x; g < w.ng; g += blockDim.x) {
        float2 t;
        if (cs > 1) {
            t = gn_peer(gs, g, 0);
            for (int k = 1; k < cs; ++k) t = __fadd2_rn(t, gn_peer(gs, g, k));
        } else {
            t = gs[g];
        }
        fin[g] = gn_bwd_fin(a, t, w.b * a.G + w.g0 + g);
    }
    gn_bwd_write_cols<VEC>(a, w, st, rank, cs, w.b);
    __syncthreads();
    if (cs > 1) cluster_arrive();  // this CTA has read its peers' sums
    if (w.on) {
        GnBwdOut<T, VEC, ONE> out;
        out.init(a, c, [&](int g) { return fin[min(g - w.g0, w.ng - 1)]; });
        T* yp = static_cast<T*>(a.y) + w.b * a.yb + (row0 + w.r) * a.yr + c;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < visits) X::store(yp + int64_t(v) * a.par * a.yr, out.apply(ch, rx[v], rdy[v]));
    }
    if (cs > 1) cluster_wait();
}

template <class T, int VEC, bool ONE, int ACT>
__global__ void __launch_bounds__(kGnMaxThreads) gn_bwd_sums(const GnArgs a) {
    using X = GnVec<T, VEC>;
    constexpr int U = 4;
    extern __shared__ float2 sm[];
    grid_release();
    grid_wait();
    const int cs = a.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int64_t unit = blockIdx.x / a.chunks;
    const int k = static_cast<int>(blockIdx.x - unit * a.chunks);
    const GnTile w = gn_tile<VEC>(a, unit);
    const int stride = a.tile * VEC;
    float2* st = sm;
    float2* gs = st + a.par * stride;

    const int rows = static_cast<int>(gn_chunk_len(a.S, a.chunk_rows, k));
    const int c = w.c0 + w.col * VEC;
    if (w.on) {
        const int visits = GnVisits(rows, a.par).of(w.r);
        const int64_t row = k * a.chunk_rows + w.r;
        const T* xp = static_cast<const T*>(a.x) + w.b * a.xb + row * a.xr + c;
        const T* dyp = static_cast<const T*>(a.dy) + w.b * a.dyb + row * a.dyr + c;
        const int64_t xstep = int64_t(a.par) * a.xr, dystep = int64_t(a.par) * a.dyr;
        GnBwdCh<T, VEC, ONE, ACT> ch;
        ch.init(a, w.b, c);
        float2 t1[X::H], t2[X::H];
#pragma unroll
        for (int i = 0; i < X::H; ++i) t1[i] = t2[i] = make_float2(0.f, 0.f);
        for (int v0 = 0; v0 < visits;) {
            const int stop = min(visits, v0 + kGnSumRows);
            float2 s1[X::H], s2[X::H];
#pragma unroll
            for (int i = 0; i < X::H; ++i) s1[i] = s2[i] = make_float2(0.f, 0.f);
            for (; v0 < stop; v0 += U) {
                typename X::Raw rx[U], rdy[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v0 + u < stop) {
                        rx[u] = X::load(xp + u * xstep);
                        rdy[u] = X::load(dyp + u * dystep);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v0 + u < stop) {
#pragma unroll
                        for (int i = 0; i < X::H; ++i) {
                            const float2 d = ch.diff(rx[u], i);
                            const float2 dz = ch.dz(rdy[u], d, i);
                            s1[i] = __fadd2_rn(s1[i], dz);
                            s2[i] = __ffma2_rn(dz, d, s2[i]);
                        }
                    }
                xp += U * xstep;
                dyp += U * dystep;
            }
            v0 = stop;
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                t1[i] = __fadd2_rn(t1[i], s1[i]);
                t2[i] = __fadd2_rn(t2[i], s2[i]);
            }
        }
        gn_bwd_put<VEC>(st + w.r * stride, a.tile, w.col, t1, t2);
    }
    __syncthreads();
    gn_bwd_merge_threads<T, VEC>(a, w, st, stride, gs);
    if (cs > 1)
        cluster_barrier();
    else
        __syncthreads();
    const int p0 = k / cs, parts = a.chunks / cs;
    for (int g = rank + cs * static_cast<int>(threadIdx.x); g < w.ng; g += cs * blockDim.x) {
        float2 t;
        if (cs > 1) {
            t = gn_peer(gs, g, 0);
            for (int j = 1; j < cs; ++j) t = __fadd2_rn(t, gn_peer(gs, g, j));
        } else {
            t = gs[g];
        }
        const int gg = w.g0 + g;
        const int ti = a.tpg == 1 ? 0 : w.t - (gg * a.D / VEC) / a.tile;
        a.part[((w.b * a.G + gg) * a.tpg + ti) * parts + p0] = t;
    }
    gn_bwd_write_cols<VEC>(a, w, st, rank, cs, w.b * parts + p0);
    if (cs > 1) cluster_barrier();  // no CTA leaves while a peer reads its sums
}

template <class T, int VEC, bool ONE, int ACT>
__global__ void __launch_bounds__(kGnMaxThreads) gn_bwd_apply(const GnArgs a) {
    using X = GnVec<T, VEC>;
    constexpr int U = 4;
    extern __shared__ float2 sm[];
    grid_release();
    grid_wait();
    float2* fin = sm;
    const int64_t id = int64_t(gridDim.x) - 1 - blockIdx.x;  // last chunks first, as in the forward
    const int64_t unit = id / a.out_chunks;
    const int k = static_cast<int>(id - unit * a.out_chunks);
    const GnTile w = gn_tile<VEC>(a, unit);
    const int parts = a.chunks / a.cluster;
    int lanes = 32;
    while (lanes > 1 && lanes * w.ng > static_cast<int>(blockDim.x)) lanes >>= 1;
    const int lane = threadIdx.x & (lanes - 1);
    const int rounds = (w.ng * lanes + blockDim.x - 1) / blockDim.x;
    for (int it = 0; it < rounds; ++it) {
        const int g = (static_cast<int>(threadIdx.x) + it * static_cast<int>(blockDim.x)) / lanes;
        const int gg = w.g0 + (g < w.ng ? g : 0);
        const int64_t bg = w.b * a.G + gg;
        const int touched = a.tpg == 1 ? 1 : ((gg + 1) * a.D - 1) / VEC / a.tile - gg * a.D / VEC / a.tile + 1;
        const float2* src = a.part + bg * a.tpg * parts;
        float2 t = make_float2(0.f, 0.f);
        if (g < w.ng)
#pragma unroll 4
            for (int i = lane; i < touched * parts; i += lanes) t = __fadd2_rn(t, src[i]);
        t.x = group_sum(t.x, lanes);
        t.y = group_sum(t.y, lanes);
        if (g < w.ng && lane == 0) fin[g] = gn_bwd_fin(a, t, bg);
    }
    __syncthreads();
    if (!w.on) return;
    const int visits = GnVisits(static_cast<int>(gn_chunk_len(a.S, a.out_rows, k)), a.par).of(w.r);
    const int c = w.c0 + w.col * VEC;
    GnBwdCh<T, VEC, ONE, ACT> ch;
    ch.init(a, w.b, c);
    GnBwdOut<T, VEC, ONE> out;
    out.init(a, c, [&](int g) { return fin[min(g - w.g0, w.ng - 1)]; });
    const int64_t row = k * a.out_rows + w.r;
    const T* xp = static_cast<const T*>(a.x) + w.b * a.xb + row * a.xr + c;
    const T* dyp = static_cast<const T*>(a.dy) + w.b * a.dyb + row * a.dyr + c;
    T* yp = static_cast<T*>(a.y) + w.b * a.yb + row * a.yr + c;
    const int64_t xstep = int64_t(a.par) * a.xr, dystep = int64_t(a.par) * a.dyr, ystep = int64_t(a.par) * a.yr;
    for (int v = 0; v < visits; v += U) {
        typename X::Raw rx[U], rdy[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u < visits) {
                rx[u] = X::load(xp + u * xstep);
                rdy[u] = X::load(dyp + u * dystep);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u < visits) X::store(yp + u * ystep, out.apply(ch, rx[u], rdy[u]));
        xp += U * xstep;
        dyp += U * dystep;
        yp += U * ystep;
    }
}

// ------------------------------------------------------------ launch
template <class T, int VEC, bool ONE, int ACT>
cudaError_t gn_launch_bwd(const gn_plan& p, const GnArgs& a, int64_t B, cudaStream_t s) {
    const int64_t units = B * a.tiles;
    const int channels = a.tile * VEC;
    const int groups = static_cast<int>(gn_tile_groups(channels, a.D, false));
    const size_t smem = static_cast<size_t>(gn_smem_bytes(a.par, channels, groups, p.threads));
    if (p.path == GN_PATH_CHIP) {
        const void* k = nullptr;
        switch (p.per_thread) {
            case 1: k = reinterpret_cast<const void*>(gn_bwd_chip<T, VEC, ONE, ACT, 1>); break;
            case 2: k = reinterpret_cast<const void*>(gn_bwd_chip<T, VEC, ONE, ACT, 2>); break;
            case 4: k = reinterpret_cast<const void*>(gn_bwd_chip<T, VEC, ONE, ACT, 4>); break;
            default: return cudaErrorInvalidValue;
        }
        return gn_launch(k, units * a.cluster, p.threads, smem, a.cluster, s, a);
    }
    const cudaError_t e = gn_launch(reinterpret_cast<const void*>(gn_bwd_sums<T, VEC, ONE, ACT>), units * a.chunks,
                                    p.threads, smem, a.cluster, s, a);
    if (e != cudaSuccess) return e;
    return gn_launch(reinterpret_cast<const void*>(gn_bwd_apply<T, VEC, ONE, ACT>), units * a.out_chunks, p.threads,
                     static_cast<size_t>(gn_smem_bytes(0, 0, groups, 0)), 1, s, a);
}

template <class T, int VEC, bool ONE>
cudaError_t gn_launch_bwd_act(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    switch (act) {
        case NORM_ACT_SILU: return gn_launch_bwd<T, VEC, ONE, NORM_ACT_SILU>(p, a, B, s);
        case NORM_ACT_GELU: return gn_launch_bwd<T, VEC, ONE, NORM_ACT_GELU>(p, a, B, s);
        default: return gn_launch_bwd<T, VEC, ONE, NORM_ACT_NONE>(p, a, B, s);
    }
}

template <class T>
cudaError_t gn_dispatch_bwd(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, float* dgamma, float* dbeta,
                            cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    const bool one = a.D % p.vec_elems == 0;
    int64_t partials = 0;
    if (B > 0 && a.S > 0) {
        partials = p.path == GN_PATH_CHIP ? B : B * (a.chunks / a.cluster);
        cudaError_t e;
        if (p.vec_elems == full)
            e = one ? gn_launch_bwd_act<T, full, true>(p, a, act, B, s) : gn_launch_bwd_act<T, full, false>(p, a, act, B, s);
        else if (sizeof(T) == 2 && p.vec_elems == 2)
            e = one ? gn_launch_bwd_act<T, sizeof(T) == 2 ? 2 : 1, true>(p, a, act, B, s)
                    : gn_launch_bwd_act<T, sizeof(T) == 2 ? 2 : full, false>(p, a, act, B, s);
        else
            e = gn_launch_bwd_act<T, 1, true>(p, a, act, B, s);
        if (e != cudaSuccess) return e;
        if (partials == 1) return cudaSuccess;  // the kernel wrote dgamma and dbeta themselves
    }
    // the partial rows of the column gradients, in a fixed order (none: zeros)
    const float* ws = a.colg;
    int32_t N = a.C;
    float *o0 = dgamma, *o1 = dbeta;
    void* cargs[] = {&ws, &partials, &N, &o0, &o1};
    const bool wide = N % 4 == 0 && (reinterpret_cast<uintptr_t>(ws) & 15u) == 0;
    const bool many = partials > 64;
    const int cols = wide ? 128 : 32;
    const void* fn = wide ? (many ? reinterpret_cast<const void*>(norm_bwd_colsum<2, 4, 32>)
                                  : reinterpret_cast<const void*>(norm_bwd_colsum<2, 4, 8>))
                          : (many ? reinterpret_cast<const void*>(norm_bwd_colsum<2, 1, 32>)
                                  : reinterpret_cast<const void*>(norm_bwd_colsum<2, 1, 8>));
    return launch_pdl(fn, dim3(static_cast<unsigned>((N + cols - 1) / cols)), dim3(many ? 1024 : 256), 0, 1, s, cargs);
}

}  // namespace libnorm
