// Group norm backward kernels.
//
//   gn_bwd_chip   a CTA, or a cluster, holds all rows of a sample's tile (x
//                 and dy) in registers: the sums and dx from one read.
//   gn_bwd_split_sums,  for tiles that do not fit a cluster: row chunks are
//   gn_bwd_split_apply  summed into the workspace; the second launch merges
//                       them and writes dx from a second read of x and dy.
//
// With d = x - mean, A = rstd gamma, z = d A + beta, dz = dy act'(z), the two
// sums S1 = sum dz and S2 = sum dz d per channel give everything: dbeta = S1,
// dgamma = rstd S2, and per group m1 = sum_c gamma S1 / n,
// m2 = sum_c gamma S2 / n (n = S D), from which
//     dx = A dz - rstd m1 - d rstd^3 m2.
// Per-thread sums in fp32 over at most kGnSumRows rows, then blocks of them.
//
// What bounds them (one GB300, copy bandwidth 6.8 TB/s, calls from a graph
// over inputs beyond L2):
//   gn_bwd_chip   launch and latency: bf16 2x256x1280 6.7 us, its two samples
//                 in clusters of 8 so that the column sums need no launch.
//   split         HBM, with x and dy read twice where they exceed L2: bf16
//                 4x65536x256 106 us, 6.3 TB/s of its 671 MB (sums 49 us at 5.7
//                 TB/s, two thirds of the issue slots in use; apply 64 at 6.2).
//                 f16 8x4096x320 23 us; f32 3x1517x180, two launches of about
//                 4 us, 9.0 us.
// A persistent kernel over bands of rows that stay in L2 took 173 us where the
// two launches then took 106.
#pragma once

#include "gn_kernels.cuh"
#include "norm_bwd.cuh"  // the fixed-order column sum of partial rows

namespace libnorm {

// (128 is no faster and its sums are off by a third more: dgamma of f32
// 13x28608x128 1.7e-7 with 32, 2.2e-7 with 128, against 64 bits.)
constexpr int kGnSumRows = 32;

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
        GnWalk k(c, a);
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
        GnWalk k(c, a);
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
// in row 0 of st as (S1, rstd S2), its share of (dbeta, dgamma), and the
// groups' gamma-weighted sums of them in gs. Every
// thread of the CTA calls it, after a barrier. Order of the additions: fixed
// by the CTA's shape.
template <class T, int VEC>
__device__ __forceinline__ void gn_bwd_merge_threads(const GnArgs& a, const GnTile& w, float2* st, int stride,
                                                     float2* gs) {
    // `deep` threads per state add every deep-th row slot, halve what is left
    // while it is more than 8, and one adds the rest. (Few channels leave up to
    // 256: one chain of them was off by 5 u of the root of the terms' squares.)
    const int deep = min(a.par, max(1, small_quot(blockDim.x, stride)));
    int left = a.par;
    if (deep > 1) {
        const int d = small_quot(threadIdx.x, stride), i = static_cast<int>(threadIdx.x) - d * stride;
        if (d < deep) {
            float2 t = st[d * stride + i];
#pragma unroll 4
            for (int r = d + deep; r < a.par; r += deep) t = __fadd2_rn(t, st[r * stride + i]);
            st[d * stride + i] = t;
        }
        __syncthreads();
        for (left = deep; left > 8;) {
            const int half = (left + 1) >> 1;
            if (d + half < left) st[d * stride + i] = __fadd2_rn(st[d * stride + i], st[(d + half) * stride + i]);
            __syncthreads();
            left = half;
        }
    }
    for (int i = threadIdx.x; i < stride; i += blockDim.x) {
        float2 t = st[i];
#pragma unroll 4
        for (int r = 1; r < left; ++r) t = __fadd2_rn(t, st[r * stride + i]);
        const int j = VEC == 1 ? 0 : quot(i, a.by_tile);
        const int ch = VEC == 1 ? i : (i - j * a.tile) * VEC + j;
        if (ch < w.nc) st[i] = make_float2(t.x, t.y * a.rstd[w.b * a.G + quot(w.c0 + ch, a.by_D)]);
    }
    __syncthreads();
    const T* gamma = static_cast<const T*>(a.gamma) + w.c0;
    const GnShare sh(w.ng);
    const int lanes = sh.lanes, lane = threadIdx.x & (lanes - 1);
    for (int base = 0; base < w.ng << sh.bits; base += blockDim.x) {
        const int g = (base + static_cast<int>(threadIdx.x)) >> sh.bits;
        float2 t = make_float2(0.f, 0.f);
        if (g < w.ng) {
            const int lo = max((w.g0 + g) * a.D - w.c0, 0);
            const int hi = min((w.g0 + g + 1) * a.D - w.c0, w.nc);
            for (int ch = lo + lane; ch < hi; ch += lanes)
                t = __ffma2_rn(f2_splat(gn_elem(gamma + ch)), st[gn_at<VEC>(ch, a.tile)], t);
        }
        group_sum2(t.x, t.y, lanes);
        if (g < w.ng && lane == 0) gs[g] = t;
    }
}

// The column sums of the cluster's `cl` CTAs, channels shared out over them,
// into partial row `row` of the column gradients.
template <int VEC>
__device__ __forceinline__ void gn_bwd_write_cols(const GnArgs& a, const GnTile& w, const float2* st, int rank,
                                                  int cl, int64_t row) {
    const int per = cl == 1 ? w.nc : small_quot(w.nc + cl - 1, cl);
    const int hi = min(w.nc, (rank + 1) * per);
    for (int ch = rank * per + static_cast<int>(threadIdx.x); ch < hi; ch += blockDim.x) {
        const int at = gn_at<VEC>(ch, a.tile);
        float2 t;
        if (cl > 1) {
            t = gn_peer(st, at, 0);
            for (int k = 1; k < cl; ++k) t = __fadd2_rn(t, gn_peer(st, at, k));
        } else {
            t = st[at];
        }
        a.colg[row * a.col_pitch + w.c0 + ch] = t.y;
        a.colb[row * a.col_pitch + w.c0 + ch] = t.x;
    }
}

// (u, v) of a group from its sums (m1 n, rstd m2 n).
__device__ __forceinline__ float2 gn_bwd_fin(const GnArgs& a, float2 t, int64_t bg) {
    const float inv = 1.f / (static_cast<float>(a.S) * static_cast<float>(a.D));
    const float r = a.rstd[bg];
    return make_float2(r * (t.x * inv), r * (r * (t.y * inv)));
}

template <class T, int VEC, bool ONE, int ACT, int V>
__global__ void __launch_bounds__(kGnMaxThreads) gn_bwd_chip(const GnArgs a) {
    using X = GnVec<T, VEC>;
    extern __shared__ float2 sm[];
    grid_release();
    grid_wait();
    // A cluster holds a sample's tile (cs CTAs), or, where all samples fit
    // (join), every sample's, so that the column sums meet in it too.
    const int cs = a.cluster, cl = cs * a.join;
    const int place = cl > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int own = place & ~(cs - 1);  // the first CTA of this sample
    const int rank = place - own;
    const int unit = quot(blockIdx.x, a.by_cluster);
    const GnTile w = gn_tile<VEC>(a, a.join > 1 ? (own >> a.cluster_bits) * a.tiles + unit : unit);
    const int stride = a.tile * VEC;
    float2* st = sm;
    float2* gs = st + a.par * stride;
    float2* fin = gs + w.ng;

    const int64_t row0 = int64_t(rank) * a.chunk_rows;
    const int rows = static_cast<int>(gn_chunk_len(a.S, a.chunk_rows, rank));
    const int c = w.c0 + w.col * VEC;
    const int visits = w.on ? GnVisits(rows, a).of(w.r) : 0;
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
    if (cl > 1)
        cluster_barrier();
    else
        __syncthreads();
    for (int g = threadIdx.x; g < w.ng; g += blockDim.x) {
        float2 t;
        if (cs > 1) {
            t = gn_peer(gs, g, own);
            for (int k = 1; k < cs; ++k) t = __fadd2_rn(t, gn_peer(gs, g, own + k));
        } else {
            t = gs[g];
        }
        fin[g] = gn_bwd_fin(a, t, w.b * a.G + w.g0 + g);
    }
    if (a.join > 1)
        gn_bwd_write_cols<VEC>(a, w, st, place, cl, 0);
    else
        gn_bwd_write_cols<VEC>(a, w, st, rank, cs, w.b);
    __syncthreads();
    if (cl > 1) cluster_arrive();  // this CTA has read its peers' sums
    if (w.on) {
        GnBwdOut<T, VEC, ONE> out;
        out.init(a, c, [&](int g) { return fin[min(g - w.g0, w.ng - 1)]; });
        T* yp = static_cast<T*>(a.y) + w.b * a.yb + (row0 + w.r) * a.yr + c;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < visits) X::store(yp + int64_t(v) * a.par * a.yr, out.apply(ch, rx[v], rdy[v]));
    }
    if (cl > 1) cluster_wait();
}

// Row chunk k of a tile: its groups' sums and its partial row of the column
// gradients into the workspace.
template <class T, int VEC, bool ONE, int ACT>
__device__ __forceinline__ void gn_bwd_sums(const GnArgs& a, const GnTile& w, int k, float2* sm, void* ring) {
    using X = GnVec<T, VEC>;
    const int stride = a.tile * VEC;
    float2* st = sm;
    float2* gs = st + a.par * stride;

    const int rows = static_cast<int>(gn_chunk_len(a.S, a.chunk_rows, k));
    const int c = w.c0 + w.col * VEC;
    const int visits = w.on ? GnVisits(rows, a).of(w.r) : 0;
    const int64_t row = k * a.chunk_rows + w.r;
    const T* const p[2] = {static_cast<const T*>(a.x) + w.b * a.xb + row * a.xr + c,
                           static_cast<const T*>(a.dy) + w.b * a.dyb + row * a.dyr + c};
    const int64_t step[2] = {int64_t(a.par) * a.xr, int64_t(a.par) * a.dyr};
    grid_wait();
    grid_release();
    GnStream<T, VEC, 2> rows_in(p, step, visits, ring);
    if (w.on) {
        GnBwdCh<T, VEC, ONE, ACT> ch;
        ch.init(a, w.b, c);
        // full blocks of rows are added up in the row slot's states
        float2 s1[X::H], s2[X::H];
        float2* mine = st + w.r * stride + w.col;
        auto fold = [&](bool first) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float2 t = make_float2((j & 1) ? s1[j / 2].y : s1[j / 2].x, (j & 1) ? s2[j / 2].y : s2[j / 2].x);
                mine[j * a.tile] = first ? t : __fadd2_rn(mine[j * a.tile], t);
            }
        };
#pragma unroll
        for (int i = 0; i < X::H; ++i) s1[i] = s2[i] = make_float2(0.f, 0.f);
        rows_in.run([&](int v, const auto& raw) {
            if (v > 0 && (v & (kGnSumRows - 1)) == 0) {
                fold(v == kGnSumRows);
#pragma unroll
                for (int i = 0; i < X::H; ++i) s1[i] = s2[i] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                const float2 d = ch.diff(raw[0], i);
                const float2 dz = ch.dz(raw[1], d, i);
                s1[i] = __fadd2_rn(s1[i], dz);
                s2[i] = __ffma2_rn(dz, d, s2[i]);
            }
        });
        fold(visits <= kGnSumRows);
    }
    __syncthreads();
    gn_bwd_merge_threads<T, VEC>(a, w, st, stride, gs);
    __syncthreads();
    for (int g = threadIdx.x; g < w.ng; g += blockDim.x) {
        const int gg = w.g0 + g;
        const int ti = a.tpg == 1 ? 0 : w.t - quot(gg * a.D / VEC, a.by_tile);
        static_cast<float2*>(a.part)[((w.b * a.G + gg) * a.tpg + ti) * a.chunks + k] = gs[g];
    }
    gn_bwd_write_cols<VEC>(a, w, st, 0, 1, w.b * a.chunks + k);
}

// Output row chunk k of a tile.
template <class T, int VEC, bool ONE, int ACT>
__device__ __forceinline__ void gn_bwd_apply(const GnArgs& a, const GnTile& w, int k, float2* sm, void* ring) {
    using X = GnVec<T, VEC>;
    float2* fin = sm;
    const int c = w.c0 + w.col * VEC;
    const int visits = w.on ? GnVisits(static_cast<int>(gn_chunk_len(a.S, a.out_rows, k)), a).of(w.r) : 0;
    // last rows first: what was summed last is the likeliest in L2
    const int64_t row = k * a.out_rows + w.r + int64_t(visits - 1) * a.par;
    const T* const p[2] = {static_cast<const T*>(a.x) + w.b * a.xb + row * a.xr + c,
                           static_cast<const T*>(a.dy) + w.b * a.dyb + row * a.dyr + c};
    const int64_t step[2] = {-int64_t(a.par) * a.xr, -int64_t(a.par) * a.dyr};
    grid_wait();  // before every read, as in the forward
    GnStream<T, VEC, 2> rows_in(p, step, visits, ring);
    GnBwdCh<T, VEC, ONE, ACT> ch;
    if (w.on) ch.init(a, w.b, c);
    const GnShare sh(w.ng);
    const int lanes = sh.lanes, lane = threadIdx.x & (lanes - 1);
    for (int base = 0; base < w.ng << sh.bits; base += blockDim.x) {
        const int g = (base + static_cast<int>(threadIdx.x)) >> sh.bits;
        const int gg = w.g0 + (g < w.ng ? g : 0);
        const int64_t bg = w.b * a.G + gg;
        const int touched = a.tpg == 1 ? 1 : quot(((gg + 1) * a.D - 1) / VEC, a.by_tile) - quot(gg * a.D / VEC, a.by_tile) + 1;
        const float2* src = static_cast<const float2*>(a.part) + bg * a.tpg * a.chunks;
        float2 t = make_float2(0.f, 0.f);
        if (g < w.ng)
#pragma unroll 4
            for (int i = lane; i < touched * a.chunks; i += lanes) t = __fadd2_rn(t, src[i]);
        group_sum2(t.x, t.y, lanes);
        if (g < w.ng && lane == 0) fin[g] = gn_bwd_fin(a, t, bg);
    }
    __syncthreads();
    if (!w.on) return;
    GnBwdOut<T, VEC, ONE> out;
    out.init(a, c, [&](int g) { return fin[min(g - w.g0, w.ng - 1)]; });
    T* yp = static_cast<T*>(a.y) + w.b * a.yb + row * a.yr + c;
    const int64_t ystep = -int64_t(a.par) * a.yr;
    rows_in.run([&](int, const auto& raw) {
        X::store(yp, out.apply(ch, raw[0], raw[1]));
        yp += ystep;
    });
}

// dgamma and dbeta of 32 columns from the partial rows: warp w adds rows w,
// w + warps, ... in that order, in blocks of kGnAddRows, then the warps' sums
// in warp order. (One chain of 2048 rows was off by 424 u where all had one
// sign.)
constexpr int kGnAddRows = 16;
__device__ __forceinline__ void gn_bwd_add_cols(const GnArgs& a, int block, float2* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int c = block * 32 + lane;
    float2 t = make_float2(0.f, 0.f);
    if (c < a.C)
        for (int p = warp; p < a.partials;) {
            const int stop = min(a.partials, p + kGnAddRows * warps);
            float2 block = make_float2(0.f, 0.f);
#pragma unroll 8
            for (; p < stop; p += warps)
                block = __fadd2_rn(block, make_float2(a.colg[p * a.col_pitch + c], a.colb[p * a.col_pitch + c]));
            t = __fadd2_rn(t, block);
        }
    sm[threadIdx.x] = t;
    __syncthreads();
    if (warp == 0 && c < a.C) {
        for (int w = 1; w < warps; ++w) t = __fadd2_rn(t, sm[w * 32 + lane]);
        a.dgamma[c] = t.x;
        a.dbeta[c] = t.y;
    }
}

// Row i of a.folds: the sum of the partial rows [P i / folds, P (i + 1) /
// folds) of 2 C values, 32 columns per CTA. Order fixed as above. Blocks of
// kGnSumRows rows, and these with the error of each addition kept (Knuth's
// two-sum): there may be 2^31 rows, which are counted in 64 bits for that.
static __global__ void __launch_bounds__(256) gn_bwd_fold(const GnArgs a) {
    __shared__ float sm[256];
    grid_release();
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.y, width = 2 * a.C, c = blockIdx.x * 32 + lane;
    const int64_t lo = int64_t(a.partials) * i / a.folds, hi = int64_t(a.partials) * (i + 1) / a.folds;
    float t = 0.f, rest = 0.f;
    if (c < width)
        for (int64_t p = lo + warp; p < hi;) {
            const int64_t stop = min(hi, p + kGnSumRows * 8);
            float block = 0.f;
#pragma unroll 8
            for (; p < stop; p += 8) block += a.colg[p * a.col_pitch + c];
            const float s = t + block, b = s - t;
            rest += (t - (s - b)) + (block - b);
            t = s;
        }
    if (isfinite(t)) t += rest;  // (an infinite sum has no rest)
    sm[threadIdx.x] = t;
    __syncthreads();
    if (warp == 0 && c < width) {
        for (int w = 1; w < 8; ++w) t += sm[w * 32 + lane];
        a.fold[int64_t(i) * width + c] = t;
    }
}

// The split path's two launches; the second also adds the partial rows of the
// column gradients, in its first CTAs, where they are not folded first.
__host__ __device__ __forceinline__ int gn_adders(const GnArgs& a) {
    return a.partials > 1 && a.folds == 0 ? (a.C + 31) / 32 : 0;
}

template <class T, int VEC, bool ONE, int ACT>
__global__ void __launch_bounds__(kGnMaxThreads, 2) gn_bwd_split_sums(const GnArgs a) {
    extern __shared__ __align__(16) float2 states[];  // the merges' states, then the row stream's slots
    const int unit = quot(blockIdx.x, a.by_chunks);
    gn_bwd_sums<T, VEC, ONE, ACT>(a, gn_tile<VEC>(a, unit), static_cast<int>(blockIdx.x) - unit * a.chunks,
                                  states, states + 2 * a.ring_at);
}

template <class T, int VEC, bool ONE, int ACT>
__global__ void __launch_bounds__(kGnMaxThreads, 2) gn_bwd_split_apply(const GnArgs a) {
    extern __shared__ __align__(16) float2 states[];
    grid_release();
    const int adders = gn_adders(a);
    const int i = static_cast<int>(blockIdx.x) - adders;
    if (i < 0) {
        grid_wait();
        gn_bwd_add_cols(a, blockIdx.x, states);
        return;
    }
    const int unit = quot(i, a.by_out_chunks);
    gn_bwd_apply<T, VEC, ONE, ACT>(a, gn_tile<VEC>(a, unit), i - unit * a.out_chunks, states,
                                   states + 2 * a.ring_at);
}

// ------------------------------------------------------------ launch
template <class T, int VEC, bool ONE, int ACT>
cudaError_t gn_launch_bwd(const gn_plan& p, const GnArgs& a, int64_t B, cudaStream_t s) {
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
        return gn_launch(k, B * a.tiles * a.cluster, p.threads, smem, a.cluster * a.join, s, a);
    }
    const int64_t units = B * a.tiles;
    const auto all = [&](int64_t rows) {
        return smem + GnStream<T, VEC, 2>::ring_bytes((rows + a.par - 1) / a.par, p.threads);
    };
    const cudaError_t e = gn_launch(reinterpret_cast<const void*>(gn_bwd_split_sums<T, VEC, ONE, ACT>),
                                    units * a.chunks, p.threads, all(a.chunk_rows), 1, s, a);
    if (e != cudaSuccess) return e;
    const int64_t adders = gn_adders(a);
    return gn_launch(reinterpret_cast<const void*>(gn_bwd_split_apply<T, VEC, ONE, ACT>),
                     units * a.out_chunks + adders, p.threads, all(a.out_rows), 1, s, a);
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
cudaError_t gn_dispatch_bwd(const gn_plan& p, const GnArgs& a, norm_act act, int64_t B, cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    constexpr int pair = sizeof(T) == 2 ? 2 : full;  // (fp32 has no 2-element accesses)
    if (B > 0 && a.S > 0) {
        const bool one = a.D % p.vec_elems == 0;
        cudaError_t e;
        if (p.vec_elems == full)
            e = one ? gn_launch_bwd_act<T, full, true>(p, a, act, B, s) : gn_launch_bwd_act<T, full, false>(p, a, act, B, s);
        else if (p.vec_elems == pair)
            e = one ? gn_launch_bwd_act<T, pair, true>(p, a, act, B, s) : gn_launch_bwd_act<T, pair, false>(p, a, act, B, s);
        else
            e = gn_launch_bwd_act<T, 1, true>(p, a, act, B, s);
        // one partial row: the kernel wrote dgamma and dbeta; the split path's
        // second launch adds a moderate number of them itself
        if (e != cudaSuccess || a.partials == 1 || (p.path != GN_PATH_CHIP && a.folds == 0)) return e;
    }
    // The partial rows of the column gradients (none: zeros), in a fixed order.
    const float* ws = a.colg;
    int64_t partials = a.partials;
    if (a.folds > 0) {
        void* fargs[] = {const_cast<GnArgs*>(&a)};
        const dim3 grid(static_cast<unsigned>((2 * a.C + 31) / 32), static_cast<unsigned>(a.folds));
        const cudaError_t e = launch_pdl(reinterpret_cast<const void*>(gn_bwd_fold), grid, dim3(256), 0, 1, s, fargs);
        if (e != cudaSuccess) return e;
        ws = a.fold;
        partials = a.folds;
    }
    int32_t N = a.C;
    float *o0 = a.dgamma, *o1 = a.dbeta;
    void* cargs[] = {&ws, &partials, &N, &o0, &o1};
    const bool wide = N % 4 == 0;
    const bool many = partials > 64;
    const int cols = wide ? 128 : 32;
    const void* fn = wide ? (many ? reinterpret_cast<const void*>(norm_bwd_colsum<2, 4, 32>)
                                  : reinterpret_cast<const void*>(norm_bwd_colsum<2, 4, 8>))
                          : (many ? reinterpret_cast<const void*>(norm_bwd_colsum<2, 1, 32>)
                                  : reinterpret_cast<const void*>(norm_bwd_colsum<2, 1, 8>));
    return launch_pdl(fn, dim3(static_cast<unsigned>((N + cols - 1) / cols)), dim3(many ? 1024 : 256), 0, 1, s, cargs);
}

}  // namespace libnorm
