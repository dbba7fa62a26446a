// Group norm forward kernels.
//
//   gn_fwd_chip   a CTA, or a cluster, holds all rows of a sample's tile in
//                 registers: statistics, activation and output from one read.
//   gn_fwd_sums,  for tiles that do not fit a cluster: the first kernel sums
//   gn_fwd_apply  row chunks into the workspace, the second merges the chunks
//                 and writes y from a second read of x (from L2 where it fits).
//
// Statistics: differences d = x - K from a shift K near the data, so that a
// group whose mean dwarfs its spread keeps its digits (x - K of nearby values
// is exact). Per-thread states (count, mean, M2 = sum (d - mean)^2) merge in
// the k-way form mean = sum n_t m_t / n, M2 = sum M2_t + n_t (m_t - mean)^2,
// which is what any sequence of pairwise merges reaches; the variance is
// never formed as E[x^2] - E[x]^2 of unshifted values. All in fp32.
#pragma once

#include "gn_kernels.cuh"

namespace libnorm {

// Merges the CTA's thread states st[r * stride + u] (mean, M2 of
// visits(r) * WIDTH values each) into the groups' states gs[g - g0]; one warp
// per group. Every thread of the CTA calls it, after a barrier.
template <int WIDTH>
__device__ __forceinline__ void gn_merge_threads(const GnArgs& a, const GnTile& w, const float2* st, int stride,
                                                 int64_t rows, float2* gs) {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < w.ng; g += blockDim.x >> 5) {
        const int lo = max((w.g0 + g) * a.D - w.c0, 0) / WIDTH;
        const int hi = min((w.g0 + g + 1) * a.D - w.c0, w.nc) / WIDTH;
        const int n = hi - lo;
        float s = 0.f;
        for (int i = lane; i < n * a.par; i += 32) {
            const int r = i / n;
            s = fmaf(static_cast<float>(gn_visits(rows, r, a.par)), st[r * stride + lo + (i - r * n)].x, s);
        }
        const float count = static_cast<float>(rows) * static_cast<float>(n);
        const float mean = rows > 0 ? group_sum(s, 32) / count : 0.f;
        float q = 0.f;
        for (int i = lane; i < n * a.par; i += 32) {
            const int r = i / n;
            const int v = gn_visits(rows, r, a.par);
            if (v > 0) {
                const float2 e = st[r * stride + lo + (i - r * n)];
                const float d = e.x - mean;
                q += fmaf(static_cast<float>(v * WIDTH) * d, d, e.y);
            }
        }
        q = group_sum(q, 32);
        if (lane == 0) gs[g] = make_float2(mean, q);
    }
}

// y = act(d * s + o) per channel: s = rstd * gamma, o = beta - mu * s, with
// mu the group's mean relative to the shift K and d = x - K.
template <class T, int VEC, int ACT>
struct GnOut {
    using X = GnVec<T, VEC>;
    float2 K[X::H], s[X::H], o[X::H];

    // fin(g): float2 (mu, rstd) of group g; shift(g): K of group g.
    template <class Fin, class Shift>
    __device__ __forceinline__ void init(const GnArgs& a, int c, Fin fin, Shift shift) {
        const T* gamma = static_cast<const T*>(a.gamma) + c;
        const T* beta = static_cast<const T*>(a.beta) + c;
        const auto rg = X::load(gamma), rb = X::load(beta);
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            const int ga = (c + 2 * i) / a.D;
            const int gb = VEC == 1 ? ga : (c + 2 * i + 1) / a.D;
            const float2 fa = fin(ga), fb = fin(gb);
            const float2 gm = X::get(rg, i), be = X::get(rb, i);
            K[i] = make_float2(shift(ga), shift(gb));
            s[i] = make_float2(fa.y * gm.x, fb.y * gm.y);
            o[i] = make_float2(fmaf(-fa.x, s[i].x, be.x), fmaf(-fb.x, s[i].y, be.y));
        }
    }
    __device__ __forceinline__ typename X::Raw apply(const typename X::Raw& r) const {
        typename X::Raw out = X::zero();
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            const float2 z = __ffma2_rn(f2_sub(X::get(r, i), K[i]), s[i], o[i]);
            X::set(out, i, make_float2(gn_act<ACT>(z.x), gn_act<ACT>(z.y)));
        }
        return out;
    }
};

template <class T, int VEC, bool ONE, int ACT, int V>
__global__ void __launch_bounds__(kGnMaxThreads) gn_fwd_chip(const GnArgs a) {
    using X = GnVec<T, VEC>;
    extern __shared__ float2 sm[];
    grid_release();
    grid_wait();
    const int cs = a.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const GnTile w = gn_tile<VEC>(a, blockIdx.x / cs);
    const int stride = ONE ? a.tile : a.tile * VEC;
    float2* st = sm;
    float2* gs = st + a.par * stride;
    const int gcap = ONE ? (a.tile * VEC) / a.D : (a.tile * VEC - 1 + a.D - 1) / a.D + 1;
    float2* fin = gs + gcap;

    const int64_t row0 = int64_t(rank) * a.chunk_rows;
    const int rows = static_cast<int>(gn_chunk_len(a.S, a.chunk_rows, rank));
    const int c = w.c0 + w.col * VEC;
    const T* xs = static_cast<const T*>(a.x) + w.b * a.xb;
    const T* xp = xs + (row0 + w.r) * a.xr + c;
    typename X::Raw raw[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (w.on && w.r + v * a.par < rows) raw[v] = X::load(xp + int64_t(v) * a.par * a.xr);

    // the shift of a group: its first element in the sample's first row
    float2 K[X::H];
#pragma unroll
    for (int i = 0; i < X::H; ++i) {
        K[i] = make_float2(0.f, 0.f);
        if (w.on) {
            if (ONE && i > 0)
                K[i] = K[0];
            else {
                const int ga = (c + 2 * i) / a.D;
                K[i].x = gn_elem(xs + int64_t(ga) * a.D);
                K[i].y = VEC == 1 ? 0.f : ONE ? K[i].x : gn_elem(xs + int64_t((c + 2 * i + 1) / a.D) * a.D);
            }
        }
    }
    const int visits = w.on ? gn_visits(rows, w.r, a.par) : 0;
    float2 s[X::H], q[X::H];
#pragma unroll
    for (int i = 0; i < X::H; ++i) s[i] = q[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < visits) {
#pragma unroll
            for (int i = 0; i < X::H; ++i) s[i] = __fadd2_rn(s[i], f2_sub(X::get(raw[v], i), K[i]));
        }
    const float inv = visits > 0 ? 1.f / static_cast<float>(visits) : 0.f;
    if constexpr (ONE) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < X::H; ++i) t += f2_sum<VEC>(s[i]);
        const float m = t * inv * (1.f / VEC);
#pragma unroll
        for (int i = 0; i < X::H; ++i) s[i] = f2_splat(m);
    } else {
#pragma unroll
        for (int i = 0; i < X::H; ++i) s[i] = __fmul2_rn(s[i], f2_splat(inv));
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < visits) {
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                const float2 d = f2_sub(f2_sub(X::get(raw[v], i), K[i]), s[i]);
                q[i] = __ffma2_rn(d, d, q[i]);
            }
        }
    if (w.on) {
        if constexpr (ONE) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < X::H; ++i) t += f2_sum<VEC>(q[i]);
            st[w.r * stride + w.col] = make_float2(s[0].x, t);
        } else {
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                st[w.r * stride + w.col * VEC + 2 * i] = make_float2(s[i].x, q[i].x);
                st[w.r * stride + w.col * VEC + 2 * i + 1] = make_float2(s[i].y, q[i].y);
            }
        }
    }
    __syncthreads();
    gn_merge_threads<ONE ? VEC : 1>(a, w, st, stride, rows, gs);
    if (cs > 1)
        cluster_barrier();
    else
        __syncthreads();
    const float count = static_cast<float>(a.S) * static_cast<float>(a.D);
    for (int g = threadIdx.x; g < w.ng; g += blockDim.x) {
        float mu, m2;
        if (cs > 1) {
            float t = 0.f;
            for (int k = 0; k < cs; ++k)
                t = fmaf(static_cast<float>(gn_chunk_len(a.S, a.chunk_rows, k)), gn_peer(gs, g, k).x, t);
            mu = t / static_cast<float>(a.S);
            m2 = 0.f;
            for (int k = 0; k < cs; ++k) {
                const float2 e = gn_peer(gs, g, k);
                const float d = e.x - mu;
                m2 += fmaf(static_cast<float>(gn_chunk_len(a.S, a.chunk_rows, k)) * static_cast<float>(a.D) * d, d, e.y);
            }
        } else {
            mu = gs[g].x;
            m2 = gs[g].y;
        }
        const float rstd = rsqrtf(m2 / count + a.eps);
        fin[g] = make_float2(mu, rstd);
        if (rank == 0) {
            const int64_t at = w.b * a.G + w.g0 + g;
            if (a.mean) a.mean[at] = gn_elem(xs + int64_t(w.g0 + g) * a.D) + mu;
            if (a.rstd) a.rstd[at] = rstd;
        }
    }
    __syncthreads();
    if (cs > 1) cluster_arrive();  // this CTA has read its peers' states
    if (w.on) {
        GnOut<T, VEC, ACT> out;
        out.init(a, c, [&](int g) { return fin[g - w.g0]; }, [&](int) { return 0.f; });
#pragma unroll
        for (int i = 0; i < X::H; ++i) out.K[i] = K[i];
        T* yp = static_cast<T*>(a.y) + w.b * a.yb + (row0 + w.r) * a.yr + c;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < visits) X::store(yp + int64_t(v) * a.par * a.yr, out.apply(raw[v]));
    }
    if (cs > 1) cluster_wait();
}

// Rows a thread adds with one shift before it merges them into its running
// state: the shifted sum of squares then loses at most a few of fp32's bits
// even where that shift lies far from the other rows.
constexpr int kGnShiftRows = 128;

template <class T, int VEC, bool ONE>
__global__ void __launch_bounds__(kGnMaxThreads) gn_fwd_sums(const GnArgs a) {
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
    const int stride = ONE ? a.tile : a.tile * VEC;
    float2* st = sm;
    float2* gs = st + a.par * stride;

    const int64_t rows = gn_chunk_len(a.S, a.chunk_rows, k);
    const int c = w.c0 + w.col * VEC;
    const T* xs = static_cast<const T*>(a.x) + w.b * a.xb;
    const T* xp = xs + (k * a.chunk_rows + w.r) * a.xr + c;
    const int visits = w.on ? gn_visits(rows, w.r, a.par) : 0;
    const int64_t step = int64_t(a.par) * a.xr;

    float2 K[X::H], s[X::H], q[X::H];  // of the rows since the last merge
    float2 m[X::H], m2[X::H];          // merged: mean relative to the group's first element, M2
    float2 G0[X::H];
#pragma unroll
    for (int i = 0; i < X::H; ++i) {
        s[i] = q[i] = m[i] = m2[i] = K[i] = G0[i] = make_float2(0.f, 0.f);
        if (w.on) {
            if (ONE && i > 0)
                G0[i] = G0[0];
            else {
                G0[i].x = gn_elem(xs + int64_t((c + 2 * i) / a.D) * a.D);
                G0[i].y = VEC == 1 ? 0.f : ONE ? G0[i].x : gn_elem(xs + int64_t((c + 2 * i + 1) / a.D) * a.D);
            }
        }
    }
    int merged = 0;
    for (int v0 = 0; v0 < visits;) {
        const int stop = min(visits, v0 + kGnShiftRows);
        const int n = stop - v0;
        {
            const auto first = X::load(xp);
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                K[i] = X::get(first, i);
                s[i] = q[i] = make_float2(0.f, 0.f);
            }
        }
        for (; v0 < stop; v0 += U) {
            typename X::Raw raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + u < stop) raw[u] = X::load(xp + u * step);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + u < stop) {
#pragma unroll
                    for (int i = 0; i < X::H; ++i) {
                        const float2 d = f2_sub(X::get(raw[u], i), K[i]);
                        s[i] = __fadd2_rn(s[i], d);
                        q[i] = __ffma2_rn(d, d, q[i]);
                    }
                }
            xp += U * step;
        }
        v0 = stop;
        // merge: this block's mean relative to its own shift is s / n
        const float fn = static_cast<float>(n), inv = 1.f / fn;
        const float tot = static_cast<float>(merged + n);
        const float wb = fn / tot, wab = static_cast<float>(merged) * wb;
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            const float2 d = __fmul2_rn(s[i], f2_splat(inv));
            float2 b2 = make_float2(fmaf(-s[i].x, d.x, q[i].x), fmaf(-s[i].y, d.y, q[i].y));
            b2.x = b2.x < 0.f ? 0.f : b2.x;  // (a NaN stays one)
            b2.y = b2.y < 0.f ? 0.f : b2.y;
            const float2 mb = __fadd2_rn(f2_sub(K[i], G0[i]), d);
            const float2 e = f2_sub(mb, m[i]);
            m[i] = __ffma2_rn(e, f2_splat(wb), m[i]);
            m2[i] = __fadd2_rn(__ffma2_rn(__fmul2_rn(e, f2_splat(wab)), e, m2[i]), b2);
        }
        merged += n;
    }
    if (w.on) {
        if constexpr (ONE) {
            float t = 0.f, p = 0.f;
#pragma unroll
            for (int i = 0; i < X::H; ++i) t += f2_sum<VEC>(m[i]);
            const float mean = t * (1.f / VEC);
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                const float2 e = f2_sub(m[i], f2_splat(mean));
                p += f2_sum<VEC>(__ffma2_rn(__fmul2_rn(e, f2_splat(static_cast<float>(merged))), e, m2[i]));
            }
            st[w.r * stride + w.col] = make_float2(mean, p);
        } else {
#pragma unroll
            for (int i = 0; i < X::H; ++i) {
                st[w.r * stride + w.col * VEC + 2 * i] = make_float2(m[i].x, m2[i].x);
                st[w.r * stride + w.col * VEC + 2 * i + 1] = make_float2(m[i].y, m2[i].y);
            }
        }
    }
    __syncthreads();
    gn_merge_threads<ONE ? VEC : 1>(a, w, st, stride, rows, gs);
    if (cs > 1)
        cluster_barrier();
    else
        __syncthreads();
    // the cluster's chunks, groups shared out over its CTAs
    const int p0 = k / cs, parts = a.chunks / cs;
    for (int g = rank + cs * static_cast<int>(threadIdx.x); g < w.ng; g += cs * blockDim.x) {
        const int gg = w.g0 + g;
        float mu, p2;
        if (cs > 1) {
            float t = 0.f, n = 0.f;
            for (int j = 0; j < cs; ++j) {
                const float nj = static_cast<float>(gn_chunk_len(a.S, a.chunk_rows, int64_t(p0) * cs + j));
                t = fmaf(nj, gn_peer(gs, g, j).x, t);
                n += nj;
            }
            mu = n > 0.f ? t / n : 0.f;
            const float width = static_cast<float>(min((gg + 1) * a.D, w.c0 + w.nc) - max(gg * a.D, w.c0));
            p2 = 0.f;
            for (int j = 0; j < cs; ++j) {
                const float nj = static_cast<float>(gn_chunk_len(a.S, a.chunk_rows, int64_t(p0) * cs + j));
                if (nj > 0.f) {
                    const float2 e = gn_peer(gs, g, j);
                    const float d = e.x - mu;
                    p2 += fmaf(nj * width * d, d, e.y);
                }
            }
        } else {
            mu = gs[g].x;
            p2 = gs[g].y;
        }
        const int64_t bg = w.b * a.G + gg;
        const int ti = w.t - static_cast<int>((int64_t(gg) * a.D / VEC) / a.tile);
        a.part[(bg * a.tpg + ti) * parts + p0] = make_float2(mu, p2);
        if (p0 == 0 && ti == 0) a.shift[bg] = gn_elem(xs + int64_t(gg) * a.D);
    }
    if (cs > 1) cluster_barrier();  // no CTA leaves while a peer reads its states
}

template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnMaxThreads) gn_fwd_apply(const GnArgs a) {
    using X = GnVec<T, VEC>;
    constexpr int U = 4;
    extern __shared__ float2 sm[];
    grid_release();
    grid_wait();
    float2* fin = sm;                                   // (mu, rstd) per group of the tile
    float* shift = reinterpret_cast<float*>(sm + (a.tile * VEC - 1 + a.D - 1) / a.D + 1);
    // last chunks first: what the sums kernel read last is the likeliest in L2
    const int64_t id = int64_t(gridDim.x) - 1 - blockIdx.x;
    const int64_t unit = id / a.out_chunks;
    const int k = static_cast<int>(id - unit * a.out_chunks);
    const GnTile w = gn_tile<VEC>(a, unit);
    const int parts = a.chunks / a.cluster;
    const int64_t part_rows = a.chunk_rows * a.cluster;
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < w.ng; g += blockDim.x >> 5) {
        // every tile and merged chunk of the group, lanes side by side
        const int gg = w.g0 + g;
        const int64_t bg = w.b * a.G + gg;
        const int t0 = static_cast<int>((int64_t(gg) * a.D / VEC) / a.tile);
        const int t1 = static_cast<int>(((int64_t(gg) + 1) * a.D - 1) / VEC / a.tile);
        const int n = (t1 - t0 + 1) * parts;
        const float2* src = a.part + bg * a.tpg * parts;
        float s = 0.f;
        for (int i = lane; i < n; i += 32) {
            const int ti = i / parts, p = i - ti * parts;
            const int lo = max(gg * a.D, (t0 + ti) * a.tile * VEC);
            const int hi = min((gg + 1) * a.D, (t0 + ti + 1) * a.tile * VEC);
            s = fmaf(static_cast<float>(gn_chunk_len(a.S, part_rows, p)) * static_cast<float>(hi - lo), src[i].x, s);
        }
        const float count = static_cast<float>(a.S) * static_cast<float>(a.D);
        const float mu = group_sum(s, 32) / count;
        float q = 0.f;
        for (int i = lane; i < n; i += 32) {
            const int ti = i / parts, p = i - ti * parts;
            const int lo = max(gg * a.D, (t0 + ti) * a.tile * VEC);
            const int hi = min((gg + 1) * a.D, (t0 + ti + 1) * a.tile * VEC);
            const float2 e = src[i];
            const float d = e.x - mu;
            q += fmaf(static_cast<float>(gn_chunk_len(a.S, part_rows, p)) * static_cast<float>(hi - lo) * d, d, e.y);
        }
        q = group_sum(q, 32);
        if (lane == 0) {
            const float rstd = rsqrtf(q / count + a.eps);
            const float K = a.shift[bg];
            fin[g] = make_float2(mu, rstd);
            shift[g] = K;
            if (k == 0 && t0 == w.t) {
                if (a.mean) a.mean[bg] = K + mu;
                if (a.rstd) a.rstd[bg] = rstd;
            }
        }
    }
    __syncthreads();
    if (!w.on) return;
    const int64_t rows = gn_chunk_len(a.S, a.out_rows, k);
    const int visits = gn_visits(rows, w.r, a.par);
    const int c = w.c0 + w.col * VEC;
    GnOut<T, VEC, ACT> out;
    out.init(a, c, [&](int g) { return fin[g - w.g0]; }, [&](int g) { return shift[g - w.g0]; });
    const int64_t row = k * a.out_rows + w.r;
    const T* xp = static_cast<const T*>(a.x) + w.b * a.xb + row * a.xr + c;
    T* yp = static_cast<T*>(a.y) + w.b * a.yb + row * a.yr + c;
    const int64_t xstep = int64_t(a.par) * a.xr, ystep = int64_t(a.par) * a.yr;
    for (int v = 0; v < visits; v += U) {
        typename X::Raw raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u < visits) raw[u] = X::load(xp + u * xstep);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u < visits) X::store(yp + u * ystep, out.apply(raw[u]));
        xp += U * xstep;
        yp += U * ystep;
    }
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
    const size_t smem = static_cast<size_t>(gn_smem_bytes(a.par, ONE ? a.tile : channels, groups));
    if (p.path == GN_PATH_CHIP) {
        const GnKernel k = act == NORM_ACT_SILU   ? gn_pick_chip<T, VEC, ONE, NORM_ACT_SILU>(p.per_thread)
                           : act == NORM_ACT_GELU ? gn_pick_chip<T, VEC, ONE, NORM_ACT_GELU>(p.per_thread)
                                                  : gn_pick_chip<T, VEC, ONE, NORM_ACT_NONE>(p.per_thread);
        if (k == nullptr) return cudaErrorInvalidValue;
        return gn_launch(reinterpret_cast<const void*>(k), units * a.cluster, p.threads, smem, a.cluster, s, a);
    }
    const cudaError_t e = gn_launch(reinterpret_cast<const void*>(gn_fwd_sums<T, VEC, ONE>), units * a.chunks,
                                    p.threads, smem, a.cluster, s, a);
    if (e != cudaSuccess) return e;
    const GnKernel k = act == NORM_ACT_SILU   ? gn_fwd_apply<T, VEC, NORM_ACT_SILU>
                       : act == NORM_ACT_GELU ? gn_fwd_apply<T, VEC, NORM_ACT_GELU>
                                              : gn_fwd_apply<T, VEC, NORM_ACT_NONE>;
    return gn_launch(reinterpret_cast<const void*>(k), units * a.out_chunks, p.threads,
                     static_cast<size_t>(gn_smem_bytes(0, 0, groups)), 1, s, a);
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
