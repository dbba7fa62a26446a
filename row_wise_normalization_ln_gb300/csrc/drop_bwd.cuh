// Backward of dropout, residual add and norm (and of the plain fused add):
//   LayerNorm: xhat = (h - mean) rstd, g = dy gamma,
//              d = dh + rstd (g - mean(g) - xhat mean(g xhat))
//   RMSNorm:   d = dh + rstd dy w - h rstd^3 mean(dy w h), rstd from h
//   dresidual = d,  dx = d keep / P(keep),  dgamma = sum dy xhat,  dbeta = sum dy
// A row's dy, dh and h are read from the ring twice: for the two sums, and
// for the outputs. Column sums stay in registers; after kDropChain rows they
// are added to the thread's own part of a partial row (in the workspace; in
// shared memory where the teams of a CTA have columns in common), so that no
// chain of additions is long.
#pragma once

#include "drop_kernels.cuh"
#include "norm_bwd.cuh"

namespace libnorm {

template <class T, int VEC, int V, bool LN>
__global__ void __launch_bounds__(kDropMaxThreads) drop_bwd(const __grid_constant__ DropArgs a) {
    using X = GnVec<T, VEC>;
    using Raw = typename X::Raw;
    constexpr int H = X::H, NA = LN ? 2 : 1;
    extern __shared__ __align__(16) char smem[];
    __shared__ DropSums sums;
    DropPlace pl;
    pl.set<VEC, V>(a);
    grid_release();
    grid_wait();
    const void* const from[3] = {a.hin, a.dy, a.dh};
    using Ring = DropRing<T, VEC, V, 3>;
    Ring ring(a, pl, smem, from);
    uint4* words = reinterpret_cast<uint4*>(smem + a.words_at);
    float* shared_cols = reinterpret_cast<float*>(smem + a.sums_at);
    const DropMask mask(a);
    const bool drop = a.limit != 0;
    float2 ms = make_float2(0.f, 0.f);  // mean and rstd, a row ahead
    const auto ahead = [&](int64_t row) {
        if (LN && row < a.M) ms = make_float2(__ldg(a.mean + row), __ldg(a.rstd + row));
    };
    ahead(pl.row);
    Raw gv[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < pl.nv) gv[j] = X::load(static_cast<const T*>(a.gamma) + (pl.f0 + j * pl.step) * VEC);
    float2 acc[NA][V][H];
#pragma unroll
    for (int k = 0; k < NA; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) acc[k][j][i] = make_float2(0.f, 0.f);
    // Where the sums of chains go: this thread's columns of the CTA's (or
    // cluster's) partial row, or its slots of shared memory.
    float* part = a.ws + static_cast<int64_t>(blockIdx.x / pl.C) * NA * a.N;
    bool begun = false;
    const auto fold = [&] {
#pragma unroll
        for (int k = 0; k < NA; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < pl.nv) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        float* to = a.lanes > 0 ? shared_cols + ((k * V + j) * VEC + 2 * i) * blockDim.x + threadIdx.x
                                                : part + static_cast<int64_t>(k) * a.N + (pl.f0 + j * pl.step) * VEC + 2 * i;
                        const int next = a.lanes > 0 ? blockDim.x : 1;
                        to[0] = begun ? to[0] + acc[k][j][i].x : acc[k][j][i].x;
                        if (VEC > 1) to[next] = begun ? to[next] + acc[k][j][i].y : acc[k][j][i].y;
                        acc[k][j][i] = make_float2(0.f, 0.f);
                    }
                }
        begun = true;
    };
    int chain = 0;
    for (int64_t it = 0; it < pl.iters; ++it) {
        const int parity = static_cast<int>(it & 1);
        const int64_t row = pl.row + it * pl.rows_step;
        const bool on = row < a.M;
        const float2 nmu = f2_splat(-ms.x), rs2 = f2_splat(ms.y);
        DropRowMask<T, VEC, V> keep(mask, drop && a.dx, a, pl, row, words);
        ring.wait();
        if constexpr (Ring::kAsync) ring.send();  // into the slot read a row ago
        float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (on && j < pl.nv) {
                const Raw hr = ring.get(0, j), yr = ring.get(1, j);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 hv = X::get(hr, i);
                    const float2 g = __fmul2_rn(X::get(yr, i), X::get(gv[j], i));
                    if constexpr (LN) {
                        const float2 xh = __fmul2_rn(__fadd2_rn(hv, nmu), rs2);
                        s0 = __fadd2_rn(s0, g);
                        s1 = __ffma2_rn(g, xh, s1);
                    } else {
                        s0 = __ffma2_rn(hv, hv, s0);
                        s1 = __ffma2_rn(g, hv, s1);
                    }
                }
            }
        ahead(row + pl.rows_step);
        const float2 S = drop_sum(sums, pl, parity, make_float2(f2_sum<VEC>(s0), f2_sum<VEC>(s1)));
        // LayerNorm: mean(g), mean(g xhat); RMSNorm: rstd, rstd^3 mean(g h)
        float c0 = S.x * a.invN, c1 = S.y * a.invN;
        if constexpr (!LN) {
            c0 = rsqrtf(fmaf(S.x, a.invN, a.eps));
            c1 = c0 * c0 * c0 * c1;
        }
        const float2 n0 = f2_splat(-c0), n1 = f2_splat(-c1), p0 = f2_splat(c0);
        const int64_t at = row * a.N + static_cast<int64_t>(pl.f0) * VEC;
        const float2 scale = f2_splat(a.scale);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (on && j < pl.nv) {
                const Raw hr = ring.get(0, j), yr = ring.get(1, j);
                const Raw er = a.dh ? ring.get(2, j) : X::zero();
                Raw orr = X::zero(), oxr = X::zero();
                keep.access(j);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 hv = X::get(hr, i), yv = X::get(yr, i);
                    const float2 g = __fmul2_rn(yv, X::get(gv[j], i));
                    float2 d;
                    if constexpr (LN) {
                        const float2 xh = __fmul2_rn(__fadd2_rn(hv, nmu), rs2);
                        d = __ffma2_rn(rs2, __ffma2_rn(xh, n1, __fadd2_rn(g, n0)), X::get(er, i));
                        acc[0][j][i] = __ffma2_rn(yv, xh, acc[0][j][i]);
                        acc[NA - 1][j][i] = __fadd2_rn(acc[NA - 1][j][i], yv);
                    } else {
                        d = __ffma2_rn(hv, n1, __ffma2_rn(g, p0, X::get(er, i)));
                        acc[0][j][i] = __ffma2_rn(__fmul2_rn(yv, hv), p0, acc[0][j][i]);
                    }
                    X::set(orr, i, d);
                    if (a.dx) {
                        float2 dx = __fmul2_rn(d, scale);
                        if (!keep.lo(i)) dx.x = 0.f;
                        if (VEC > 1 && !keep.hi(i)) dx.y = 0.f;
                        X::set(oxr, i, dx);
                    }
                }
                X::store(static_cast<T*>(a.dres) + at + j * pl.step * VEC, orr);
                if (a.dx) X::store(static_cast<T*>(a.dx) + at + j * pl.step * VEC, oxr);
            }
        ring.advance();
        if constexpr (!Ring::kAsync) ring.send();
        if (++chain == kDropChain) {
            fold();
            chain = 0;
        }
    }
    fold();
    if (a.lanes > 0) {
        // the teams' sums of each column, in order
        __syncthreads();
        const int teams = blockDim.x / a.lanes;
        for (int i = threadIdx.x; i < NA * a.N; i += blockDim.x) {
            const int k = i / a.N, c = i - k * a.N, f = c / VEC, e = c - f * VEC;
            const int j = f / a.lanes, tl = f - j * a.lanes;
            const float* src = shared_cols + ((k * V + j) * VEC + e) * blockDim.x + tl;
            float t = 0.f;
            for (int u = 0; u < teams; ++u) t += src[u * a.lanes];
            part[i] = t;
        }
    }
    if (pl.C > 1) cluster_barrier();  // no CTA leaves while a peer may read its sums
}

template <class T, int VEC, int V, bool LN>
cudaError_t drop_launch_bwd(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    const void* fn = reinterpret_cast<const void*>(drop_bwd<T, VEC, V, LN>);
    a.words_at = static_cast<int32_t>(drop_ring_bytes(VEC, sizeof(T), V, p.threads, a.stages, 3));
    a.sums_at = static_cast<int32_t>(a.words_at + drop_mask_bytes(VEC, V, p.threads, a.lanes));
    const size_t smem = static_cast<size_t>(a.sums_at + (a.lanes > 0 ? drop_sums_bytes(LN, VEC, V, p.threads) : 0));
    int64_t grid = 0;
    if (a.M > 0) {
        int64_t most = 0;
        cudaError_t e = drop_resident(fn, p.threads, smem, p.cluster, &most);
        if (e != cudaSuccess) return e;
        grid = std::min(p.grid, most);
        e = drop_launch(fn, grid, p.threads, smem, p.cluster, s, a);
        if (e != cudaSuccess) return e;
    }
    return launch_drop_colsum(a, grid / p.cluster, LN, s);
}

template <class T, bool LN>
cudaError_t drop_bwd_of(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    if (p.vec_elems == full) {
        switch (p.per_thread) {
            case 1: return drop_launch_bwd<T, full, 1, LN>(p, a, s);
            case 2: return drop_launch_bwd<T, full, 2, LN>(p, a, s);
            case 4:
                if constexpr (sizeof(T) == 4) return drop_launch_bwd<T, full, 4, LN>(p, a, s);
        }
    } else if (p.vec_elems == 1) {
        switch (p.per_thread) {
            case 4: return drop_launch_bwd<T, 1, 4, LN>(p, a, s);
            case 16: return drop_launch_bwd<T, 1, 16, LN>(p, a, s);
        }
    }
    return cudaErrorInvalidValue;
}

template <class T>
cudaError_t drop_dispatch_bwd(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return ln ? drop_bwd_of<T, true>(p, a, s) : drop_bwd_of<T, false>(p, a, s);
}

}  // namespace libnorm
