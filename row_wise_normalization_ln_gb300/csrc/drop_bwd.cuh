// Backward of dropout, residual add and norm (and of the plain fused add):
//   LayerNorm: xhat = (h - mean) rstd, g = dy gamma,
//              d = dh + rstd (g - mean(g) - xhat mean(g xhat))
//   RMSNorm:   d = dh + rstd dy w - h rstd^3 mean(dy w h), rstd from h
//   dresidual = d,  dx = d keep / P(keep),  dgamma = sum dy xhat,  dbeta = sum dy
// The R rows of a step are read from shared memory twice: for their sums, which
// meet behind one barrier, and for the outputs. Column sums stay in registers;
// after kDropChain rows they are added to the thread's own part of a partial
// row (in the workspace; in shared memory where the teams of a CTA have
// columns in common), so that no chain of additions is long.
#pragma once

#include "drop_kernels.cuh"

namespace libnorm {

template <class T, int VEC, int V, int R, bool LN, bool GROUP>
__global__ void __launch_bounds__(kDropMaxThreads) drop_bwd(const __grid_constant__ DropArgs a) {
    using P = DropPlace<VEC, V, GROUP>;
    using X = DropVec<T, VEC>;
    using Raw = typename X::Raw;
    constexpr int H = X::H, NA = LN ? 2 : 1;
    constexpr bool kElems = VEC == 1;
    extern __shared__ __align__(16) char smem[];
    __shared__ DropSums<2 * R> sums;
    const P pl(a);
    if (!GROUP) sums.clear();
    grid_release();
    grid_wait();
    const DropMask mask(a);
    const bool drop = a.limit != 0 && a.dx;
    const void* const from[3] = {a.hin, a.dy, a.dh};
    using Ring = std::conditional_t<kElems, DropStage<T, 3>, DropRing<T, VEC, V, R, 3, P>>;
    const int cta_col = kElems ? pl.rank * pl.warps * P::kRun : 0;
    const int cta_cols = kElems ? max(0, min(a.N - cta_col, pl.warps * P::kRun)) : 0;
    uint4* const words = reinterpret_cast<uint4*>(smem + a.words_at);
    const int words_row = kElems ? (pl.warps * P::kRun) / 8 + 2 : 0;
    float* const shared_cols = reinterpret_cast<float*>(smem + a.sums_at);
    Ring ring = [&] {
        if constexpr (kElems)
            return Ring(a, pl.block, pl.blocks_step, cta_col, cta_cols, smem, from);
        else
            return Ring(a, pl, smem, from);
    }();
    const auto row_words = [&](int64_t it) {
        const int64_t row = pl.block + it * pl.blocks_step;
        if (kElems && drop && row < a.M)
            drop_stage_words(mask, static_cast<uint64_t>(row) * a.N + cta_col, cta_cols, words + (it & 1) * words_row);
    };
    if constexpr (kElems) {
        for (int64_t i = 0; i < a.stages - 1; ++i) ring.send(i);
        row_words(0);
    }
    const int64_t step = pl.blocks_step * R * a.N;
    int64_t row = pl.block * R;
    int64_t at = row * a.N + pl.col;
    int64_t rows = a.M - row;
    uint64_t group = VEC > 1 ? static_cast<uint64_t>(at) / VEC : 0;
    float2 ms[R];  // mean and rstd, a step ahead
    const auto ahead = [&](int64_t first, int64_t left) {
        if constexpr (LN) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < left) ms[r] = make_float2(__ldg(a.mean + first + r), __ldg(a.rstd + first + r));
        }
    };
#pragma unroll
    for (int r = 0; r < R; ++r) ms[r] = make_float2(0.f, 0.f);
    ahead(row, rows);
    Raw gv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        gv[j] = X::zero();
        if (pl.on(j)) gv[j] = pl.load(static_cast<const T*>(a.gamma) + pl.col, j);
    }
    float2 acc[NA][V][H];
#pragma unroll
    for (int k = 0; k < NA; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) acc[k][j][i] = make_float2(0.f, 0.f);
    // Where the sums of chains go: this thread's columns of the CTA's (or
    // cluster's) partial row, or its slots of shared memory.
    float* const part = a.ws + static_cast<int64_t>(blockIdx.x / pl.C) * NA * a.N;
    bool begun = false;
    const auto fold = [&] {
#pragma unroll
        for (int k = 0; k < NA; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (pl.on(j)) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        float *x, *y;
                        if (GROUP) {
                            x = shared_cols + ((k * V + j) * VEC + 2 * i) * blockDim.x + threadIdx.x;
                            y = x + blockDim.x;
                        } else {
                            x = part + static_cast<int64_t>(k) * a.N + pl.col + pl.at(j) + 2 * i;
                            y = x + (kElems ? 32 : 1);
                        }
                        const float2 v = acc[k][j][i];
                        *x = begun ? *x + v.x : v.x;
                        if (!kElems || 2 * j + 1 < pl.nv) *y = begun ? *y + v.y : v.y;
                        acc[k][j][i] = make_float2(0.f, 0.f);
                    }
                }
        begun = true;
    };
    int chain = 0;
    const int64_t most = GROUP ? a.M - static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.lanes) * R : rows;
    const int64_t iters = most > 0 ? (most + pl.blocks_step * R - 1) / (pl.blocks_step * R) : 0;
    if constexpr (kElems) {
        if (a.stages == 3) copy_async_wait<1>();
        else copy_async_wait<2>();
        __syncthreads();
    }
    for (int64_t it = 0; it < iters; ++it) {
        const int parity = static_cast<int>(it & 1);
        if constexpr (!kElems) {
            ring.wait();
            ring.send(pl);  // into the slots read a step ago
        }
        // Access j of h, dy, dh of row r.
        const T* src[3] = {nullptr, nullptr, nullptr};
        if constexpr (kElems) {
#pragma unroll
            for (int n = 0; n < 3; ++n)
                if (from[n]) src[n] = ring.row(n, it) + (pl.col - cta_col);
        }
        const auto get = [&](int r, int n, int j) {
            if constexpr (kElems) return ring.get(pl, src[n], j);
            else return ring.get(r, n, j);
        };
        float s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 nmu = f2_splat(-ms[r].x), rs2 = f2_splat(ms[r].y);
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (r < rows && pl.on(j)) {
                    const Raw hr = get(r, 0, j), yr = get(r, 1, j);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float2 hv = X::get(hr, i);
                        const float2 g = __fmul2_rn(X::get(yr, i), X::get(gv[j], i));
                        if constexpr (LN) {
                            // (an element that is not there has g = 0)
                            s0 = __fadd2_rn(s0, g);
                            s1 = __ffma2_rn(g, __fmul2_rn(__fadd2_rn(hv, nmu), rs2), s1);
                        } else {
                            s0 = __ffma2_rn(hv, hv, s0);
                            s1 = __ffma2_rn(g, hv, s1);
                        }
                    }
                }
            s[2 * r] = s0.x + s0.y;
            s[2 * r + 1] = s1.x + s1.y;
        }
        float2 now[R];
#pragma unroll
        for (int r = 0; r < R; ++r) now[r] = ms[r];
        ahead(row + pl.blocks_step * R, rows - pl.blocks_step * R);
        if constexpr (kElems) {
            if (a.stages == 3) copy_async_wait<0>();
            else copy_async_wait<1>();  // the next row has landed; the barrier makes it everyone's
            if (pl.warps == 1) __syncthreads();
        }
        drop_sum<2 * R>(sums, pl, parity, s);
        if constexpr (kElems) {
            ring.send(it + a.stages - 1);  // into the slot whose row every thread is done with
            row_words(it + 1);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 nmu = f2_splat(-now[r].x), rs2 = f2_splat(now[r].y);
            // LayerNorm: mean(g), mean(g xhat); RMSNorm: rstd, rstd^3 mean(g h)
            float c0 = s[2 * r] * a.invN, c1 = s[2 * r + 1] * a.invN;
            if constexpr (!LN) {
                c0 = rsqrtf(fmaf(s[2 * r], a.invN, a.eps));
                c1 = c0 * c0 * c0 * c1;
            }
            const float2 n0 = f2_splat(-c0), n1 = f2_splat(-c1), p0 = f2_splat(c0), scale = f2_splat(a.scale);
            T* const rp = static_cast<T*>(a.dres) + at + r * a.N;
            T* const xp = static_cast<T*>(a.dx) + at + r * a.N;
            const unsigned short* ws = nullptr;
            if constexpr (kElems)
                ws = reinterpret_cast<const unsigned short*>(words + parity * words_row) + ((at - (pl.col - cta_col)) & 7) + (pl.col - cta_col);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (r < rows && pl.on(j)) {
                    const Raw hr = get(r, 0, j), yr = get(r, 1, j);
                    Raw er = X::zero(), orr = X::zero(), oxr = X::zero();
                    if (a.dh) er = get(r, 2, j);
                    DropWords<VEC> w;
                    if (drop) {
                        if constexpr (kElems) w.take(ws + pl.at(j));
                        else w.take(mask, group + r * (a.N / VEC) + pl.at(j) / VEC);
                    }
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
                            if (drop && !w.lo(mask, i)) dx.x = 0.f;
                            if (drop && !w.hi(mask, i)) dx.y = 0.f;
                            X::set(oxr, i, dx);
                        }
                    }
                    pl.store(rp, j, orr);
                    if (a.dx) pl.store(xp, j, oxr);
                }
        }
        if constexpr (!kElems) ring.advance();
        chain += R;
        if (chain >= kDropChain) {
            fold();
            chain = 0;
        }
        row += pl.blocks_step * R;
        at += step;
        if (VEC > 1) group += static_cast<uint64_t>(step) / VEC;
        rows -= pl.blocks_step * R;
    }
    fold();
    if (GROUP) {
        // the teams' sums of each column, in order
        __syncthreads();
        const int teams = blockDim.x / a.lanes;
        for (int i = threadIdx.x; i < NA * a.N; i += blockDim.x) {
            const int k = i / a.N, c = i - k * a.N, f = c / VEC, e = c - f * VEC;
            const int j = f / a.lanes, tl = f - j * a.lanes;
            const float* p = shared_cols + ((k * V + j) * VEC + e) * blockDim.x + tl;
            float t = 0.f;
            for (int u = 0; u < teams; ++u) t += p[u * a.lanes];
            part[i] = t;
        }
    }
    if (pl.C > 1) cluster_barrier();  // no CTA leaves while a peer may read its sums
}

template <class T, int VEC, int V, int R, bool LN, bool GROUP>
cudaError_t drop_launch_bwd(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    const void* fn = reinterpret_cast<const void*>(drop_bwd<T, VEC, V, R, LN, GROUP>);
    a.pitch = static_cast<int32_t>(VEC == 1 ? drop_pitch(sizeof(T), V, p.threads) : 0);
    a.words_at = static_cast<int32_t>(drop_ring_bytes(VEC, sizeof(T), V, p.threads, R, a.stages, 3));
    a.sums_at = static_cast<int32_t>(a.words_at + drop_words_bytes(VEC, V, p.threads));
    const size_t smem = static_cast<size_t>(a.sums_at + (GROUP ? drop_sums_bytes(LN, VEC, V, p.threads) : 0));
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
    const int V = p.per_thread, R = p.rounds;
    if (p.vec_elems == 1) {
        if (V == 2) return drop_launch_bwd<T, 1, 2, 1, LN, false>(p, a, s);
        return drop_launch_bwd<T, 1, 8, 1, LN, false>(p, a, s);
    }
    if (p.mapping == NORM_MAP_GROUP) {
        if (V == 1) return drop_launch_bwd<T, full, 1, 4, LN, true>(p, a, s);
        return drop_launch_bwd<T, full, 2, 2, LN, true>(p, a, s);
    }
    if (V == 1) return R == 1 ? drop_launch_bwd<T, full, 1, 1, LN, false>(p, a, s) : drop_launch_bwd<T, full, 1, 4, LN, false>(p, a, s);
    if constexpr (sizeof(T) == 4)
        return R == 1 ? drop_launch_bwd<T, full, 4, 1, LN, false>(p, a, s) : drop_launch_bwd<T, full, 4, 2, LN, false>(p, a, s);
    else
        return drop_launch_bwd<T, full, 2, 2, LN, false>(p, a, s);
}

template <class T>
cudaError_t drop_dispatch_bwd(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return ln ? drop_bwd_of<T, true>(p, a, s) : drop_bwd_of<T, false>(p, a, s);
}

}  // namespace libnorm
