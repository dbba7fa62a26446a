// Dropout, residual add and norm, forward:
//   h = residual + x keep / P(keep)  (rounded to the row's type),  y = norm(h).
//
// A thread holds its values of R rows as fp32 pairs from the add to the
// output. LayerNorm: a warp's values are shifted by its first one, K (a mean
// that dwarfs the spread costs no digits), its mean and M2 formed in two
// passes over the registers, and the warps' states (n, K + mean, M2) meet
// behind one barrier by the merge rule in its k-way form, the means as
// differences from the first warp's K:
//   m_w = (K_w - K_0) + mean_w,  mean = sum n_w m_w / N,  M2 = sum M2_w + n_w (m_w - mean)^2.
// RMSNorm: sums of squares.
#pragma once

#include "drop_kernels.cuh"

namespace libnorm {

// The states of a CTA's warps (and of a cluster's CTAs) of R rows.
template <int R>
struct DropStates {
    float K[2][R][kDropMaxThreads / 32], mean[2][R][kDropMaxThreads / 32], m2[2][R][kDropMaxThreads / 32];
    float cta[2][3][R];
    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < 3 * 2 * R * (kDropMaxThreads / 32); i += blockDim.x) (&K[0][0][0])[i] = 0.f;
        __syncthreads();
    }
};

template <int N>
__device__ __forceinline__ float drop_down(float v) {  // sum over aligned blocks of N lanes
#pragma unroll
    for (int off = N / 2; off > 0; off /= 2) v += __shfl_xor_sync(kFullMask, v, off);
    return v;
}

template <class T, int VEC, int V, int R, bool LN, bool GROUP>
__global__ void __launch_bounds__(kDropMaxThreads) drop_fwd(const __grid_constant__ DropArgs a) {
    using P = DropPlace<VEC, V, GROUP>;
    using X = DropVec<T, VEC>;
    using Raw = typename X::Raw;
    constexpr int H = X::H;
    constexpr bool kElems = VEC == 1;
    extern __shared__ __align__(16) char smem[];
    __shared__ std::conditional_t<LN, DropStates<R>, DropSums<R>> sums;
    const P pl(a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!GROUP) sums.clear();
    grid_release();
    grid_wait();
    const DropMask mask(a);
    const bool drop = a.limit != 0;
    const void* const from[2] = {a.x, a.residual};
    using Ring = std::conditional_t<kElems, DropStage<T, 2>, DropRing<T, VEC, V, R, 2, P>>;
    // Elements: the CTA's part of a row.
    const int cta_col = kElems ? pl.rank * pl.warps * P::kRun : 0;
    const int cta_cols = kElems ? max(0, min(a.N - cta_col, pl.warps * P::kRun)) : 0;
    uint4* const words = reinterpret_cast<uint4*>(smem + a.words_at);
    const int words_row = kElems ? (pl.warps * P::kRun) / 8 + 2 : 0;
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
    Raw gv[V], bv[LN ? V : 1];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        gv[j] = X::zero();
        if (pl.on(j)) gv[j] = pl.load(static_cast<const T*>(a.gamma) + pl.col, j);
        if constexpr (LN) {
            bv[j] = X::zero();
            if (pl.on(j)) bv[j] = pl.load(static_cast<const T*>(a.beta) + pl.col, j);
        }
    }
    // LayerNorm: elements of this warp's part, of the warps whose states this
    // lane merges, of the CTA's.
    const DropShare<R> sh;
    constexpr int E = DropShare<R>::kEach, L = DropShare<R>::kLanes;
    float n_warp = 0.f, n_of[E], n_cta = 0.f;
    if constexpr (LN) {
        n_warp = GROUP ? static_cast<float>(a.N) : P::count(a, pl.rank, warp);
#pragma unroll
        for (int i = 0; i < E; ++i) n_of[i] = !GROUP && sh.w0 + i < pl.warps ? P::count(a, pl.rank, sh.w0 + i) : 0.f;
        if (!GROUP) n_cta = P::count_cta(a, pl.rank);
    }
    const float inv_warp = n_warp > 0.f ? 1.f / n_warp : 0.f, inv_cta = n_cta > 0.f ? 1.f / n_cta : 0.f;

    const int64_t step = pl.blocks_step * R * a.N;
    int64_t at = pl.block * R * a.N + pl.col;  // the thread's first element of the block's first row
    int64_t rows = a.M - pl.block * R;         // from there to the end
    uint64_t group = VEC > 1 ? static_cast<uint64_t>(at) / VEC : 0;
    // The teams of a CTA, and of a warp, take the same number of steps.
    const int64_t most = GROUP ? a.M - static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.lanes) * R : rows;
    const int64_t iters = most > 0 ? (most + pl.blocks_step * R - 1) / (pl.blocks_step * R) : 0;
    if constexpr (kElems) {
        if (a.stages == 3) copy_async_wait<1>();
        else copy_async_wait<2>();
        __syncthreads();
    }
    for (int64_t it = 0; it < iters; ++it) {
        const int parity = static_cast<int>(it & 1);
        float2 d[R][V][H];
        float s[R];
        if constexpr (!kElems) {
            ring.wait();
            ring.send(pl);  // into the slots read a block ago
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool on = r < rows;
            T* const hp = static_cast<T*>(a.h) + at + r * a.N;
            const T *xs = nullptr, *rs = nullptr;
            const unsigned short* ws = nullptr;
            if constexpr (kElems) {
                xs = ring.row(0, it) + (pl.col - cta_col);
                rs = ring.row(1, it) + (pl.col - cta_col);
                ws = reinterpret_cast<const unsigned short*>(words + parity * words_row) + ((at - (pl.col - cta_col)) & 7) + (pl.col - cta_col);
            }
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int i = 0; i < H; ++i) d[r][j][i] = make_float2(0.f, 0.f);
                if (on && pl.on(j)) {
                    Raw xr, rr, hr = X::zero();
                    if constexpr (kElems) {
                        xr = ring.get(pl, xs, j);
                        rr = ring.get(pl, rs, j);
                    } else {
                        xr = ring.get(r, 0, j);
                        rr = ring.get(r, 1, j);
                    }
                    DropWords<VEC> w;
                    if (drop) {
                        if constexpr (kElems) w.take(ws + pl.at(j));
                        else w.take(mask, group + r * (a.N / VEC) + pl.at(j) / VEC);
                    }
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float2 xv = X::get(xr, i);
                        float2 hv = X::get(rr, i);
                        if (!drop || w.lo(mask, i)) hv.x = fmaf(xv.x, a.scale, hv.x);
                        if (!drop || w.hi(mask, i)) hv.y = fmaf(xv.y, a.scale, hv.y);
                        X::set(hr, i, hv);
                    }
                    pl.store(hp, j, hr);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        d[r][j][i] = X::get(hr, i);
                        if (!LN) sum = __ffma2_rn(d[r][j][i], d[r][j][i], sum);
                    }
                }
            }
            if (!LN) s[r] = sum.x + sum.y;
        }
        if constexpr (!kElems) ring.advance();
        if constexpr (kElems) {
            ring.send(it + a.stages - 1);  // into the slot read before the last barrier
            row_words(it + 1);
            if (a.stages == 3) copy_async_wait<1>();
            else copy_async_wait<2>();     // the next row has landed; the barrier below makes it everyone's
        }
        float rstd[R], mu[R];
        if constexpr (LN) {
            float K[R], K0[R], mean[R], q[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                K[r] = __shfl_sync(kFullMask, d[r][0][0].x, GROUP ? lane & ~(pl.unit - 1) : 0);
                const float2 k2 = f2_splat(-K[r]);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (pl.on(j)) {
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            d[r][j][i] = __fadd2_rn(d[r][j][i], k2);
                            if (kElems && 2 * j + 1 >= pl.nv) d[r][j][i].y = 0.f;
                            sum = __fadd2_rn(sum, d[r][j][i]);
                        }
                    }
                s[r] = sum.x + sum.y;
            }
            if (GROUP) {
#pragma unroll
                for (int r = 0; r < R; ++r) mean[r] = group_sum(s[r], pl.unit) * inv_warp;
            } else {
                const float t = warp_sums<R>(s);
#pragma unroll
                for (int r = 0; r < R; ++r) mean[r] = __shfl_sync(kFullMask, t, R == 1 ? 0 : r * (32 / R)) * inv_warp;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 nm = f2_splat(-mean[r]);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (pl.on(j)) {
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            float2 e = __fadd2_rn(d[r][j][i], nm);
                            if (kElems && 2 * j + 1 >= pl.nv) e.y = 0.f;
                            sum = __ffma2_rn(e, e, sum);
                        }
                    }
                q[r] = sum.x + sum.y;
                K0[r] = K[r];
            }
            if (GROUP) {
#pragma unroll
                for (int r = 0; r < R; ++r) q[r] = group_sum(q[r], pl.unit);
            } else {
                float m2 = warp_sums<R>(q);  // of row lane / (32 / R)
                float m = mean[0], k = K[0];
#pragma unroll
                for (int r = 1; r < R; ++r)
                    if (lane / (32 / R) == r) m = mean[r], k = K[r];
                if (pl.warps > 1) {
                    if ((lane & (32 / R - 1)) == 0) {
                        const int r = lane / (32 / R);
                        sums.K[parity][r][warp] = k;
                        sums.mean[parity][r][warp] = m;
                        sums.m2[parity][r][warp] = m2;
                    }
                    __syncthreads();
                    k = sums.K[parity][sh.idx][0];
                    float t = 0.f, dm[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        dm[i] = (sums.K[parity][sh.idx][sh.w0 + i] - k) + sums.mean[parity][sh.idx][sh.w0 + i];
                        if (n_of[i] > 0.f) t = fmaf(n_of[i], dm[i], t);
                    }
                    m = drop_down<L>(t) * inv_cta;
                    t = 0.f;
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (n_of[i] > 0.f) t += fmaf(n_of[i] * (dm[i] - m), dm[i] - m, sums.m2[parity][sh.idx][sh.w0 + i]);
                    m2 = drop_down<L>(t);
                } else if (kElems) {
                    __syncthreads();
                }
                constexpr int S = R == 1 ? 0 : 32 / R;
                if (pl.C > 1) {
                    if (warp == 0 && (lane & (32 / R - 1)) == 0) {
                        sums.cta[parity][0][lane / (32 / R)] = k;
                        sums.cta[parity][1][lane / (32 / R)] = m;
                        sums.cta[parity][2][lane / (32 / R)] = m2;
                    }
                    cluster_barrier();
                    const float n = lane < pl.C ? P::count_cta(a, lane) : 0.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float pk = 0.f, pm = 0.f, pq = 0.f;
                        if (n > 0.f) {
                            pk = drop_peer(&sums.cta[parity][0][r], static_cast<uint32_t>(lane));
                            pm = drop_peer(&sums.cta[parity][1][r], static_cast<uint32_t>(lane));
                            pq = drop_peer(&sums.cta[parity][2][r], static_cast<uint32_t>(lane));
                        }
                        K0[r] = __shfl_sync(kFullMask, pk, 0);
                        const float dm = n > 0.f ? (pk - K0[r]) + pm : 0.f;
                        mean[r] = __shfl_sync(kFullMask, drop_down<8>(n * dm), 0) * a.invN;
                        q[r] = __shfl_sync(kFullMask, drop_down<8>(fmaf(n * (dm - mean[r]), dm - mean[r], pq)), 0);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        mean[r] = __shfl_sync(kFullMask, m, r * S);
                        q[r] = __shfl_sync(kFullMask, m2, r * S);
                        K0[r] = __shfl_sync(kFullMask, k, r * S);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                rstd[r] = rsqrtf(fmaf(q[r], a.invN, a.eps));
                mu[r] = mean[r] - (K[r] - K0[r]);  // from this warp's K
                if (r < rows && pl.first) {
                    const int64_t row = pl.block * R + it * pl.blocks_step * R + r;
                    if (a.mean) a.mean[row] = K0[r] + mean[r];
                    if (a.rstd) a.rstd[row] = rstd[r];
                }
            }
        } else {
            if (kElems && pl.warps == 1) __syncthreads();
            drop_sum<R>(sums, pl, parity, s);
#pragma unroll
            for (int r = 0; r < R; ++r) rstd[r] = rsqrtf(fmaf(s[r], a.invN, a.eps));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 rs2 = f2_splat(rstd[r]), nmr = f2_splat(LN ? -mu[r] * rstd[r] : 0.f);
            T* const yp = static_cast<T*>(a.y) + at + r * a.N;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (r < rows && pl.on(j)) {
                    Raw yr = X::zero();
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        if constexpr (LN)
                            X::set(yr, i, __ffma2_rn(__ffma2_rn(d[r][j][i], rs2, nmr), X::get(gv[j], i), X::get(bv[j], i)));
                        else
                            X::set(yr, i, __fmul2_rn(__fmul2_rn(d[r][j][i], X::get(gv[j], i)), rs2));
                    }
                    pl.store(yp, j, yr);
                }
        }
        at += step;
        if (VEC > 1) group += static_cast<uint64_t>(step) / VEC;
        rows -= pl.blocks_step * R;
    }
    if (pl.C > 1) cluster_barrier();  // no CTA leaves while a peer may read its state
}

template <class T, int VEC, int V, int R, bool LN, bool GROUP>
cudaError_t drop_launch_fwd(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    const void* fn = reinterpret_cast<const void*>(drop_fwd<T, VEC, V, R, LN, GROUP>);
    a.pitch = static_cast<int32_t>(VEC == 1 ? drop_pitch(sizeof(T), V, p.threads) : 0);
    a.words_at = static_cast<int32_t>(drop_ring_bytes(VEC, sizeof(T), V, p.threads, R, a.stages, 2));
    const size_t smem = static_cast<size_t>(a.words_at + drop_words_bytes(VEC, V, p.threads));
    int64_t most = 0;
    const cudaError_t e = drop_resident(fn, p.threads, smem, p.cluster, &most);
    if (e != cudaSuccess) return e;
    return drop_launch(fn, std::min(p.grid, most), p.threads, smem, p.cluster, s, a);
}

template <class T, bool LN>
cudaError_t drop_fwd_of(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    const int V = p.per_thread, R = p.rounds;
    if (p.vec_elems == 1) {
        if (V == 2) return drop_launch_fwd<T, 1, 2, 1, LN, false>(p, a, s);
        return drop_launch_fwd<T, 1, 8, 1, LN, false>(p, a, s);
    }
    if (p.mapping == NORM_MAP_GROUP) {
        if (V == 1) return drop_launch_fwd<T, full, 1, 4, LN, true>(p, a, s);
        return drop_launch_fwd<T, full, 2, 2, LN, true>(p, a, s);
    }
    if (V == 1) return R == 1 ? drop_launch_fwd<T, full, 1, 1, LN, false>(p, a, s) : drop_launch_fwd<T, full, 1, 4, LN, false>(p, a, s);
    if constexpr (sizeof(T) == 4)
        return R == 1 ? drop_launch_fwd<T, full, 4, 1, LN, false>(p, a, s) : drop_launch_fwd<T, full, 4, 2, LN, false>(p, a, s);
    else
        return V == 2 ? drop_launch_fwd<T, full, 2, 2, LN, false>(p, a, s) : drop_launch_fwd<T, full, 4, 1, LN, false>(p, a, s);
}

template <class T>
cudaError_t drop_dispatch_fwd(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return ln ? drop_fwd_of<T, true>(p, a, s) : drop_fwd_of<T, false>(p, a, s);
}

}  // namespace libnorm
