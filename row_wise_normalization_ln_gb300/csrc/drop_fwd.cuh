// Dropout, residual add and norm, forward:
//   h = residual + x keep / P(keep)  (rounded to the row's type),  y = norm(h).
//
// A thread holds its values of the row as fp32 pairs from the add to the
// output (LayerNorm: less K, the row's first residual + x, so that a mean that
// dwarfs the spread costs no digits). LayerNorm: each warp forms the state
// (n, sum, M2) of its part in two passes over the registers, and the states
// meet in one barrier (drop_merge); RMSNorm: sums of squares.
#pragma once

#include "drop_kernels.cuh"

namespace libnorm {

template <class T, int VEC, int V, bool LN>
__global__ void __launch_bounds__(kDropMaxThreads) drop_fwd(const __grid_constant__ DropArgs a) {
    using X = GnVec<T, VEC>;
    using Raw = typename X::Raw;
    constexpr int H = X::H;
    extern __shared__ __align__(16) char smem[];
    __shared__ DropSums sums;
    DropPlace pl;
    pl.set<VEC, V>(a);
    grid_release();
    grid_wait();
    const void* const from[2] = {a.x, a.residual};
    using Ring = DropRing<T, VEC, V, 2>;
    Ring ring(a, pl, smem, from);
    uint4* words = reinterpret_cast<uint4*>(smem + a.words_at);
    const DropMask mask(a);
    const bool drop = a.limit != 0;
    // rows' first values, a row ahead: K
    float kx = 0.f, kr = 0.f;
    const auto ahead = [&](int64_t row) {
        if (LN && row < a.M) {
            kx = gn_elem(static_cast<const T*>(a.x) + row * a.N);
            kr = gn_elem(static_cast<const T*>(a.residual) + row * a.N);
        }
    };
    ahead(pl.row);
    Raw gv[V], bv[LN ? V : 1];
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < pl.nv) {
            const int c = (pl.f0 + j * pl.step) * VEC;
            gv[j] = X::load(static_cast<const T*>(a.gamma) + c);
            if constexpr (LN) bv[j] = X::load(static_cast<const T*>(a.beta) + c);
        }
    // elements of this warp (of the row, where lanes share it), for its state
    const int nacc = (a.N + VEC - 1) / VEC;
    const auto count = [&](int warp) {  // of a warp of this CTA
        const int at = (pl.rank * static_cast<int>(blockDim.x) + warp * 32) * V;
        return static_cast<float>(max(0, min(nacc - at, 32 * V)) * VEC);
    };
    const float n_unit = a.lanes > 0 ? static_cast<float>(a.N) : count(threadIdx.x >> 5);
    const float inv_unit = n_unit > 0.f ? 1.f / n_unit : 0.f;
    const int lane = threadIdx.x & 31, ww = drop_pow2(pl.warps);
    const float n_lane = lane < pl.warps ? count(lane) : 0.f;
    const int slice = V * static_cast<int>(blockDim.x);
    const auto count_cta = [&](int rank) { return static_cast<float>(max(0, min(nacc - rank * slice, slice)) * VEC); };
    const float n_cta = count_cta(pl.rank), n_peer = lane < pl.C ? count_cta(lane) : 0.f;
    const float inv_cta = n_cta > 0.f ? 1.f / n_cta : 0.f;

    // The first row's K has been read by every thread that needs it before
    // any h is written (which may be where it came from); later rows' is, a
    // row ahead, before a barrier.
    if (pl.C > 1) cluster_barrier();
    else __syncthreads();
    for (int64_t it = 0; it < pl.iters; ++it) {
        const int parity = static_cast<int>(it & 1);
        const int64_t row = pl.row + it * pl.rows_step;
        const bool on = row < a.M;
        float K = kx + kr;
        if (!isfinite(K)) K = 0.f;  // (of a value that may be dropped, or spoils the row anyway)
        const float2 k2 = f2_splat(-K);
        float2 d[V][H];
        float2 s2 = make_float2(0.f, 0.f);
        DropRowMask<T, VEC, V> keep(mask, drop, a, pl, row, words);
        ring.wait();
        if constexpr (Ring::kAsync) ring.send();  // into the slot read a row ago
        T* hp = static_cast<T*>(a.h) + row * a.N + static_cast<int64_t>(pl.f0) * VEC;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (on && j < pl.nv) {
                const Raw xr = ring.get(0, j), rr = ring.get(1, j);
                keep.access(j);
                Raw hr = X::zero();
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 xv = X::get(xr, i);
                    float2 hv = X::get(rr, i);
                    if (keep.lo(i)) hv.x = fmaf(xv.x, a.scale, hv.x);
                    if (keep.hi(i)) hv.y = fmaf(xv.y, a.scale, hv.y);
                    X::set(hr, i, hv);
                }
                X::store(hp + j * pl.step * VEC, hr);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 hv = X::get(hr, i);
                    if constexpr (LN) {
                        d[j][i] = __fadd2_rn(hv, k2);
                        if (VEC == 1) d[j][i].y = 0.f;
                        s2 = __fadd2_rn(s2, d[j][i]);
                    } else {
                        d[j][i] = hv;
                        s2 = __ffma2_rn(hv, hv, s2);
                    }
                }
            }
        ring.advance();
        if constexpr (!Ring::kAsync) ring.send();
        ahead(row + pl.rows_step);
        float mu = 0.f, rs;
        if constexpr (LN) {
            // this warp's state
            float2 st;
            st.x = group_sum(s2.x + s2.y, pl.unit);
            const float2 nm = f2_splat(-(st.x * inv_unit));
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (on && j < pl.nv) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        float2 e = __fadd2_rn(d[j][i], nm);
                        if (VEC == 1) e.y = 0.f;
                        q = __ffma2_rn(e, e, q);
                    }
                }
            st.y = group_sum(q.x + q.y, pl.unit);
            if (pl.warps > 1) {
                if (lane == 0) sums.warp[parity][threadIdx.x >> 5] = st;
                __syncthreads();
                st = drop_merge(n_lane, lane < pl.warps ? sums.warp[parity][lane] : make_float2(0.f, 0.f), inv_cta, ww);
            }
            if (pl.C > 1) {
                if (pl.warps == 1) __syncwarp();
                if (threadIdx.x == 0) sums.cta[parity] = st;
                cluster_barrier();
                st = drop_merge(n_peer, lane < pl.C ? drop_peer(&sums.cta[parity], static_cast<uint32_t>(lane)) : make_float2(0.f, 0.f),
                                a.invN, 8);
            }
            if (pl.warps == 1) __syncwarp();  // (K of the next row, as the barrier does)
            mu = st.x * a.invN;
            rs = rsqrtf(fmaf(st.y, a.invN, a.eps));
            if (on && pl.first) {
                if (a.mean) a.mean[row] = K + mu;
                if (a.rstd) a.rstd[row] = rs;
            }
        } else {
            rs = rsqrtf(fmaf(drop_sum(sums, pl, parity, make_float2(s2.x + s2.y, 0.f)).x, a.invN, a.eps));
        }
        const float2 rs2 = f2_splat(rs), nmr = f2_splat(-mu * rs);
        T* yp = static_cast<T*>(a.y) + row * a.N + static_cast<int64_t>(pl.f0) * VEC;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (on && j < pl.nv) {
                Raw yr = X::zero();
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if constexpr (LN)
                        X::set(yr, i, __ffma2_rn(__ffma2_rn(d[j][i], rs2, nmr), X::get(gv[j], i), X::get(bv[j], i)));
                    else
                        X::set(yr, i, __fmul2_rn(__fmul2_rn(d[j][i], X::get(gv[j], i)), rs2));
                }
                X::store(yp + j * pl.step * VEC, yr);
            }
    }
    if (pl.C > 1) cluster_barrier();  // no CTA leaves while a peer may read its state
}

template <class T, int VEC, int V, bool LN>
cudaError_t drop_launch_fwd(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    const void* fn = reinterpret_cast<const void*>(drop_fwd<T, VEC, V, LN>);
    a.words_at = static_cast<int32_t>(drop_ring_bytes(VEC, sizeof(T), V, p.threads, a.stages, 2));
    const size_t smem = static_cast<size_t>(a.words_at + drop_mask_bytes(VEC, V, p.threads, a.lanes));
    int64_t most = 0;
    const cudaError_t e = drop_resident(fn, p.threads, smem, p.cluster, &most);
    if (e != cudaSuccess) return e;
    return drop_launch(fn, std::min(p.grid, most), p.threads, smem, p.cluster, s, a);
}

template <class T, bool LN>
cudaError_t drop_fwd_of(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    if (p.vec_elems == full) {
        switch (p.per_thread) {
            case 1: return drop_launch_fwd<T, full, 1, LN>(p, a, s);
            case 2: return drop_launch_fwd<T, full, 2, LN>(p, a, s);
            case 4: return drop_launch_fwd<T, full, 4, LN>(p, a, s);
        }
    } else if (p.vec_elems == 1) {
        switch (p.per_thread) {
            case 4: return drop_launch_fwd<T, 1, 4, LN>(p, a, s);
            case 16: return drop_launch_fwd<T, 1, 16, LN>(p, a, s);
        }
    }
    return cudaErrorInvalidValue;
}

template <class T>
cudaError_t drop_dispatch_fwd(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return ln ? drop_fwd_of<T, true>(p, a, s) : drop_fwd_of<T, false>(p, a, s);
}

}  // namespace libnorm
