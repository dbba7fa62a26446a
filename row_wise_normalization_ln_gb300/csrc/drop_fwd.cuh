// Dropout, residual add and norm, forward:
//   h = residual + x keep / P(keep)  (rounded to the row's type),  y = norm(h).
//
// A thread holds its values of R rows, as they are stored, from the add to the
// output. LayerNorm, in two passes over the registers: a warp's sum gives a
// first mean A, rounded; about A the sum r of the differences and that of
// their squares, q, are formed. A + r / n is the mean and q - r^2 / n = M2
// whatever A's error is: neither a mean that dwarfs the spread nor one that
// vanishes beside it costs digits. The warps' states (n, A + c, M2), c = r / n,
// meet behind one barrier by the merge rule in its k-way form, the means as
// differences from the first warp's A:
//   m_w = (A_w - A_0) + c_w,  mean = sum n_w m_w / N,  M2 = sum M2_w + n_w (m_w - mean)^2.
// The output is ((h - A_0) rstd - mean rstd) gamma + beta: the row's mean A_0 + mean
// is rounded for the caller alone (a mean of 3e4 beside a spread of 1 would lose
// its last 2e-3).
// RMSNorm: sums of squares.
//
// RMSNorm bf16 65536 x 2048 171 us, 6.3 TB/s, memory bound; 4096 x 5001 29.2;
// LayerNorm 8192 x 4096 42.7, 6.3 TB/s; 4096 x 8192 43.4, 4096 x 5001 35.3: the chain of
// sums, barrier and merge of a row is longer than its bytes take, and 2 (3) CTAs an
// SM hide part of it. 23 (RMSNorm) and 34 instructions an element, half of them
// the mask's and the conversions'. f32 128 x 1024 2.2 us: latency.
#pragma once

#include "drop_kernels.cuh"

namespace libnorm {

// The states of a CTA's warps (and of a cluster's CTAs) of R rows.
template <int R>
struct DropStates {
    float A[2][R][kDropMaxThreads / 32], mean[2][R][kDropMaxThreads / 32], m2[2][R][kDropMaxThreads / 32];
    float cta[2][3][R];
};

template <int N>
__device__ __forceinline__ float drop_down(float v) {  // sum over aligned blocks of N lanes
#pragma unroll
    for (int off = N / 2; off > 0; off /= 2) v += __shfl_xor_sync(kFullMask, v, off);
    return v;
}

// ASIDE: beta lies in shared memory: LayerNorm's parameters of four accesses
// are 32 registers, and with all of them wide rows have one CTA an SM rather
// than two (bf16 4096 x 8192 54 us, with beta aside 45.4, with both 47.6; 4096 x 5001
// 45, 35.9, 36.2). Narrow rows, in CTAs of at most 128 threads, do without
// (16384 x 1024 22.9 us, aside 25.4).
template <class T, int VEC, int V, int R, bool LN, bool GROUP, bool ASIDE = false>
__global__ void __launch_bounds__(LN && V == 4 && !ASIDE ? kDropNarrow : VEC * V >= 32 ? 256 : kDropMaxThreads, VEC * V >= 32 ? 2 : 1) drop_fwd(const __grid_constant__ DropArgs a) {
    using P = DropPlace<VEC, V, GROUP>;
    using X = DropVec<T, VEC>;
    using Raw = typename X::Raw;
    constexpr int H = X::H;
    constexpr bool kElems = VEC == 1;
    extern __shared__ __align__(16) char smem[];
    __shared__ std::conditional_t<LN, DropStates<R>, DropSums<R>> sums;
    const P pl(a, R);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_release();
    grid_wait();
    const DropMask mask(a);
    const bool drop = a.limit != 0;
    const bool full = pl.full;
    const void* const from[2] = {a.x, a.residual};
    using Ring = std::conditional_t<kElems, DropStage<T, 2>, DropRing<T, VEC, V, R, 2, false, P>>;
    // Elements: the CTA's part of a row.
    const int cta_col = kElems ? pl.rank * pl.warps * P::kRun : 0;
    const int cta_cols = kElems ? max(0, min(a.N - cta_col, pl.warps * P::kRun)) : 0;
    uint4* const words = reinterpret_cast<uint4*>(smem + a.words_at);
    const uint32_t words_at = smem_addr(words);
    const int words_row = kElems ? (pl.warps * P::kRun) / 8 + 2 : 0;
    Ring ring = [&] {
        if constexpr (kElems)
            return Ring(a, pl.first_row, pl.teams, cta_col, cta_cols, smem, from);
        else
            return Ring(a, smem);
    }();
    const int64_t rows_step = pl.teams * R;
    const int64_t row_step = static_cast<int64_t>(pl.stride) * a.N;  // elements from one row of a step to the next
    int64_t row = pl.first_row;
    const auto row_words = [&](int parity, int64_t row) {
        if (kElems && drop && row < a.M)
            drop_stage_words(mask, static_cast<uint64_t>(row) * a.N + cta_col, cta_cols, words + parity * words_row);
    };
    for (int i = 0; i < a.stages - 1; ++i)
        if constexpr (kElems) ring.send();
        else ring.send(a, pl, from, row + i * rows_step);
    row_words(0, row);
    // The parameters of the thread's columns.
    Raw params[V][LN && !ASIDE ? 2 : 1];
    const uint32_t aside = words_at + threadIdx.x * 16;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int k = 0; k < (LN ? 2 : 1); ++k) {
            Raw v = X::zero();
            if (pl.on(j)) v = pl.param(static_cast<const T*>(k == 0 ? a.gamma : a.beta), j);
            if constexpr (ASIDE) {
                if (k == 1) {
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(aside + j * blockDim.x * 16), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                    continue;
                }
            }
            params[j][LN && !ASIDE ? k : 0] = v;
        }
    const auto param = [&](int j, int k) {
        if constexpr (ASIDE) {
            if (k == 1) {
                Raw v;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "r"(aside + j * blockDim.x * 16)
                             : "memory");
                return v;
            }
        }
        return params[j][LN && !ASIDE ? k : 0];
    };
    // LayerNorm: elements of this warp's part, of the warps whose states this
    // lane merges, of the CTA's.
    const DropShare<R> sh;
    constexpr int E = DropShare<R>::kEach, L = DropShare<R>::kLanes;
    float n_warp = 0.f, n_of[E], n_cta = 0.f;
    if constexpr (LN) {
        n_warp = GROUP ? static_cast<float>(a.N) : pl.count(a, pl.rank, warp - pl.warp0);
#pragma unroll
        for (int i = 0; i < E; ++i) n_of[i] = !GROUP && sh.w0 + i < pl.warps ? pl.count(a, pl.rank, sh.w0 + i) : 0.f;
        if (!GROUP) n_cta = pl.count_cta(a, pl.rank);
    }
    const float inv_warp = n_warp > 0.f ? 1.f / n_warp : 0.f, inv_cta = n_cta > 0.f ? 1.f / n_cta : 0.f;

    const auto has = [&](int r) { return row + r * pl.stride < a.M; };
    int parity = 0;
    // A team's rows end its steps; the lanes of a warp take as many as the first of them.
    int64_t first = GROUP ? __shfl_sync(kFullMask, row, 0) : row;
    if constexpr (kElems) {
        if (a.stages == 3) copy_async_wait<1>();
        else copy_async_wait<2>();
        __syncthreads();
    }
    for (; first < a.M; first += rows_step, row += rows_step, parity ^= 1) {
        const int64_t at = row * a.N + pl.col;  // the thread's first element of the step's first row
        const uint64_t group = VEC > 1 ? static_cast<uint64_t>(at) / VEC : 0;
        Raw h[R][V];
        float s[R];
        if constexpr (!kElems) {
            ring.wait();
            ring.clear_head(pl);
            ring.send(a, pl, from, row + (a.stages - 1) * rows_step);  // into the slots read a step ago
        }
        // h, and the first sums; FULL: every access of the warp is there (elements; vectors look at each).
        const auto add = [&](auto whole) {
            constexpr bool FULL = decltype(whole)::value;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool on = has(r);
                T* const hp = static_cast<T*>(a.h) + at + r * row_step;
                [[maybe_unused]] uint32_t xs = 0, rs = 0, ws = 0;
                if constexpr (kElems) {
                    const int in = pl.col - cta_col;
                    xs = ring.row(0) + in * sizeof(T);
                    rs = ring.row(1) + in * sizeof(T);
                    ws = words_at + parity * words_row * 16 + (static_cast<uint32_t>((at - in) & 7) + in) * 2;
                }
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (!FULL) h[r][j] = X::zero();
                    if (FULL || (on && pl.looks(j))) {
                        Raw xr, rr, hr = X::zero();
                        if constexpr (kElems) {
                            xr = ring.template get<FULL>(xs, j, pl.nv);
                            rr = ring.template get<FULL>(rs, j, pl.nv);
                        } else {
                            xr = ring.get(r, 0, j);
                            rr = ring.get(r, 1, j);
                        }
                        DropWords<VEC, LN> w;
                        if (drop) {
                            if constexpr (kElems) w.take(ws + pl.at(j) * 2);
                            else w.take(mask, group + r * (row_step / VEC) + pl.at(j) / VEC);
                        }
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const float2 xv = X::get(xr, i);
                            float2 hv = X::get(rr, i);
                            if (w.lo(mask, i)) hv.x = fmaf(xv.x, a.scale, hv.x);
                            if (w.hi(mask, i)) hv.y = fmaf(xv.y, a.scale, hv.y);
                            X::set(hr, i, hv);
                        }
                        pl.template store<FULL>(hp, j, hr);
                        h[r][j] = hr;
                        // (what is not in the row is 0)
#pragma unroll
                        for (int i = 0; i < H; ++i) sum = LN ? X::sum(hr, i, sum) : X::fma(hr, hr, i, sum);
                    }
                }
                s[r] = sum.x + sum.y;
            }
        };
        const bool whole_step = pl.straight && has(R - 1);
        if (whole_step) add(std::true_type{});
        else add(std::false_type{});
        ring.advance();
        if constexpr (kElems) {
            ring.send();  // into the slot read before the last barrier
            row_words(parity ^ 1, row + rows_step);
            if (a.stages == 3) copy_async_wait<1>();
            else copy_async_wait<2>();     // the next row has landed; the barrier below makes it everyone's
        }
        float rstd[R], A0[R], off[R];  // LayerNorm: y = ((h - A0) rstd + off) gamma + beta
        if constexpr (LN) {
            float A[R], mean[R], q[R];
            if (GROUP) {
#pragma unroll
                for (int r = 0; r < R; ++r) A[r] = group_sum(s[r], pl.unit) * inv_warp;
            } else {
                const float t = warp_sums<R>(s);
#pragma unroll
                for (int r = 0; r < R; ++r) A[r] = __shfl_sync(kFullMask, t, R == 1 ? 0 : r * (32 / R)) * inv_warp;
            }
            float qr[2 * R];  // of the rows: sums of squares, sums of differences
            const auto differences = [&](auto whole) {
                constexpr bool FULL = decltype(whole)::value;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 squares = make_float2(0.f, 0.f), sum = squares;
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (FULL || pl.looks(j)) {
                            float2 e[H];
#pragma unroll
                            for (int i = 0; i < H; ++i) e[i] = X::plus(h[r][j], i, -A[r]);
                            if (!FULL && (kElems || !pl.whole(j))) {
#pragma unroll
                                for (int i = 0; i < H; ++i) {
                                    if (!pl.valid(j, 2 * i)) e[i].x = 0.f;
                                    if (!pl.valid(j, 2 * i + 1)) e[i].y = 0.f;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < H; ++i) {
                                squares = __ffma2_rn(e[i], e[i], squares);
                                sum = __fadd2_rn(sum, e[i]);
                            }
                        }
                    qr[r] = squares.x + squares.y;
                    qr[R + r] = sum.x + sum.y;
                }
            };
            if (full) differences(std::true_type{});
            else differences(std::false_type{});
            if (GROUP) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float d = group_sum(qr[R + r], pl.unit);
                    mean[r] = d * inv_warp;
                    q[r] = fmaf(-d, mean[r], group_sum(qr[r], pl.unit));
                    q[r] = q[r] < 0.f ? 0.f : q[r];  // (of equal values)
                    A0[r] = A[r];
                }
            } else {
                const float t = warp_sums<2 * R>(qr);
                const int mine = lane / (32 / R);  // the row whose state this lane has
                const float d = __shfl_sync(kFullMask, t, 16 + mine * (16 / R));
                float k = A[0], m = d * inv_warp;
                float m2 = fmaf(-d, m, __shfl_sync(kFullMask, t, mine * (16 / R)));
                m2 = m2 < 0.f ? 0.f : m2;  // (of equal values)
#pragma unroll
                for (int r = 1; r < R; ++r)
                    if (mine == r) k = A[r];
                if (pl.warps > 1) {
                    if ((lane & (32 / R - 1)) == 0) {
                        const int r = lane / (32 / R);
                        sums.A[parity][r][warp] = k;
                        sums.mean[parity][r][warp] = m;
                        sums.m2[parity][r][warp] = m2;
                    }
                    pl.sync();
                    const int w0 = pl.warp0 + sh.w0;
                    k = sums.A[parity][sh.idx][pl.warp0];
                    float t = 0.f, dm[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        dm[i] = 0.f;
                        if (n_of[i] > 0.f) {
                            dm[i] = (sums.A[parity][sh.idx][w0 + i] - k) + sums.mean[parity][sh.idx][w0 + i];
                            t = fmaf(n_of[i], dm[i], t);
                        }
                    }
                    m = drop_down<L>(t) * inv_cta;
                    t = 0.f;
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (n_of[i] > 0.f) t += fmaf(n_of[i] * (dm[i] - m), dm[i] - m, sums.m2[parity][sh.idx][w0 + i]);
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
                    const float n = lane < pl.C ? pl.count_cta(a, lane) : 0.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float pk = 0.f, pm = 0.f, pq = 0.f;
                        if (n > 0.f) {
                            pk = drop_peer(&sums.cta[parity][0][r], static_cast<uint32_t>(lane));
                            pm = drop_peer(&sums.cta[parity][1][r], static_cast<uint32_t>(lane));
                            pq = drop_peer(&sums.cta[parity][2][r], static_cast<uint32_t>(lane));
                        }
                        A0[r] = __shfl_sync(kFullMask, pk, 0);
                        const float dm = n > 0.f ? (pk - A0[r]) + pm : 0.f;
                        mean[r] = __shfl_sync(kFullMask, drop_down<8>(n * dm), 0) * a.invN;
                        q[r] = __shfl_sync(kFullMask, drop_down<8>(fmaf(n * (dm - mean[r]), dm - mean[r], pq)), 0);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        if (R == 1) {  // (every lane has the row's)
                            mean[r] = m;
                            q[r] = m2;
                            A0[r] = k;
                            continue;
                        }
                        mean[r] = __shfl_sync(kFullMask, m, r * S);
                        q[r] = __shfl_sync(kFullMask, m2, r * S);
                        A0[r] = __shfl_sync(kFullMask, k, r * S);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                rstd[r] = rsqrtf(fmaf(q[r], a.invN, a.eps));
                off[r] = -mean[r] * rstd[r];
                if (has(r) && pl.first) {
                    if (a.mean) a.mean[row + r * pl.stride] = A0[r] + mean[r];
                    if (a.rstd) a.rstd[row + r * pl.stride] = rstd[r];
                }
            }
        } else {
            drop_put<R>(sums, pl, parity, s);
            if constexpr (!GROUP) {
                if (kElems && pl.warps == 1) __syncthreads();
                else pl.sync();
                drop_get<R>(sums, pl, parity, s);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) rstd[r] = rsqrtf(fmaf(s[r], a.invN, a.eps));
        }
        const auto emit = [&](auto whole) {
            constexpr bool FULL = decltype(whole)::value;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 rs2 = f2_splat(rstd[r]);
                [[maybe_unused]] const float2 off2 = f2_splat(LN ? off[r] : 0.f);
                T* const yp = static_cast<T*>(a.y) + at + r * row_step;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (FULL || (has(r) && pl.looks(j))) {
                        Raw yr = X::zero();
                        const Raw gv = param(j, 0);
                        [[maybe_unused]] Raw bv;
                        if constexpr (LN) bv = param(j, 1);
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            if constexpr (LN)
                                X::set(yr, i, __ffma2_rn(__ffma2_rn(X::plus(h[r][j], i, -A0[r]), rs2, off2), X::get(gv, i), X::get(bv, i)));
                            else
                                X::set(yr, i, __fmul2_rn(X::mul(h[r][j], gv, i), rs2));
                        }
                        pl.template store<FULL>(yp, j, yr);
                    }
            }
        };
        if (whole_step) emit(std::true_type{});
        else emit(std::false_type{});
    }
    if (pl.C > 1) cluster_barrier();  // no CTA leaves while a peer may read its state
}

template <class T, int VEC, int V, int R, bool LN, bool GROUP, bool ASIDE = false>
cudaError_t drop_launch_fwd(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    const void* fn = reinterpret_cast<const void*>(drop_fwd<T, VEC, V, R, LN, GROUP, ASIDE>);
    a.pitch = static_cast<int32_t>(VEC == 1 ? drop_pitch(sizeof(T), V, p.threads) : 0);
    a.words_at = static_cast<int32_t>(drop_ring_bytes(VEC, sizeof(T), V, p.threads, R, a.stages, 2, 0));
    const size_t smem = static_cast<size_t>(a.words_at + drop_words_bytes(VEC, V, p.threads) + drop_param_bytes(LN, VEC, V, p.threads));
    int64_t grid = 0;
    const cudaError_t e = drop_grid(fn, p, a, smem, &grid);
    if (e != cudaSuccess) return e;
    return drop_launch(fn, grid, p.threads, smem, p.cluster, s, a);
}

template <class T, bool LN>
cudaError_t drop_fwd_of(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    const int V = p.per_thread, R = p.rounds;
    if (p.vec_elems == 1) return drop_launch_fwd<T, 1, 8, 1, LN, false>(p, a, s);
    if (p.mapping == NORM_MAP_GROUP) return drop_launch_fwd<T, full, 2, 2, LN, true>(p, a, s);
    if (V == 1) return R == 1 ? drop_launch_fwd<T, full, 1, 1, LN, false>(p, a, s) : drop_launch_fwd<T, full, 1, 4, LN, false>(p, a, s);
    if (LN && p.threads > kDropNarrow) return drop_launch_fwd<T, full, 4, 1, LN, false, LN>(p, a, s);
    return drop_launch_fwd<T, full, 4, 1, LN, false>(p, a, s);
}

template <class T>
cudaError_t drop_dispatch_fwd(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return ln ? drop_fwd_of<T, true>(p, a, s) : drop_fwd_of<T, false>(p, a, s);
}

}  // namespace libnorm
