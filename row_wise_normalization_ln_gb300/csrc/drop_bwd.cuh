// Backward of dropout, residual add and norm (and of the plain fused add):
//   LayerNorm: xhat = (h - mean) rstd, g = dy gamma,
//              d = dh + rstd (g - mean(g) - xhat mean(g xhat))
//   RMSNorm:   d = dh + rstd dy w - h rstd^3 mean(dy w h), rstd from h
//   dresidual = d,  dx = d keep / P(keep),  dgamma = sum dy xhat,  dbeta = sum dy
// The R rows of a step are read from shared memory twice: for their sums, and
// for the outputs. (Forming the sums of the next step before the outputs of
// this one, so that they meet meanwhile, costs the registers and shared memory
// of a second step: LayerNorm bf16 4096 x 8192 80 us to 107.) Column sums stay in
// registers; after kDropChain rows they are added to the thread's own part of
// a partial row (in the workspace; in shared memory where the teams of a CTA
// have columns in common), so that no chain of additions is long.
//
// LayerNorm bf16 4096 x 8192 72 us, 4.7 TB/s; RMSNorm 61.5; RMSNorm f32 2047 x 5000
// 42; RMSNorm bf16 65536 x 2048 208, 6.5 TB/s. Wide rows are bound by instructions
// and their latency: one team of 16 warps is all that an SM has, it waits as a
// whole at each barrier, and issues in 53% of the cycles; both readings of a row
// unpack it and form dy gamma and h - mean, 40 instructions an element where the
// plain norm's backward, with the row in registers, takes 22. The mask is little
// of it (without dropout 68). Rows of up to 512 vectors that fill their teams
// have several of them an SM and come near the copy.
#pragma once

#include "drop_kernels.cuh"

namespace libnorm {

template <class T, int VEC, int V, int R, bool LN, bool GROUP>
__global__ void __launch_bounds__(kDropMaxThreads, 1) drop_bwd(const __grid_constant__ DropArgs a) {
    using P = DropPlace<VEC, V, GROUP>;
    using X = DropVec<T, VEC>;
    using Raw = typename X::Raw;
    constexpr int H = X::H, NA = LN ? 2 : 1;
    constexpr bool kElems = VEC == 1;
    extern __shared__ __align__(16) char smem[];
    __shared__ DropSums<2 * R> sums;
    const P pl(a, R);
    grid_release();
    grid_wait();
    const DropMask mask(a);
    const bool drop = a.limit != 0 && a.dx;
    const void* const from[3] = {a.hin, a.dy, a.dh};
    using Ring = std::conditional_t<kElems, DropStage<T, 3>, DropRing<T, VEC, V, R, 3, LN, P>>;
    // Elements: the CTA's part of a row.
    const int cta_col = kElems ? pl.rank * pl.warps * P::kRun : 0;
    const int cta_cols = kElems ? max(0, min(a.N - cta_col, pl.warps * P::kRun)) : 0;
    const int in = pl.col - cta_col;
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
    Raw gamma[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        gamma[j] = X::zero();
        if (pl.on(j)) gamma[j] = pl.param(static_cast<const T*>(a.gamma), j);
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
    float* const part = a.ws + static_cast<int64_t>(blockIdx.x / pl.C) * a.partial_pitch;
    float* const shared_cols = reinterpret_cast<float*>(smem + a.sums_at);
    const int team_size = GROUP ? a.lanes : a.team;
    const bool teams = VEC > 1 && static_cast<int>(blockDim.x) > team_size;
    bool begun = false;
    const auto put = [&](float* p, float v) { *p = begun ? *p + v : v; };
    const auto fold = [&] {
#pragma unroll
        for (int k = 0; k < NA; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (pl.on(j)) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float2 v = acc[k][j][i];
                        acc[k][j][i] = make_float2(0.f, 0.f);
                        if (teams) {
                            float* const x = shared_cols + ((k * V + j) * VEC + 2 * i) * blockDim.x + threadIdx.x;
                            put(x, v.x);
                            put(x + blockDim.x, v.y);
                        } else {
                            float* const x = part + static_cast<int64_t>(k) * a.N + pl.col + pl.at(j) + 2 * i;
                            if (pl.valid(j, 2 * i)) put(x, v.x);
                            if (pl.valid(j, 2 * i + 1)) put(x + (kElems ? 32 : 1), v.y);
                        }
                    }
                }
        begun = true;
    };
    const auto has = [&](int r) { return row + r * pl.stride < a.M; };
    const auto stat = [&](int r) {
        if constexpr (!LN) return make_float2(0.f, 0.f);
        else if constexpr (kElems) return make_float2(__ldg(a.mean + row), __ldg(a.rstd + row));
        else return ring.stat(pl, r);
    };
    const auto read = [&](auto whole, int r, int n, int j) {
        [[maybe_unused]] constexpr bool FULL = decltype(whole)::value;
        if constexpr (kElems) return ring.template get<FULL>(ring.row(n) + in * sizeof(T), j, pl.nv);
        else return ring.get(r, n, j);
    };
    float s[2 * R];
    // This thread's part of the step's sums.
    const auto total = [&](auto whole) {
        [[maybe_unused]] constexpr bool FULL = decltype(whole)::value;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
            if (FULL || has(r)) {
                const float mean = stat(r).x;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (FULL || pl.looks(j)) {
                        const Raw hr = read(whole, r, 0, j), yr = read(whole, r, 1, j);
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const float2 g = X::mul(yr, gamma[j], i);
                            if constexpr (LN) {
                                // sums of g and g (h - mean): an element that is not there has g = 0
                                s0 = __fadd2_rn(s0, g);
                                s1 = __ffma2_rn(g, X::plus(hr, i, -mean), s1);
                            } else {
                                s0 = X::fma(hr, hr, i, s0);
                                s1 = __ffma2_rn(g, X::get(hr, i), s1);
                            }
                        }
                    }
            }
            s[2 * r] = s0.x + s0.y;
            s[2 * r + 1] = s1.x + s1.y;
        }
    };
    int parity = 0;
    // The outputs of the step, from its sums.
    const auto emit = [&](auto whole) {
        constexpr bool FULL = decltype(whole)::value;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (FULL || has(r)) {
                // xhat = (h - mean) rstd (RMSNorm: mean 0), d = dh + rstd (g - mean(g) - xhat mean(g xhat))
                const int64_t at = (row + r * pl.stride) * a.N + pl.col;  // the thread's first element of the row
                const float2 st = stat(r);
                float rs = st.y;
                if constexpr (!LN) rs = rsqrtf(fmaf(s[2 * r], a.invN, a.eps));
                const float2 n0 = f2_splat(-s[2 * r] * a.invN), n1 = f2_splat(-rs * (s[2 * r + 1] * a.invN));
                const float2 rs2 = f2_splat(rs), scale = f2_splat(a.scale);
                T* const rp = static_cast<T*>(a.dres) + at;
                T* const xp = static_cast<T*>(a.dx) + at;
                [[maybe_unused]] uint32_t ws = 0;
                if constexpr (kElems) ws = words_at + parity * words_row * 16 + (static_cast<uint32_t>((at - in) & 7) + in) * 2;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (FULL || pl.looks(j)) {
                        const Raw hr = read(whole, r, 0, j), yr = read(whole, r, 1, j);
                        Raw er = X::zero(), orr = X::zero(), oxr = X::zero();
                        if (a.dh) er = read(whole, r, 2, j);
                        float2 d[H];
                        DropWords<VEC, LN> w;
                        if (drop) {
                            if constexpr (kElems) w.take(ws + pl.at(j) * 2);
                            else w.take(mask, static_cast<uint64_t>(at + pl.at(j)) / VEC);
                        }
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            float2 g = X::mul(yr, gamma[j], i), xh;
                            const float2 yv = X::get(yr, i);
                            if constexpr (LN) {
                                xh = X::plus(hr, i, -st.x);
                                g = __fadd2_rn(g, n0);
                                acc[NA - 1][j][i] = __fadd2_rn(acc[NA - 1][j][i], yv);
                            } else {
                                xh = X::get(hr, i);
                            }
                            xh = __fmul2_rn(xh, rs2);
                            acc[0][j][i] = __ffma2_rn(yv, xh, acc[0][j][i]);
                            d[i] = __ffma2_rn(rs2, __ffma2_rn(xh, n1, g), X::get(er, i));
                            X::set(orr, i, d[i]);
                        }
                        pl.template store<FULL>(rp, j, orr);
                        if (a.dx) {
#pragma unroll
                            for (int i = 0; i < H; ++i) {
                                const float2 dx = __fmul2_rn(d[i], scale);
                                X::set(oxr, i, make_float2(w.lo(mask, i) ? dx.x : 0.f, w.hi(mask, i) ? dx.y : 0.f));
                            }
                            pl.template store<FULL>(xp, j, oxr);
                        }
                    }
            }
    };
    int chain = 0;
    // A team's rows end its steps; the lanes of a warp take as many as the first of them.
    int64_t first = GROUP ? __shfl_sync(kFullMask, row, 0) : row;
    if constexpr (kElems) {
        if (a.stages == 3) copy_async_wait<1>();
        else copy_async_wait<2>();
        __syncthreads();
    }
    for (; first < a.M; first += rows_step, row += rows_step, parity ^= 1) {
        const bool whole_step = pl.straight && has(R - 1);
        if constexpr (!kElems) {
            ring.wait();
            ring.clear_head(pl);
            if (LN) __syncwarp();  // everyone's copies of the statistics; everyone is done with the last step's
            ring.send(a, pl, from, row + (a.stages - 1) * rows_step);
        }
        if (kElems ? whole_step : pl.most == V && has(R - 1)) total(std::true_type{});
        else total(std::false_type{});
        drop_put<2 * R>(sums, pl, parity, s);
        if constexpr (!GROUP) {
            if (kElems && pl.warps == 1) __syncthreads();
            else pl.sync();
            drop_get<2 * R>(sums, pl, parity, s);
        }
        if (whole_step) emit(std::true_type{});
        else emit(std::false_type{});
        ring.advance();
        if constexpr (kElems) {
            ring.send();  // into the slot read before the last barrier
            row_words(parity ^ 1, row + rows_step);
            if (a.stages == 3) copy_async_wait<1>();
            else copy_async_wait<2>();
            __syncthreads();  // the next row has landed for everyone
        }
        chain += R;
        if (chain >= kDropChain) {
            fold();
            chain = 0;
        }
    }
    fold();
    if (teams) {
        // the teams' sums of each column, in order
        __syncthreads();
        const int n = blockDim.x / team_size;
        for (int i = threadIdx.x; i < NA * a.N; i += blockDim.x) {
            const int k = i / a.N;
            float t = 0.f;
            for (int u = 0; u < n; ++u) {
                const int c = i - k * a.N + P::lead_of(a, static_cast<int64_t>(blockIdx.x) * n + u);
                int j, tl;  // access, thread of the team
                if (GROUP) {
                    j = c / (VEC * a.lanes);
                    tl = c / VEC - j * a.lanes;
                } else {
                    const int w = c / P::kRun, f = (c - w * P::kRun) / VEC;
                    j = f / 32;
                    tl = w * 32 + f - j * 32;
                }
                t += shared_cols[((k * V + j) * VEC + c % VEC) * blockDim.x + u * team_size + tl];
            }
            part[i] = t;
        }
    }
    if (pl.C > 1) cluster_barrier();  // no CTA leaves while a peer may read its sums
}

template <class T, int VEC, int V, int R, bool LN, bool GROUP>
cudaError_t drop_launch_bwd(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    const void* fn = reinterpret_cast<const void*>(drop_bwd<T, VEC, V, R, LN, GROUP>);
    a.partial_pitch = drop_partial_pitch((LN ? 2 : 1) * a.N);
    a.pitch = static_cast<int32_t>(VEC == 1 ? drop_pitch(sizeof(T), V, p.threads) : 0);
    a.words_at = static_cast<int32_t>(drop_ring_bytes(VEC, sizeof(T), V, p.threads, R, a.stages, 3, a.stat_bytes));
    a.sums_at = static_cast<int32_t>(a.words_at + drop_words_bytes(VEC, V, p.threads));
    const bool teams = p.threads > (GROUP ? a.lanes : a.team);
    const size_t smem = static_cast<size_t>(a.sums_at + (teams ? drop_sums_bytes(LN, VEC, V, p.threads) : 0));
    int64_t grid = 0;
    cudaError_t e = drop_grid(fn, p, a, smem, &grid);
    if (e != cudaSuccess) return e;
    e = drop_launch(fn, grid, p.threads, smem, p.cluster, s, a);
    if (e != cudaSuccess) return e;
    return launch_drop_colsum(a, grid / p.cluster, LN, s);
}

template <class T, bool LN>
cudaError_t drop_bwd_of(const norm_plan& p, DropArgs& a, cudaStream_t s) {
    constexpr int full = 16 / sizeof(T);
    const int V = p.per_thread;
    if (p.vec_elems == 1) return drop_launch_bwd<T, 1, 8, 1, LN, false>(p, a, s);
    if (p.mapping == NORM_MAP_GROUP) return drop_launch_bwd<T, full, 2, 2, LN, true>(p, a, s);
    if (V == 1) return drop_launch_bwd<T, full, 1, 4, LN, false>(p, a, s);
    if constexpr (sizeof(T) == 4) return drop_launch_bwd<T, full, 4, 1, LN, false>(p, a, s);
    else return drop_launch_bwd<T, full, 2, 2, LN, false>(p, a, s);
}

template <class T>
cudaError_t drop_dispatch_bwd(const norm_plan& p, DropArgs& a, bool ln, cudaStream_t s) {
    return ln ? drop_bwd_of<T, true>(p, a, s) : drop_bwd_of<T, false>(p, a, s);
}

}  // namespace libnorm
