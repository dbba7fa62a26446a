// RMSNorm of query and key heads with the rotary rotation in the same pass,
// forward and backward, for sm_103a.
//
// A head is D values of one token: r = 1 / sqrt(mean x^2 + eps), z = x r w,
// and the pairs (a, b) of its first R values turn by the token's angle:
//   y_a = z_a c - z_b s,   y_b = z_b c + z_a s.
// Backward, with dz = dy turned back (s -> -s) and g = dz w:
//   dx = r g - x r^3 mean(g x),   dw = sum dz x r.
//
// 2^lanes_log neighbouring lanes own a head; a lane holds pairs of accesses
// (a, b) of VEC values whose elements are each other's partners in the
// rotation (i and i + R / 2; interleaved vectors hold whole pairs, and any two
// accesses do), so the rotation needs no exchange and a cosine is loaded once
// per pair. A warp works on one token and walks its heads, 32 / lanes at a
// time: the token's angles and the weight stay in registers, and a batch of
// heads is in flight before the first is reduced. The sums of a head meet in
// butterflies over its lanes; nothing meets across warps until the backward's
// column sums.
#pragma once

#include "gn_kernels.cuh"
#include "rope_args.h"

namespace libnorm {

// VEC values of an access as fp32 pairs (one value: the second of the pair is 0).
template <class T, int VEC>
struct RopeVals {
    using X = GnVec<T, VEC>;
    static constexpr int H = X::H;
    float2 v[H];
    __device__ __forceinline__ void widen(const typename X::Raw& r) {
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = X::get(r, i);
    }
    __device__ __forceinline__ typename X::Raw round() const {
        typename X::Raw r = X::zero();
#pragma unroll
        for (int i = 0; i < H; ++i) X::set(r, i, v[i]);
        return r;
    }
};

// A lane's place in a head: where its accesses start and how they turn.
// ILV: pairs (2 i, 2 i + 1) within an access (VEC > 1).
template <int VEC, int NP, bool ILV>
struct RopeLane {
    static constexpr bool kInside = ILV && VEC > 1;
    int a[NP], b[NP];    // first element of each access of a pair; -1: none
    bool ra[NP], rb[NP]; // it turns
    int ca[NP], cb[NP];  // its first angle (kInside: b's own; otherwise they share a's)

    __device__ __forceinline__ RopeLane(const RopeArgs& g, int lane) {
        const int lanes = 1 << g.lanes_log;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int p = lane + j * lanes;
            a[j] = b[j] = -1;
            ra[j] = rb[j] = false;
            ca[j] = cb[j] = 0;
            if (p >= g.npairs) continue;
            if constexpr (kInside) {
                a[j] = p * VEC;
                b[j] = (g.npairs + p) * VEC < g.D ? (g.npairs + p) * VEC : -1;
                ra[j] = a[j] < g.R;
                rb[j] = b[j] >= 0 && b[j] < g.R;
                ca[j] = a[j] / 2;
                cb[j] = rb[j] ? b[j] / 2 : 0;
            } else if (p < g.rot_pairs) {
                a[j] = ILV ? 2 * p : p * VEC;
                b[j] = ILV ? 2 * p + 1 : g.R / 2 + p * VEC;
                ra[j] = rb[j] = true;
                ca[j] = p * VEC;
            } else {
                const int q = p - g.rot_pairs, half = g.npairs - g.rot_pairs;
                a[j] = g.R + q * VEC;
                b[j] = g.R + (half + q) * VEC < g.D ? g.R + (half + q) * VEC : -1;
            }
        }
    }
};

// A token's angles for a lane's pairs: cosines and sines of pairs of elements
// (a, b); kInside: half of them a's, half b's.
template <int VEC, int NP, bool ILV>
struct RopeAngles {
    static constexpr bool kInside = ILV && VEC > 1;
    static constexpr int W = VEC == 1 ? 1 : VEC / 2;  // float2s per access and pair
    float2 c[NP][W], s[NP][W];

    // n floats of a table row (n <= 8, whole float4s where the rows are aligned and n >= 4)
    template <int N>
    static __device__ __forceinline__ void fetch(float* to, const float* p, bool vec) {
        if constexpr (N % 4 == 0) {
            if (vec) {
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
                    to[i] = v.x;
                    to[i + 1] = v.y;
                    to[i + 2] = v.z;
                    to[i + 3] = v.w;
                }
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = __ldg(p + i);
    }
    __device__ __forceinline__ void load(const RopeArgs& g, const RopeLane<VEC, NP, ILV>& l, int64_t pos) {
        const float* cp = g.cos + pos * g.table_pitch;
        const float* sp = g.sin + pos * g.table_pitch;
        const bool vec = g.vec_table != 0;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            float tc[2 * W], ts[2 * W];
            if constexpr (kInside) {
                if (l.ra[j]) {
                    fetch<W>(tc, cp + l.ca[j], vec);
                    fetch<W>(ts, sp + l.ca[j], vec);
                }
                if (l.rb[j]) {
                    fetch<W>(tc + W, cp + l.cb[j], vec);
                    fetch<W>(ts + W, sp + l.cb[j], vec);
                }
            } else if (l.ra[j]) {
                fetch<VEC>(tc, cp + l.ca[j], vec);
                fetch<VEC>(ts, sp + l.ca[j], vec);
            }
            if constexpr (VEC == 1) tc[1] = ts[1] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                c[j][i] = make_float2(tc[2 * i], tc[2 * i + 1]);
                s[j][i] = make_float2(ts[2 * i], ts[2 * i + 1]);
            }
        }
    }
    // The pair j of accesses turned by the angle, or (BACK) against it.
    template <bool BACK, class V>
    __device__ __forceinline__ void turn(const RopeLane<VEC, NP, ILV>& l, int j, V& a, V& b) const {
        if constexpr (kInside) {
            // (angles k of an access: element pair k)
            const auto at = [](const float2* t, int k) { return (k & 1) ? t[k >> 1].y : t[k >> 1].x; };
#pragma unroll
            for (int k = 0; k < W; ++k) {
                if (l.ra[j]) {
                    const float co = at(c[j], k), si = BACK ? -at(s[j], k) : at(s[j], k);
                    const float2 v = a.v[k];
                    a.v[k] = make_float2(fmaf(v.x, co, -(v.y * si)), fmaf(v.y, co, v.x * si));
                }
                if (l.rb[j]) {
                    const float co = at(c[j], W + k), si = BACK ? -at(s[j], W + k) : at(s[j], W + k);
                    const float2 v = b.v[k];
                    b.v[k] = make_float2(fmaf(v.x, co, -(v.y * si)), fmaf(v.y, co, v.x * si));
                }
            }
        } else if (l.ra[j]) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 si = BACK ? make_float2(-s[j][i].x, -s[j][i].y) : s[j][i];
                const float2 va = a.v[i], vb = b.v[i];
                a.v[i] = __ffma2_rn(va, c[j][i], __fmul2_rn(make_float2(-vb.x, -vb.y), si));
                b.v[i] = __ffma2_rn(vb, c[j][i], __fmul2_rn(va, si));
            }
        }
    }
};

__device__ __forceinline__ int64_t rope_position(const RopeArgs& g, int t, int s) {
    if (g.pos_bytes == 8) return __ldg(static_cast<const long long*>(g.positions) + t);
    if (g.pos_bytes == 4) return __ldg(static_cast<const int*>(g.positions) + t);
    return s;
}

// Where a warp's task lies: the token's offset in each tensor, the first head
// group and the one after the last.
struct RopeTask {
    int t, b, s, slot, end;
    __device__ __forceinline__ RopeTask(const RopeArgs& g, const RopeSide& sd, int task) {
        t = quot(task, sd.by_chunks);
        slot = (task - t * sd.chunks) * g.chunk_slots;
        end = min(sd.slots, slot + g.chunk_slots);
        b = quot(t, g.by_S);
        s = t - b * g.S;
    }
};

template <class T>
__device__ __forceinline__ T* rope_at(const norm_heads& h, const RopeTask& k) {
    return static_cast<T*>(h.data) + k.b * h.batch + k.s * h.token;
}

// The weight of a lane's accesses, widened.
template <class T, int VEC, int NP, bool ILV>
struct RopeWeight {
    RopeVals<T, VEC> a[NP], b[NP];
    __device__ __forceinline__ RopeWeight(const RopeLane<VEC, NP, ILV>& l, const T* w) {
        using X = GnVec<T, VEC>;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            a[j].widen(l.a[j] >= 0 ? X::load(w + l.a[j]) : X::zero());
            b[j].widen(l.b[j] >= 0 ? X::load(w + l.b[j]) : X::zero());
        }
    }
};

// ------------------------------------------------------------ forward
// U heads per lane group are loaded before the first is reduced.
template <class T, int VEC, int NP, bool ILV, int U>
__global__ void __launch_bounds__(kRopeMaxWarps * 32) rope_fwd(const __grid_constant__ RopeArgs g) {
    using X = GnVec<T, VEC>;
    using V = RopeVals<T, VEC>;
    grid_release();
    const bool second = static_cast<int>(blockIdx.x) >= g.side[0].ctas;
    const RopeSide& sd = g.side[second];
    const int cta = static_cast<int>(blockIdx.x) - (second ? g.side[0].ctas : 0);
    const int64_t task = int64_t(cta) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int lanes = 1 << g.lanes_log, groups = 32 >> g.lanes_log;
    const int group = lane >> g.lanes_log;
    const RopeLane<VEC, NP, ILV> l(g, lane & (lanes - 1));
    grid_wait();
    if (task >= sd.tasks) return;  // (a whole warp)
    const RopeTask k(g, sd, static_cast<int>(task));
    const int64_t pos = rope_position(g, k.t, k.s);
    const T* x = rope_at<const T>(sd.x, k);
    T* y = rope_at<T>(sd.y, k);

    typename X::Raw xa[U][NP], xb[U][NP];
    const auto load = [&](int slot) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (slot + u) * groups + group;
            const bool on = slot + u < k.end && h < sd.heads;
            const T* p = x + h * sd.x.head;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                xa[u][j] = on && l.a[j] >= 0 ? X::load(p + l.a[j]) : X::zero();
                xb[u][j] = on && l.b[j] >= 0 ? X::load(p + l.b[j]) : X::zero();
            }
        }
    };
    load(k.slot);  // before the position is known: its latency and the table's pass meanwhile
    const RopeWeight<T, VEC, NP, ILV> w(l, static_cast<const T*>(sd.w));
    RopeAngles<VEC, NP, ILV> ang;
    const bool pad = pos < 0, none = pos >= g.P;
    if (!pad && !none) ang.load(g, l, pos);
    for (int slot = k.slot; slot < k.end;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (slot + u) * groups + group;
            const bool on = slot + u < k.end && h < sd.heads;
            V va[NP], vb[NP];
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                va[j].widen(xa[u][j]);
                vb[j].widen(xb[u][j]);
#pragma unroll
                for (int i = 0; i < X::H; ++i) {
                    ss = __ffma2_rn(va[j].v[i], va[j].v[i], ss);
                    ss = __ffma2_rn(vb[j].v[i], vb[j].v[i], ss);
                }
            }
            const float sum = group_sum(ss.x + ss.y, lanes);
            float r = rsqrtf(fmaf(sum, g.invD, g.eps));
            if (none) r = __int_as_float(0x7fffffff);  // no angle: NaN
            const float2 r2 = f2_splat(r);
            T* p = y + h * sd.y.head;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
#pragma unroll
                for (int i = 0; i < X::H; ++i) {
                    va[j].v[i] = __fmul2_rn(__fmul2_rn(va[j].v[i], r2), w.a[j].v[i]);
                    vb[j].v[i] = __fmul2_rn(__fmul2_rn(vb[j].v[i], r2), w.b[j].v[i]);
                }
                ang.template turn<false>(l, j, va[j], vb[j]);
                if (on && l.a[j] >= 0) X::store(p + l.a[j], pad ? X::zero() : va[j].round());
                if (on && l.b[j] >= 0) X::store(p + l.b[j], pad ? X::zero() : vb[j].round());
            }
        }
        slot += U;
        if (slot < k.end) load(slot);
    }
}

// ------------------------------------------------------------ backward
// Persistent: a CTA keeps one side's dw in registers over its tasks. A chain
// of additions is at most kRopeChain heads long; the sums of the chains are
// added in this lane's slots of shared memory.
constexpr int kRopeChain = 64;

template <class T, int VEC, int NP, bool ILV, int U>
__global__ void __launch_bounds__(kRopeMaxWarps * 32) rope_bwd(const __grid_constant__ RopeArgs g) {
    using X = GnVec<T, VEC>;
    using V = RopeVals<T, VEC>;
    constexpr int H = X::H;
    extern __shared__ float2 sums[];  // [NP * 2 * H][threads]
    grid_release();
    const bool second = static_cast<int>(blockIdx.x) >= g.side[0].ctas;
    const RopeSide& sd = g.side[second];
    const int cta = static_cast<int>(blockIdx.x) - (second ? g.side[0].ctas : 0);
    const int warps = blockDim.x >> 5;
    const int lane = threadIdx.x & 31;
    const int lanes = 1 << g.lanes_log, groups = 32 >> g.lanes_log;
    const int group = lane >> g.lanes_log;
    const RopeLane<VEC, NP, ILV> l(g, lane & (lanes - 1));
    V da[NP], db[NP];  // this lane's share of dw
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) da[j].v[i] = db[j].v[i] = make_float2(0.f, 0.f);
    float2* mine = sums + threadIdx.x;
#pragma unroll
    for (int i = 0; i < NP * 2 * H; ++i) mine[i * blockDim.x] = make_float2(0.f, 0.f);
    int chain = 0;
    const auto fold = [&] {
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                float2& fa = mine[((j * 2) * H + i) * blockDim.x];
                float2& fb = mine[((j * 2 + 1) * H + i) * blockDim.x];
                fa = __fadd2_rn(fa, da[j].v[i]);
                fb = __fadd2_rn(fb, db[j].v[i]);
                da[j].v[i] = db[j].v[i] = make_float2(0.f, 0.f);
            }
        chain = 0;
    };
    grid_wait();
    const RopeWeight<T, VEC, NP, ILV> w(l, static_cast<const T*>(sd.w));
    const int64_t step = int64_t(sd.ctas) * warps;
    for (int64_t task = int64_t(cta) * warps + (threadIdx.x >> 5); task < sd.tasks; task += step) {
        const RopeTask k(g, sd, static_cast<int>(task));
        const int64_t pos = rope_position(g, k.t, k.s);
        const T* x = rope_at<const T>(sd.x, k);
        const T* dy = rope_at<const T>(sd.dy, k);
        T* dx = rope_at<T>(sd.y, k);
        typename X::Raw xa[U][NP], xb[U][NP], ya[U][NP], yb[U][NP];
        const auto load = [&](int slot) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = (slot + u) * groups + group;
                const bool on = slot + u < k.end && h < sd.heads;
                const T* p = x + h * sd.x.head;
                const T* q = dy + h * sd.dy.head;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    xa[u][j] = on && l.a[j] >= 0 ? X::load(p + l.a[j]) : X::zero();
                    xb[u][j] = on && l.b[j] >= 0 ? X::load(p + l.b[j]) : X::zero();
                    ya[u][j] = on && l.a[j] >= 0 ? X::load(q + l.a[j]) : X::zero();
                    yb[u][j] = on && l.b[j] >= 0 ? X::load(q + l.b[j]) : X::zero();
                }
            }
        };
        load(k.slot);
        RopeAngles<VEC, NP, ILV> ang;
        const bool pad = pos < 0, none = pos >= g.P;
        if (!pad && !none) ang.load(g, l, pos);
        for (int slot = k.slot; slot < k.end;) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = (slot + u) * groups + group;
                const bool on = slot + u < k.end && h < sd.heads;
                V za[NP], zb[NP];
                float2 ss = make_float2(0.f, 0.f), sg = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    za[j].widen(ya[u][j]);
                    zb[j].widen(yb[u][j]);
                    ang.template turn<true>(l, j, za[j], zb[j]);
                    V va, vb;
                    va.widen(xa[u][j]);
                    vb.widen(xb[u][j]);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        ss = __ffma2_rn(va.v[i], va.v[i], ss);
                        ss = __ffma2_rn(vb.v[i], vb.v[i], ss);
                        sg = __ffma2_rn(__fmul2_rn(za[j].v[i], w.a[j].v[i]), va.v[i], sg);
                        sg = __ffma2_rn(__fmul2_rn(zb[j].v[i], w.b[j].v[i]), vb.v[i], sg);
                    }
                }
                float s0 = ss.x + ss.y, s1 = sg.x + sg.y;
                group_sum2(s0, s1, lanes);
                float r = rsqrtf(fmaf(s0, g.invD, g.eps));
                if (none) r = __int_as_float(0x7fffffff);
                const float2 r2 = f2_splat(r), m2 = f2_splat(-(r * r * r * (s1 * g.invD)));
                T* p = dx + h * sd.y.head;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    V va, vb, oa, ob;
                    va.widen(xa[u][j]);
                    vb.widen(xb[u][j]);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        oa.v[i] = __ffma2_rn(va.v[i], m2, __fmul2_rn(__fmul2_rn(za[j].v[i], w.a[j].v[i]), r2));
                        ob.v[i] = __ffma2_rn(vb.v[i], m2, __fmul2_rn(__fmul2_rn(zb[j].v[i], w.b[j].v[i]), r2));
                        if (on && !pad) {
                            da[j].v[i] = __ffma2_rn(__fmul2_rn(va.v[i], r2), za[j].v[i], da[j].v[i]);
                            db[j].v[i] = __ffma2_rn(__fmul2_rn(vb.v[i], r2), zb[j].v[i], db[j].v[i]);
                        }
                    }
                    if (on && l.a[j] >= 0) X::store(p + l.a[j], pad ? X::zero() : oa.round());
                    if (on && l.b[j] >= 0) X::store(p + l.b[j], pad ? X::zero() : ob.round());
                }
            }
            slot += U;
            if (slot < k.end) load(slot);
            chain += U;
            if (chain >= kRopeChain) fold();
        }
    }
    fold();
    __syncthreads();
    // A column's terms lie with the lanes of its place in every group of
    // every warp: added in that order, each column by one thread.
    float* part = sd.part + int64_t(cta) * g.D;
    const float* flat = reinterpret_cast<const float*>(sums);
    for (int i = threadIdx.x; i < lanes * NP * 2 * VEC; i += blockDim.x) {
        // element e of access `side` of pair j of lane q
        const int e = i % VEC, q = (i / VEC) % lanes, js = i / (VEC * lanes);
        const RopeLane<VEC, NP, ILV> lq(g, q);
        int c = -1;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (js == 2 * j) c = lq.a[j];
            if (js == 2 * j + 1) c = lq.b[j];
        }
        if (c < 0) continue;
        const float* f = flat + (js * H + e / 2) * 2 * blockDim.x + e % 2;
        float t = 0.f;
        for (int th = q; th < static_cast<int>(blockDim.x); th += lanes) t += f[2 * th];
        part[c + e] = t;
    }
}

// ------------------------------------------------------------ launch
template <class T, int VEC, int NP, bool ILV, int UF, int UB>
cudaError_t rope_launch(const norm_rope_plan& p, const RopeArgs& a, bool backward, cudaStream_t s) {
    const void* fn = backward ? reinterpret_cast<const void*>(rope_bwd<T, VEC, NP, ILV, UB>)
                              : reinterpret_cast<const void*>(rope_fwd<T, VEC, NP, ILV, UF>);
    const int threads = p.warps * 32;
    const size_t smem = backward ? size_t(NP) * 2 * GnVec<T, VEC>::H * sizeof(float2) * threads : 0;
    if (smem > 48 * 1024) {
        const cudaError_t e = gn_opt_in(fn);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.side[0].ctas + a.side[1].ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<RopeArgs*>(&a)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <class T, int VEC, int NP, int UF, int UB>
cudaError_t rope_style(const norm_rope_plan& p, const RopeArgs& a, bool interleaved, bool backward, cudaStream_t s) {
    return interleaved ? rope_launch<T, VEC, NP, true, UF, UB>(p, a, backward, s)
                       : rope_launch<T, VEC, NP, false, UF, UB>(p, a, backward, s);
}

template <class T>
cudaError_t rope_dispatch(const norm_rope_plan& p, const RopeArgs& a, bool interleaved, bool backward, cudaStream_t s) {
    if constexpr (sizeof(T) == 4) {
        if (p.vec_elems == 4 && p.pairs == 1) return rope_style<T, 4, 1, 4, 2>(p, a, interleaved, backward, s);
        if (p.vec_elems == 4 && p.pairs == 2) return rope_style<T, 4, 2, 2, 1>(p, a, interleaved, backward, s);
    } else {
        if (p.vec_elems == 8 && p.pairs == 1) return rope_style<T, 8, 1, 4, 2>(p, a, interleaved, backward, s);
        if (p.vec_elems == 2 && p.pairs == 2) return rope_style<T, 2, 2, 4, 2>(p, a, interleaved, backward, s);
        if (p.vec_elems == 2 && p.pairs == 4) return rope_style<T, 2, 4, 2, 1>(p, a, interleaved, backward, s);
    }
    if (p.vec_elems == 1 && p.pairs == 4) return rope_style<T, 1, 4, 2, 2>(p, a, interleaved, backward, s);
    if (p.vec_elems == 1 && p.pairs == 8) return rope_style<T, 1, 8, 1, 1>(p, a, interleaved, backward, s);
    return cudaErrorInvalidValue;
}

}  // namespace libnorm
