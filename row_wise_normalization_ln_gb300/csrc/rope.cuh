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
// per pair. Each lane group of a warp has a token of its own and walks its
// heads: the token's angles and the weight stay in registers, and the next
// heads are in flight while one is reduced. (With a warp's groups on
// neighbouring heads of one token a task had a quarter of the heads for the
// same preparation, and groups stood idle where the heads ran out.) The sums
// of a head meet in butterflies over its lanes; nothing meets across warps
// until the backward's column sums.
//
// bf16, 16384 tokens of 32 + 8 heads of 128: forward 56.3 us, 6.0 TB/s, backward
// 87, 5.8 TB/s, bound by memory (with a group on a head each and all of a task's
// heads in registers 73 and 168). One token 1.67 us, f16 501 x 16 x 80 2.3, f32
// backward 1023 x 24 x 96 11.7: launches and latency.
#pragma once

#include "gn_kernels.cuh"
#include "rope_args.h"

namespace libnorm {

// GnVec, and accesses of four 16-bit values.
template <class T, int VEC>
struct RopeVec : GnVec<T, VEC> {};
template <class T>
struct RopeVec16x4 {
    using Raw = uint2;
    using P = typename Gn16<T>::Pair;
    static constexpr int H = 2;
    static __device__ __forceinline__ Raw zero() { return make_uint2(0, 0); }
    static __device__ __forceinline__ Raw load(const T* p) { return *reinterpret_cast<const uint2*>(p); }
    static __device__ __forceinline__ void store(T* p, const Raw& v) { *reinterpret_cast<uint2*>(p) = v; }
    static __device__ __forceinline__ float2 get(const Raw& r, int i) { return P::widen(i == 0 ? r.x : r.y); }
    static __device__ __forceinline__ void set(Raw& r, int i, float2 v) {
        if (i == 0) r.x = P::pack(v.x, v.y);
        else r.y = P::pack(v.x, v.y);
    }
};
template <>
struct RopeVec<__nv_bfloat16, 4> : RopeVec16x4<__nv_bfloat16> {};
template <>
struct RopeVec<__half, 4> : RopeVec16x4<__half> {};

// VEC values of an access as fp32 pairs (one value: the second of the pair is 0).
template <class T, int VEC>
struct RopeVals {
    using X = RopeVec<T, VEC>;
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

// How a token's rotation acts on a lane's values: access a becomes a * ca +
// mate(a) * sa, access b becomes b * cb + mate(b) * sb, where the mate of a
// value is its partner in the rotation. Values that do not rotate have c = 1
// and s = 0 (with a mate of their own all the same: 0 * infinity is not 0,
// which the kernels look after where it can happen). BACK: against the angle.
template <class T, int VEC, int NP, bool ILV, bool BACK>
struct RopeTurn {
    using V = RopeVals<T, VEC>;
    static constexpr int H = RopeVec<T, VEC>::H;
    static constexpr bool kInside = ILV && VEC > 1;  // pairs lie within an access
    float2 c[NP][kInside ? 2 * H : H], s[NP][2 * H];  // a's, then b's (not kInside: the same cosines)

    // From a token's table rows; vec: they are on 16-byte boundaries. Not live: no angle is read, nothing turns.
    __device__ __forceinline__ void set(const RopeLane<VEC, NP, ILV>& l, const float* cp, const float* sp, bool vec, bool live = true) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if constexpr (kInside) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool on = live && (h == 0 ? l.ra[j] : l.rb[j]);
                    const int at = h == 0 ? l.ca[j] : l.cb[j];
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float co = on ? cp[at + i] : 1.f, si = on ? sp[at + i] : 0.f;
                        c[j][h * H + i] = f2_splat(co);
                        s[j][h * H + i] = BACK ? make_float2(si, -si) : make_float2(-si, si);
                    }
                }
            } else {
                float tc[VEC], ts[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) tc[i] = 1.f, ts[i] = 0.f;
                if (live && l.ra[j]) {
                    if (VEC % 4 == 0 && vec) {
#pragma unroll
                        for (int i = 0; i < VEC / 4 * 4; i += 4) {
                            const float4 x = *reinterpret_cast<const float4*>(cp + l.ca[j] + i);
                            const float4 y = *reinterpret_cast<const float4*>(sp + l.ca[j] + i);
                            tc[i] = x.x, tc[i + 1] = x.y, tc[i + 2] = x.z, tc[i + 3] = x.w;
                            ts[i] = y.x, ts[i + 1] = y.y, ts[i + 2] = y.z, ts[i + 3] = y.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) tc[i] = cp[l.ca[j] + i], ts[i] = sp[l.ca[j] + i];
                    }
                }
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 si = VEC == 1 ? make_float2(ts[0], 0.f) : make_float2(ts[2 * i], ts[2 * i + (VEC > 1)]);
                    const float2 ni = make_float2(-si.x, -si.y);
                    c[j][i] = VEC == 1 ? make_float2(tc[0], 0.f) : make_float2(tc[2 * i], tc[2 * i + (VEC > 1)]);
                    s[j][i] = BACK ? si : ni;
                    s[j][H + i] = BACK ? ni : si;
                }
            }
        }
    }
    // The weight taken in: a * ca + mate(a) * sa is then the rotation of a * w.
    __device__ __forceinline__ float2 cos_of(int j, int i, bool b) const { return c[j][kInside && b ? H + i : i]; }
    __device__ __forceinline__ float2 sin_of(int j, int i, bool b) const { return s[j][b ? H + i : i]; }
    static __device__ __forceinline__ float2 mate(const V& a, const V& b, int i, bool of_b) {
        if constexpr (kInside) {
            const float2 v = of_b ? b.v[i] : a.v[i];
            return make_float2(v.y, v.x);
        }
        return of_b ? a.v[i] : b.v[i];
    }
};

// The rotation with the weight taken in, formed once per token: a head then
// takes two instructions per pair of values.
template <class T, int VEC, int NP, bool ILV>
struct RopeWeightedTurn {
    using R = RopeTurn<T, VEC, NP, ILV, false>;
    using V = RopeVals<T, VEC>;
    static constexpr int H = R::H;
    float2 ca[NP][H], sa[NP][H], cb[NP][H], sb[NP][H];
    __device__ __forceinline__ void set(const RopeLane<VEC, NP, ILV>& l, const V (&wa)[NP], const V (&wb)[NP], const float* cp,
                                        const float* sp, bool vec) {
        R t;
        t.set(l, cp, sp, vec);
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                ca[j][i] = __fmul2_rn(wa[j].v[i], t.cos_of(j, i, false));
                cb[j][i] = __fmul2_rn(wb[j].v[i], t.cos_of(j, i, true));
                sa[j][i] = __fmul2_rn(R::mate(wa[j], wb[j], i, false), t.sin_of(j, i, false));
                sb[j][i] = __fmul2_rn(R::mate(wa[j], wb[j], i, true), t.sin_of(j, i, true));
                // (a mate's infinite weight times the sine 0 is not 0)
                if (!l.ra[j]) sa[j][i] = make_float2(0.f, 0.f);
                if (!l.rb[j]) sb[j][i] = make_float2(0.f, 0.f);
            }
    }
    // SAFE: nothing of a mate reaches a value that does not rotate.
    template <bool SAFE>
    __device__ __forceinline__ void apply(const RopeLane<VEC, NP, ILV>& l, int j, const V& a, const V& b, float2 r2, V& oa,
                                          V& ob) const {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 va = __fmul2_rn(a.v[i], ca[j][i]), vb = __fmul2_rn(b.v[i], cb[j][i]);
            float2 ta = __ffma2_rn(R::mate(a, b, i, false), sa[j][i], va), tb = __ffma2_rn(R::mate(a, b, i, true), sb[j][i], vb);
            if (SAFE && !l.ra[j]) ta = va;
            if (SAFE && !l.rb[j]) tb = vb;
            oa.v[i] = __fmul2_rn(ta, r2);
            ob.v[i] = __fmul2_rn(tb, r2);
        }
    }
};

__device__ __forceinline__ int64_t rope_position(const RopeArgs& g, int t, int s) {
    if (g.pos_bytes == 8) return __ldg(static_cast<const long long*>(g.positions) + t);
    if (g.pos_bytes == 4) return __ldg(static_cast<const int*>(g.positions) + t);
    return s;
}

// Where a lane group's task lies: its token (on: there is one), the first
// head and how many.
struct RopeTask {
    int t, b, s, head, n;
    bool on;
    __device__ __forceinline__ RopeTask(const RopeArgs& g, const RopeSide& sd, int task) {
        const int block = quot(task, sd.by_chunks);
        head = (task - block * sd.chunks) * g.chunk_heads;
        n = min(sd.heads - head, g.chunk_heads);
        const int64_t at = (static_cast<int64_t>(block) << (5 - g.lanes_log)) + ((threadIdx.x & 31) >> g.lanes_log);
        on = at < g.T;
        t = on ? static_cast<int>(at) : 0;
        b = quot(t, g.by_S);
        s = t - b * g.S;
    }
};

template <class T>
__device__ __forceinline__ T* rope_at(const norm_heads& h, const RopeTask& k) {
    return static_cast<T*>(h.data) + k.b * h.batch + k.s * h.token + k.head * h.head;
}

// The weight of a lane's accesses, widened.
template <class T, int VEC, int NP, bool ILV>
struct RopeWeight {
    RopeVals<T, VEC> a[NP], b[NP];
    __device__ __forceinline__ RopeWeight(const RopeLane<VEC, NP, ILV>& l, const T* w) {
        using X = RopeVec<T, VEC>;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            a[j].widen(l.a[j] >= 0 ? X::load(w + l.a[j]) : X::zero());
            b[j].widen(l.b[j] >= 0 ? X::load(w + l.b[j]) : X::zero());
        }
    }
};

// Sums of N values over aligned groups of `lanes` lanes, side by side.
template <int N>
__device__ __forceinline__ void rope_sum(float (&v)[N], int lanes) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        if (off >= lanes) return;
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(kFullMask, v[n], off);
    }
}

// A CTA's side and a warp's first task and step.
struct RopeShare {
    bool second;
    int cta, first, step;
    __device__ __forceinline__ explicit RopeShare(const RopeArgs& g) {
        second = static_cast<int>(blockIdx.x) >= g.side[0].ctas;
        cta = static_cast<int>(blockIdx.x) - (second ? g.side[0].ctas : 0);
        const int warps = blockDim.x >> 5;
        first = cta * warps + static_cast<int>(threadIdx.x >> 5);
        step = g.side[second].ctas * warps;
    }
};

// Whether some access of the warp does not rotate: a mate's infinity must then
// be kept out of it.
template <int VEC, int NP, bool ILV>
__device__ __forceinline__ bool rope_mixed(const RopeLane<VEC, NP, ILV>& l) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < NP; ++j) any = any || (l.a[j] >= 0 && !l.ra[j]) || (l.b[j] >= 0 && !l.rb[j]);
    return __any_sync(kFullMask, any);
}

// What a token's position says.
struct RopePlace {
    bool pad, none;
    int64_t row;  // of the tables; 0 where there is no angle
    __device__ __forceinline__ RopePlace(const RopeArgs& g, const RopeTask& k) {
        const int64_t pos = rope_position(g, k.t, k.s);
        pad = pos < 0;
        none = pos >= g.P && g.R > 0;
        row = pad || none ? 0 : pos;
    }
};

// Zeros to the heads of a padding token.
template <class T, int VEC, int NP, bool ILV>
__device__ __forceinline__ void rope_zeros(const RopeLane<VEC, NP, ILV>& l, T* y, int64_t stride, int n) {
    using X = RopeVec<T, VEC>;
#pragma unroll 1
    for (int h = 0; h < n; ++h, y += stride) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (l.a[j] >= 0) X::store(y + l.a[j], X::zero());
            if (l.b[j] >= 0) X::store(y + l.b[j], X::zero());
        }
    }
}

// A warp's heads, task after task, with the next ones in flight: every lane
// copies its own accesses asynchronously into slots of shared memory of its
// own (no barrier, no registers while they travel), kRopeRing - 1 heads ahead and
// across tasks; a slot is refilled one head after it was read. Accesses of one
// 16-bit value, which asynchronous copies do not have, are loaded when their
// head's turn comes.
template <class T, int VEC, int NP, int N>  // N tensors: x, or x and dy
struct RopeStream {
    using X = RopeVec<T, VEC>;
    using Raw = typename X::Raw;
    static constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
    static constexpr bool kAsync = kBytes >= 4;
    static constexpr int kAccess = 32 * kBytes;         // a warp's copy of one access
    static constexpr int kUnit = N * NP * 2 * kAccess;  // of a head
    static constexpr int kWarp = kAsync ? kRopeRing * kUnit : 0;

    uint32_t ring;  // this lane's first slot
    int task, step, left = 0, sent = 0;
    bool on = false;
    const T* p[N];
    int64_t stride[N];

    template <class L>
    __device__ __forceinline__ RopeStream(const RopeArgs& g, const RopeSide& sd, const L& l, void* smem, int first, int step_)
        : task(first), step(step_) {
        ring = smem_addr(smem) + (threadIdx.x >> 5) * kWarp + (threadIdx.x & 31) * kBytes;
        stride[0] = sd.x.head;
        if constexpr (N == 2) stride[1] = sd.dy.head;
        if constexpr (kAsync) {
            // places that no copy goes to are zero throughout
#pragma unroll
            for (int i = 0; i < kRopeRing * N * NP; ++i) {
                if (l.a[i % NP] < 0) zero(ring + 2 * i * kAccess);
                if (l.b[i % NP] < 0) zero(ring + (2 * i + 1) * kAccess);
            }
#pragma unroll
            for (int i = 0; i < kRopeRing - 1; ++i) send(g, sd, l);
        }
    }
    static __device__ __forceinline__ void zero(uint32_t at) {
#pragma unroll
        for (int i = 0; i < kBytes; i += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + i), "r"(0) : "memory");
    }
    __device__ __forceinline__ void enter(const RopeArgs& g, const RopeSide& sd) {
        const RopeTask k(g, sd, task);
        p[0] = rope_at<const T>(sd.x, k);
        if constexpr (N == 2) p[1] = rope_at<const T>(sd.dy, k);
        left = k.n;
        on = k.on;
        task = task < sd.tasks - step ? task + step : sd.tasks;
    }
    // Issues the copies of the next head; a group of copies is committed even
    // when none is left.
    template <class L>
    __device__ __forceinline__ void send(const RopeArgs& g, const RopeSide& sd, const L& l) {
        if (left == 0 && task < sd.tasks) enter(g, sd);
        if (left > 0) {
            const uint32_t at = ring + (sent & (kRopeRing - 1)) * kUnit;
#pragma unroll
            for (int n = 0; n < N; ++n) {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    if (on && l.a[j] >= 0) copy_async<kBytes>(at + ((n * NP + j) * 2) * kAccess, p[n] + l.a[j]);
                    if (on && l.b[j] >= 0) copy_async<kBytes>(at + ((n * NP + j) * 2 + 1) * kAccess, p[n] + l.b[j]);
                }
                p[n] += stride[n];
            }
            --left;
        }
        ++sent;
        copy_async_commit();
    }
    static __device__ __forceinline__ Raw shared(uint32_t at) {
        Raw r;
        if constexpr (kBytes == 16)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
        else if constexpr (kBytes == 8)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
        else
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
        return r;
    }
    // The accesses of the next head. `live`: this lane's token has values, `all`: every lane's of the warp (the
    // backward's others get zeros; the forward chooses its outputs).
    template <class L>
    __device__ __forceinline__ void take(const RopeArgs& g, const RopeSide& sd, const L& l, bool live, bool all, Raw (&raw)[N][NP][2]) {
        if constexpr (kAsync) {
            copy_async_wait<kRopeRing - 2>();  // this head's copies have landed
            const uint32_t from = ring + ((sent + 1) & (kRopeRing - 1)) * kUnit;  // kRopeRing - 1 heads were sent beyond it
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    raw[n][j][0] = shared(from + ((n * NP + j) * 2) * kAccess);
                    raw[n][j][1] = shared(from + ((n * NP + j) * 2 + 1) * kAccess);
                }
            send(g, sd, l);  // into the slot read one head ago
            if (N == 2 && !all) {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        if (!live) raw[n][j][0] = raw[n][j][1] = X::zero();
            }
        } else {
            if (left == 0) enter(g, sd);
#pragma unroll
            for (int n = 0; n < N; ++n) {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    raw[n][j][0] = live && l.a[j] >= 0 ? X::load(p[n] + l.a[j]) : X::zero();
                    raw[n][j][1] = live && l.b[j] >= 0 ? X::load(p[n] + l.b[j]) : X::zero();
                }
                p[n] += stride[n];
            }
            --left;
        }
    }
};

// ------------------------------------------------------------ forward
// One head of the forward from its accesses. `on`: there is a token; `pad`: it
// is padding, whose zeros are chosen, not formed (0 times an infinite root,
// angle or weight is not 0), or there is none; what such lanes hold has no say
// in how the others' heads are turned.
template <class T, int VEC, int NP, bool ILV>
__device__ __forceinline__ void rope_fwd_head(const RopeArgs& g, const RopeLane<VEC, NP, ILV>& l,
                                              const RopeWeightedTurn<T, VEC, NP, ILV>& turn,
                                              const typename RopeVec<T, VEC>::Raw (&raw)[1][NP][2], T* y, bool on, bool pad,
                                              bool mixed, int lanes, float eps) {
    using X = RopeVec<T, VEC>;
    using V = RopeVals<T, VEC>;
    V va[NP], vb[NP];
    float2 qa = make_float2(0.f, 0.f), qb = qa;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        va[j].widen(raw[0][j][0]);
        vb[j].widen(raw[0][j][1]);
#pragma unroll
        for (int i = 0; i < X::H; ++i) {
            qa = __ffma2_rn(va[j].v[i], va[j].v[i], qa);
            qb = __ffma2_rn(vb[j].v[i], vb[j].v[i], qb);
        }
    }
    qa = __fadd2_rn(qa, qb);
    float ss[1] = {qa.x + qa.y};
    rope_sum(ss, lanes);
    const float2 r2 = f2_splat(rsqrtf(fmaf(ss[0], g.invD, eps)));
    V oa[NP], ob[NP];
    if (mixed && __any_sync(kFullMask, !pad && !isfinite(ss[0]))) {
#pragma unroll
        for (int j = 0; j < NP; ++j) turn.template apply<true>(l, j, va[j], vb[j], r2, oa[j], ob[j]);
    } else {
#pragma unroll
        for (int j = 0; j < NP; ++j) turn.template apply<false>(l, j, va[j], vb[j], r2, oa[j], ob[j]);
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        if (on && l.a[j] >= 0) X::store(y + l.a[j], pad ? X::zero() : oa[j].round());
        if (on && l.b[j] >= 0) X::store(y + l.b[j], pad ? X::zero() : ob[j].round());
    }
}

// Persistent, over the stream of heads.
template <class T, int VEC, int NP, bool ILV>
__global__ void __launch_bounds__(kRopeMaxWarps * 32) rope_fwd(const __grid_constant__ RopeArgs g) {
    extern __shared__ __align__(16) char smem[];
    grid_release();
    const RopeShare share(g);
    const RopeSide& sd = g.side[share.second];
    const int lanes = 1 << g.lanes_log;
    const RopeLane<VEC, NP, ILV> l(g, threadIdx.x & (lanes - 1));
    const bool mixed = rope_mixed(l);
    grid_wait();
    RopeStream<T, VEC, NP, 1> in(g, sd, l, smem, share.first, share.step);
    const RopeWeight<T, VEC, NP, ILV> w(l, static_cast<const T*>(sd.w));
    for (int task = share.first; task < sd.tasks; task = task < sd.tasks - share.step ? task + share.step : sd.tasks) {
        const RopeTask k(g, sd, task);
        const RopePlace at(g, k);
        RopeWeightedTurn<T, VEC, NP, ILV> turn;
        turn.set(l, w.a, w.b, g.cos + at.row * g.table_pitch, g.sin + at.row * g.table_pitch, g.vec_table != 0);
        const bool live = k.on && !at.pad, all = __all_sync(kFullMask, live);
        const float eps = at.none ? __int_as_float(0x7fffffff) : g.eps;  // no angle: NaN
        T* y = rope_at<T>(sd.y, k);
        for (int h = 0; h < k.n; ++h, y += sd.y.head) {
            typename RopeVec<T, VEC>::Raw raw[1][NP][2];
            in.take(g, sd, l, live, all, raw);
            rope_fwd_head<T, VEC, NP, ILV>(g, l, turn, raw, y, k.on, !all && !live, mixed, lanes, eps);
        }
    }
}

// For few heads: a warp has one task and its heads come straight into
// registers, the first before its position is known. No shared memory to go
// through: one token of 36 heads 1.7 us instead of 2.2, 501 x 16 heads of 80
// 2.3 instead of 2.7 (but 16384 x 40 heads of 128 66 instead of 56: a load per
// lane and access in flight is too little for the latency under load).
template <class T, int VEC, int NP, bool ILV>
__global__ void __launch_bounds__(kRopeMaxWarps * 32) rope_fwd_few(const __grid_constant__ RopeArgs g) {
    using X = RopeVec<T, VEC>;
    constexpr int DEPTH = 2;
    grid_release();
    const RopeShare share(g);
    const RopeSide& sd = g.side[share.second];
    const int lanes = 1 << g.lanes_log;
    const RopeLane<VEC, NP, ILV> l(g, threadIdx.x & (lanes - 1));
    const bool mixed = rope_mixed(l);
    grid_wait();
    if (share.first >= sd.tasks) return;  // (a whole warp)
    const RopeTask k(g, sd, share.first);
    const T* x = rope_at<const T>(sd.x, k);
    typename X::Raw raw[DEPTH][1][NP][2];
    const auto load = [&](int d, int h) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            raw[d][0][j][0] = k.on && h < k.n && l.a[j] >= 0 ? X::load(x + l.a[j]) : X::zero();
            raw[d][0][j][1] = k.on && h < k.n && l.b[j] >= 0 ? X::load(x + l.b[j]) : X::zero();
        }
        x += sd.x.head;
    };
    const RopePlace at(g, k);
    load(0, 0);
    load(1, 1);
    RopeWeightedTurn<T, VEC, NP, ILV> turn;
    {
        const RopeWeight<T, VEC, NP, ILV> w(l, static_cast<const T*>(sd.w));
        turn.set(l, w.a, w.b, g.cos + at.row * g.table_pitch, g.sin + at.row * g.table_pitch, g.vec_table != 0);
    }
    const float eps = at.none ? __int_as_float(0x7fffffff) : g.eps;
    const bool some = __any_sync(kFullMask, at.pad);
    T* y = rope_at<T>(sd.y, k);
    for (int h = 0; h < k.n; h += DEPTH)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (h + d < k.n) {
                typename X::Raw now[1][NP][2];
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) now[0][j][i] = raw[d][0][j][i];
                load(d, h + d + DEPTH);
                rope_fwd_head<T, VEC, NP, ILV>(g, l, turn, now, y, k.on, some && at.pad, mixed, lanes, eps);
                y += sd.y.head;
            }
}

// ------------------------------------------------------------ backward
// Persistent: a CTA keeps one side's dw in registers over its tasks. A chain
// of additions is at most kRopeChain heads long; the sums of the chains are
// added in this lane's slots of shared memory.
constexpr int kRopeChain = 64;

template <class T, int VEC, int NP, bool ILV>
__global__ void __launch_bounds__(kRopeMaxWarps * 32) rope_bwd(const __grid_constant__ RopeArgs g) {
    using X = RopeVec<T, VEC>;
    using V = RopeVals<T, VEC>;
    using R = RopeTurn<T, VEC, NP, ILV, true>;
    constexpr int H = X::H;
    extern __shared__ __align__(16) char smem[];
    float2* sums = reinterpret_cast<float2*>(smem);  // [NP * 2 * H][threads], before the stream
    grid_release();
    const RopeShare share(g);
    const RopeSide& sd = g.side[share.second];
    const int lanes = 1 << g.lanes_log;
    const RopeLane<VEC, NP, ILV> l(g, threadIdx.x & (lanes - 1));
    const bool mixed = rope_mixed(l);
    V da[NP], db[NP];  // this lane's share of dw
    float2* mine_sums = sums + threadIdx.x;
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            da[j].v[i] = db[j].v[i] = make_float2(0.f, 0.f);
            mine_sums[((j * 2) * H + i) * blockDim.x] = mine_sums[((j * 2 + 1) * H + i) * blockDim.x] = make_float2(0.f, 0.f);
        }
    int chain = 0;
    bool padded = false;  // this lane met padding
    const auto fold = [&] {
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                float2& fa = mine_sums[((j * 2) * H + i) * blockDim.x];
                float2& fb = mine_sums[((j * 2 + 1) * H + i) * blockDim.x];
                fa = __fadd2_rn(fa, da[j].v[i]);
                fb = __fadd2_rn(fb, db[j].v[i]);
                da[j].v[i] = db[j].v[i] = make_float2(0.f, 0.f);
            }
        chain = 0;
    };
    grid_wait();
    RopeStream<T, VEC, NP, 2> in(g, sd, l, smem + NP * 2 * H * sizeof(float2) * blockDim.x, share.first, share.step);
    const RopeWeight<T, VEC, NP, ILV> w(l, static_cast<const T*>(sd.w));
    for (int task = share.first; task < sd.tasks; task = task < sd.tasks - share.step ? task + share.step : sd.tasks) {
        const RopeTask k(g, sd, task);
        const RopePlace at(g, k);
        const bool live = k.on && !at.pad, all = __all_sync(kFullMask, live);
        R turn;
        turn.set(l, g.cos + at.row * g.table_pitch, g.sin + at.row * g.table_pitch, g.vec_table != 0, live);
        // A lane whose token has no values works on zeros, which have to stay
        // zeros on their way to dw: its root is that of 1, finite for eps = 0 too.
        const float eps = !live ? 1.f : at.none ? __int_as_float(0x7fffffff) : g.eps;
        padded = padded || at.pad;
        T* dx = rope_at<T>(sd.y, k);
        for (int h = 0; h < k.n; ++h) {
            typename X::Raw raw[2][NP][2];
            in.take(g, sd, l, live, all, raw);
            V va[NP], vb[NP], ta[NP], tb[NP], za[NP], zb[NP];  // x, dy, dz
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                va[j].widen(raw[0][j][0]);
                vb[j].widen(raw[0][j][1]);
                ta[j].widen(raw[1][j][0]);
                tb[j].widen(raw[1][j][1]);
            }
            float s2[2];
            const auto sums_of = [&](auto safe) {
                float2 ssa = make_float2(0.f, 0.f), ssb = ssa, sga = ssa, sgb = ssa;
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        za[j].v[i] = __ffma2_rn(ta[j].v[i], turn.cos_of(j, i, false),
                                                __fmul2_rn(R::mate(ta[j], tb[j], i, false), turn.sin_of(j, i, false)));
                        zb[j].v[i] = __ffma2_rn(tb[j].v[i], turn.cos_of(j, i, true),
                                                __fmul2_rn(R::mate(ta[j], tb[j], i, true), turn.sin_of(j, i, true)));
                        if (decltype(safe)::value && !l.ra[j]) za[j].v[i] = ta[j].v[i];
                        if (decltype(safe)::value && !l.rb[j]) zb[j].v[i] = tb[j].v[i];
                        ssa = __ffma2_rn(va[j].v[i], va[j].v[i], ssa);
                        ssb = __ffma2_rn(vb[j].v[i], vb[j].v[i], ssb);
                        sga = __ffma2_rn(__fmul2_rn(za[j].v[i], w.a[j].v[i]), va[j].v[i], sga);
                        sgb = __ffma2_rn(__fmul2_rn(zb[j].v[i], w.b[j].v[i]), vb[j].v[i], sgb);
                    }
                ssa = __fadd2_rn(ssa, ssb);
                sga = __fadd2_rn(sga, sgb);
                s2[0] = ssa.x + ssa.y;
                s2[1] = sga.x + sga.y;
                rope_sum(s2, lanes);
            };
            sums_of(std::false_type{});
            if (mixed && __any_sync(kFullMask, !isfinite(s2[0]) || !isfinite(s2[1]))) sums_of(std::true_type{});
            const float r = rsqrtf(fmaf(s2[0], g.invD, eps));
            // dx = r (g - x r (r mean(g x)))
            const float2 r2 = f2_splat(r), m2 = f2_splat(-(r * (s2[1] * g.invD)) * r);
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                V oa, ob;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    oa.v[i] = __fmul2_rn(__ffma2_rn(va[j].v[i], m2, __fmul2_rn(za[j].v[i], w.a[j].v[i])), r2);
                    ob.v[i] = __fmul2_rn(__ffma2_rn(vb[j].v[i], m2, __fmul2_rn(zb[j].v[i], w.b[j].v[i])), r2);
                    da[j].v[i] = __ffma2_rn(__fmul2_rn(va[j].v[i], r2), za[j].v[i], da[j].v[i]);
                    db[j].v[i] = __ffma2_rn(__fmul2_rn(vb[j].v[i], r2), zb[j].v[i], db[j].v[i]);
                }
                if (live && l.a[j] >= 0) X::store(dx + l.a[j], oa.round());
                if (live && l.b[j] >= 0) X::store(dx + l.b[j], ob.round());
            }
            dx += sd.y.head;
            if (++chain == kRopeChain) fold();
        }
    }
    fold();
    // Padding's zeros, behind everything: in the loop over the heads they cost a
    // choice per store (16384 tokens 89.8 us instead of 86.9), behind a token's
    // heads registers, and with them CTAs (f32 715 x 64 heads of 128 17.5 instead
    // of 13.4).
    if (padded)
        for (int task = share.first; task < sd.tasks; task = task < sd.tasks - share.step ? task + share.step : sd.tasks) {
            const RopeTask k(g, sd, task);
            if (k.on && rope_position(g, k.t, k.s) < 0) rope_zeros<T, VEC, NP, ILV>(l, rope_at<T>(sd.y, k), sd.y.head, k.n);
        }
    __syncthreads();
    // A column's terms lie with the lanes of its place in every group of
    // every warp: added in that order, each column by one thread.
    float* part = sd.part + int64_t(share.cta) * g.D;
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
// CTAs of a kernel that fit on the device at once, asked once per kernel,
// size and device.
inline cudaError_t rope_resident(const void* fn, int threads, size_t smem, int64_t* out) try {
    static std::mutex mu;
    static std::map<std::tuple<const void*, int, int>, int64_t> cache;  // (smem follows from the kernel and threads)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    int64_t& n = cache[{fn, threads, dev}];
    if (n == 0) {
        int per = 0, sms = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, threads, smem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        n = int64_t(per) * sms;
    }
    *out = n;
    return n > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
} catch (...) {  // (no exception leaves a C entry point)
    return cudaErrorMemoryAllocation;
}

template <class T, int VEC, int NP, bool ILV>
cudaError_t rope_launch(const norm_rope_plan& p, RopeArgs& a, bool backward, cudaStream_t s) {
    const void* fn = backward ? reinterpret_cast<const void*>(rope_bwd<T, VEC, NP, ILV>)
                     : p.few  ? reinterpret_cast<const void*>(rope_fwd_few<T, VEC, NP, ILV>)
                              : reinterpret_cast<const void*>(rope_fwd<T, VEC, NP, ILV>);
    const int threads = p.warps * 32;
    const size_t smem = p.few ? 0 : static_cast<size_t>(rope_smem_bytes(VEC, sizeof(T), NP, p.warps, backward));
    if (smem > 16 * 1024) {
        const cudaError_t e = gn_opt_in(fn);
        if (e != cudaSuccess) return e;
    }
    if (!p.few) {
        int64_t most = 0;
        const cudaError_t e = rope_resident(fn, threads, smem, &most);
        if (e != cudaSuccess) return e;
        rope_share(&a, std::min(p.ctas, most));
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
    void* args[] = {&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <class T, int VEC, int NP>
cudaError_t rope_style(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s) {
    return interleaved ? rope_launch<T, VEC, NP, true>(p, a, backward, s) : rope_launch<T, VEC, NP, false>(p, a, backward, s);
}

template <class T>
cudaError_t rope_dispatch(const norm_rope_plan& p, RopeArgs& a, bool interleaved, bool backward, cudaStream_t s) {
    if (p.vec_elems == 4 && p.pairs == 1) return rope_style<T, 4, 1>(p, a, interleaved, backward, s);
    if (p.vec_elems == 4 && p.pairs == 2) return rope_style<T, 4, 2>(p, a, interleaved, backward, s);
    if constexpr (sizeof(T) == 2) {
        if (p.vec_elems == 8 && p.pairs == 1) return rope_style<T, 8, 1>(p, a, interleaved, backward, s);
        if (p.vec_elems == 2 && p.pairs == 2) return rope_style<T, 2, 2>(p, a, interleaved, backward, s);
        if (p.vec_elems == 2 && p.pairs == 4) return rope_style<T, 2, 4>(p, a, interleaved, backward, s);
    }
    if (p.vec_elems == 1 && p.pairs == 4) return rope_style<T, 1, 4>(p, a, interleaved, backward, s);
    if (p.vec_elems == 1 && p.pairs == 8) return rope_style<T, 1, 8>(p, a, interleaved, backward, s);
    return cudaErrorInvalidValue;
}

}  // namespace libnorm
