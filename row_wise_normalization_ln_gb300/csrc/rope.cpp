// Head norm + rotation entry points of the C ABI: argument checks, the launch
// planner and dispatch. Every argument error is caught here, before any CUDA
// call.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime_api.h>

#include "norm_args.h"
#include "rope_args.h"

namespace {

using libnorm::RopeArgs;
using libnorm::RopeSide;
using libnorm::kRopeMaxD;
using libnorm::kRopeMaxWarps;

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxHeads = int64_t(1) << 20;
constexpr int64_t kMaxPitch = int64_t(1) << 40;
constexpr int kCtasPerSm = 8;  // at most; a launch takes as many as fit
constexpr int kFewHeads = 64;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int elem_size(norm_dtype d) { return d == NORM_F32 ? 4 : 2; }
bool on(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

struct Shape {
    int64_t B, S, T, D, R, heads[2];
    bool interleaved, bwd;
    norm_dtype dtype;
};

norm_status check_counts(const Shape& s) {
    if (s.dtype != NORM_F32 && s.dtype != NORM_BF16 && s.dtype != NORM_F16) return NORM_ERR_DTYPE;
    if (s.D < 1 || s.D > kRopeMaxD || s.R < 0 || s.R > s.D || s.R % 2 != 0) return NORM_ERR_ARG;
    if (s.T < 0 || s.T > kMaxTokens) return NORM_ERR_ARG;
    for (int64_t h : s.heads) {
        if (h < 0 || h >= kMaxHeads) return NORM_ERR_ARG;
        if (h > 0 && s.T > (int64_t(1) << 62) / (h * s.D)) return NORM_ERR_ARG;
    }
    return NORM_OK;
}

// Whether `n` values from an address on a boundary of n values start aligned:
// heads are n values wide and, in the rotation, so are its halves or pairs.
bool width_ok(const Shape& s, int vec) {
    if (vec == 1) return true;
    return s.D % vec == 0 && (s.interleaved ? s.R : s.R / 2) % vec == 0;
}

// Pitches of a dimension of one element are not used.
norm_heads settled(norm_heads t, const Shape& s, int64_t heads) {
    if (s.B <= 1) t.batch = 0;
    if (s.S <= 1) t.token = 0;
    if (heads <= 1) t.head = 0;
    return t;
}

bool pitches_ok(const norm_heads& t) {
    for (int64_t p : {t.batch, t.token, t.head})
        if (p >= kMaxPitch || p <= -kMaxPitch) return false;
    return true;
}

bool tensor_vec(const norm_heads& t, int64_t bytes, int es) {
    return on(t.data, bytes) && t.batch * es % bytes == 0 && t.token * es % bytes == 0 && t.head * es % bytes == 0;
}

// Pairs of accesses a head has, and how many of them rotate.
void count_pairs(const Shape& s, int vec, int64_t* all, int64_t* rot) {
    if (s.interleaved && vec > 1) {
        *all = ceil_div(s.D / vec, 2);
        *rot = 0;
        return;
    }
    *rot = s.R / 2 / vec;
    *all = *rot + ceil_div((s.D - s.R) / vec, 2);
}

bool vec_known(int vec, norm_dtype dtype) { return vec == 1 || vec == 16 / elem_size(dtype) || ((vec == 2 || vec == 4) && dtype != NORM_F32); }

// The instances there are: (access width, pairs per lane).
bool pairs_known(int vec, int pairs, norm_dtype dtype) {
    if (vec == 1) return pairs == 4 || pairs == 8;
    if (vec == 2) return pairs == 2 || pairs == 4;
    return pairs == 1 || (pairs == 2 && vec == 4);
}

norm_status make_plan(const Shape& s, int vec, int num_sms, norm_rope_plan* p) {
    std::memset(p, 0, sizeof *p);
    int64_t all, rot;
    count_pairs(s, vec, &all, &rot);
    p->vec_elems = vec;
    for (int pairs : {1, 2, 4, 8}) {
        if (!pairs_known(vec, pairs, s.dtype) || all > int64_t(pairs) * 32) continue;
        p->pairs = pairs;
        int lanes = 1;
        while (int64_t(lanes) * pairs < all) lanes *= 2;
        p->lanes = lanes;
        break;
    }
    if (p->pairs == 0) return NORM_ERR_ARG;
    const int64_t blocks = ceil_div(s.T, 32 / p->lanes), most = std::max<int64_t>(1, std::max(s.heads[0], s.heads[1]));
    const int64_t total = blocks * (s.heads[0] + s.heads[1]);  // warps' heads
    p->warps = 4;
    p->few = !s.bwd && total <= int64_t(num_sms) * kFewHeads;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(p->few ? 2 : 8, total / (int64_t(num_sms) * (p->few ? 4 : 16))));
    p->heads = static_cast<int32_t>(ceil_div(most, ceil_div(most, want)));
    p->ctas = std::max<int64_t>(2, std::min<int64_t>(int64_t(num_sms) * kCtasPerSm, ceil_div(total, p->heads * p->warps)));
    return NORM_OK;
}

// Everything a launch needs beyond the tensors; NORM_ERR_PLAN if the plan
// does not fit the call.
norm_status derive(const norm_rope_plan& p, const Shape& s, int vec, RopeArgs* a) {
    if (!vec_known(p.vec_elems, s.dtype) || !pairs_known(p.vec_elems, p.pairs, s.dtype)) return NORM_ERR_PLAN;
    if (p.vec_elems > vec || !width_ok(s, p.vec_elems) || (p.few != 0 && (p.few != 1 || s.bwd))) return NORM_ERR_PLAN;
    if (p.lanes < 1 || p.lanes > 32 || (p.lanes & (p.lanes - 1)) != 0) return NORM_ERR_PLAN;
    if (p.heads < 1 || p.warps < 1 || p.warps > kRopeMaxWarps) return NORM_ERR_PLAN;
    int64_t all, rot;
    count_pairs(s, p.vec_elems, &all, &rot);
    if (all > int64_t(p.pairs) * p.lanes) return NORM_ERR_PLAN;
    if (p.ctas < 2 || p.ctas > (1 << 20)) return NORM_ERR_PLAN;
    if (!p.few && libnorm::rope_smem_bytes(p.vec_elems, elem_size(s.dtype), p.pairs, p.warps, s.bwd) > libnorm::kRopeMaxSmem) return NORM_ERR_PLAN;
    a->lanes_log = 0;
    while ((1 << a->lanes_log) < p.lanes) ++a->lanes_log;
    a->npairs = static_cast<int32_t>(all);
    a->rot_pairs = static_cast<int32_t>(rot);
    a->D = static_cast<int32_t>(s.D);
    a->R = static_cast<int32_t>(s.R);
    a->invD = 1.f / static_cast<float>(s.D);
    a->T = static_cast<int32_t>(s.T);
    const int64_t blocks = ceil_div(s.T, 32 / p.lanes);
    int64_t chunk = p.heads;
    // tasks are counted in 31 bits: fewer, larger ones where they would not fit
    while (ceil_div(std::max(s.heads[0], s.heads[1]), chunk) * blocks > kMaxTokens) chunk *= 2;
    a->chunk_heads = static_cast<int32_t>(chunk);
    for (int i = 0; i < 2; ++i) {
        RopeSide& d = a->side[i];
        d.heads = static_cast<int32_t>(s.heads[i]);
        d.chunks = static_cast<int32_t>(std::max<int64_t>(1, ceil_div(s.heads[i], chunk)));
        d.by_chunks = libnorm::fast_div(d.chunks);
        d.tasks = d.heads > 0 ? static_cast<int32_t>(blocks * d.chunks) : 0;
        d.ctas = static_cast<int32_t>(ceil_div(d.tasks, p.warps));
    }
    // a warp without a loop counts its task in 31 bits, the last CTA's idle warps too
    for (const RopeSide& d : a->side)
        if (p.few && int64_t(d.ctas) * p.warps > kMaxTokens + 1) return NORM_ERR_PLAN;
    return int64_t(a->side[0].ctas) + a->side[1].ctas <= kMaxTokens ? NORM_OK : NORM_ERR_PLAN;
}

// A partial row of D values per CTA, of which there are at most the plan's and
// one per head.
int64_t workspace_bytes(int64_t ctas, int64_t tokens, int64_t heads, int64_t D) {
    const __int128 all = static_cast<__int128>(tokens) * heads;
    return (all < ctas ? static_cast<int64_t>(all) : ctas) * D * 4;
}

norm_status done(cudaError_t e) {
    if (e == cudaSuccess) return NORM_OK;
    libnorm::note_cuda_error(static_cast<int>(e));
    return NORM_ERR_CUDA;
}

// The current device's SM count, read once per device.
norm_status device_sms(int* sms) {
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return done(e);
    int n = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return done(e);
        if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return NORM_OK;
}

// The call's checks, plan and argument block but for the workspace.
norm_status settle(const norm_rope_side* const (&in)[2], const norm_rope_angles* angles, float eps, Shape* s,
                   const norm_rope_plan* plan, norm_rope_plan* p, RopeArgs* a) {
    if (!in[0] || !in[1] || !angles) return NORM_ERR_ARG;
    if (s->B < 0 || s->S < 0 || (s->S > 0 && s->B > kMaxTokens / s->S)) return NORM_ERR_ARG;
    s->T = s->B * s->S;
    s->R = angles->R;
    s->interleaved = angles->interleaved != 0;
    for (int i = 0; i < 2; ++i) s->heads[i] = in[i]->heads;
    norm_status st = check_counts(*s);
    if (st != NORM_OK) return st;
    if (!std::isfinite(eps) || eps < 0.f || angles->reserved != 0 || angles->P < 0) return NORM_ERR_ARG;
    const int es = elem_size(s->dtype);
    for (int i = 0; i < 2; ++i)
        if (s->bwd && s->heads[i] > 0 && (!in[i]->dw || !on(in[i]->dw, 4))) return NORM_ERR_ARG;
    const bool work = s->T > 0 && (s->heads[0] > 0 || s->heads[1] > 0);
    int vec = 16 / es;
    const auto narrow = [&](auto ok) {
        while (vec > 1 && !ok(vec)) vec = es == 4 || vec == 2 ? 1 : vec / 2;
    };
    if (work) {
        if (s->R > 0) {
            if (!angles->cos || !angles->sin || !on(angles->cos, 4) || !on(angles->sin, 4)) return NORM_ERR_ARG;
            if (angles->P < 1 || angles->table_pitch < s->R / 2 || angles->table_pitch >= kMaxPitch) return NORM_ERR_ARG;
        }
        if (angles->positions) {
            if (angles->position_bytes != 4 && angles->position_bytes != 8) return NORM_ERR_ARG;
            if (!on(angles->positions, angles->position_bytes)) return NORM_ERR_ARG;
        }
        narrow([&](int v) { return width_ok(*s, v); });
        for (int i = 0; i < 2; ++i) {
            if (s->heads[i] == 0) continue;
            RopeSide& d = a->side[i];
            d.x = settled(in[i]->x, *s, s->heads[i]);
            d.y = settled(in[i]->y, *s, s->heads[i]);
            d.dy = s->bwd ? settled(in[i]->dy, *s, s->heads[i]) : d.x;
            d.w = in[i]->w;
            d.dw = in[i]->dw;
            if (!d.w || !on(d.w, es)) return NORM_ERR_ARG;
            for (const norm_heads* t : {&d.x, &d.dy, &d.y})
                if (!t->data || !on(t->data, es) || !pitches_ok(*t)) return NORM_ERR_ARG;
            // in place: the same elements
            for (const norm_heads* t : {&d.x, &d.dy})
                if (t->data == d.y.data && (t->batch != d.y.batch || t->token != d.y.token || t->head != d.y.head)) return NORM_ERR_ARG;
            narrow([&](int v) {
                const int64_t bytes = int64_t(v) * es;
                return on(d.w, bytes) && tensor_vec(d.x, bytes, es) && tensor_vec(d.dy, bytes, es) && tensor_vec(d.y, bytes, es);
            });
        }
        a->cos = angles->cos;
        a->sin = angles->sin;
        a->table_pitch = angles->table_pitch;
        a->P = angles->P;
        a->positions = angles->positions;
        a->pos_bytes = angles->positions ? angles->position_bytes : 0;
        a->vec_table = on(angles->cos, 16) && on(angles->sin, 16) && angles->table_pitch % 4 == 0 && s->R % 8 == 0;
        a->S = static_cast<int32_t>(s->S);
        a->by_S = libnorm::fast_div(s->S);
        a->eps = eps;
    } else {
        for (int i = 0; i < 2; ++i) a->side[i].dw = in[i]->dw;
        narrow([&](int v) { return width_ok(*s, v); });
    }
    if (plan) {
        *p = *plan;
    } else if (work) {
        int sms = 0;
        st = device_sms(&sms);
        if (st != NORM_OK) return st;
        st = make_plan(*s, vec, sms, p);
        if (st != NORM_OK) return st;
    } else {
        st = make_plan(*s, vec, 1, p);
        if (st != NORM_OK) return st;
    }
    return derive(*p, *s, vec, a);
}

cudaError_t launch(const norm_rope_plan& p, RopeArgs& a, const Shape& s, cudaStream_t stream) {
    switch (s.dtype) {
        case NORM_F32: return libnorm::launch_rope_f32(p, a, s.interleaved, s.bwd, stream);
        case NORM_BF16: return libnorm::launch_rope_bf16(p, a, s.interleaved, s.bwd, stream);
        default: return libnorm::launch_rope_f16(p, a, s.interleaved, s.bwd, stream);
    }
}

}  // namespace

extern "C" {

norm_status rms_fwd_rope_planned(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles,
                                 int64_t B, int64_t S, int64_t D, float eps, norm_dtype dtype, cudaStream_t stream,
                                 const norm_rope_plan* plan) {
    Shape s{B, S, 0, D, 0, {0, 0}, false, false, dtype};
    norm_rope_plan p;
    RopeArgs a{};
    const norm_rope_side* const in[2] = {q, k};
    const norm_status st = settle(in, angles, eps, &s, plan, &p, &a);
    if (st != NORM_OK || a.side[0].tasks + int64_t(a.side[1].tasks) == 0) return st;
    return done(launch(p, a, s, stream));
}

norm_status rms_fwd_rope(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles, int64_t B,
                         int64_t S, int64_t D, float eps, norm_dtype dtype, cudaStream_t stream) {
    return rms_fwd_rope_planned(q, k, angles, B, S, D, eps, dtype, stream, nullptr);
}

norm_status rms_bwd_rope_planned(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles,
                                 void* workspace, size_t workspace_size, int64_t B, int64_t S, int64_t D, float eps,
                                 norm_dtype dtype, cudaStream_t stream, const norm_rope_plan* plan) {
    Shape s{B, S, 0, D, 0, {0, 0}, false, true, dtype};
    norm_rope_plan p;
    RopeArgs a{};
    const norm_rope_side* const in[2] = {q, k};
    const norm_status st = settle(in, angles, eps, &s, plan, &p, &a);
    if (st != NORM_OK || (s.heads[0] == 0 && s.heads[1] == 0)) return st;
    if (s.T > 0) {
        const int64_t need = workspace_bytes(p.ctas, s.T, s.heads[0] + s.heads[1], D);
        if (need > 0 && (!workspace || !on(workspace, 16) || workspace_size < static_cast<size_t>(need))) return NORM_ERR_ARG;
        a.side[0].part = static_cast<float*>(workspace);
        const cudaError_t e = launch(p, a, s, stream);
        if (e != cudaSuccess) return done(e);
    }
    return done(libnorm::launch_rope_colsum(a, stream));
}

norm_status rms_bwd_rope(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles,
                         void* workspace, size_t workspace_size, int64_t B, int64_t S, int64_t D, float eps,
                         norm_dtype dtype, cudaStream_t stream) {
    return rms_bwd_rope_planned(q, k, angles, workspace, workspace_size, B, S, D, eps, dtype, stream, nullptr);
}

norm_status rope_make_plan(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t D, int64_t R, int interleaved,
                           norm_dtype dtype, int backward, int vec_elems, int num_sms, norm_rope_plan* plan) {
    const Shape s{1, tokens, tokens, D, R, {q_heads, k_heads}, interleaved != 0, backward != 0, dtype};
    const norm_status st = check_counts(s);
    if (st != NORM_OK) return st;
    if (!plan || num_sms < 1 || !vec_known(vec_elems, dtype) || !width_ok(s, vec_elems)) return NORM_ERR_ARG;
    return make_plan(s, vec_elems, num_sms, plan);
}

norm_status rope_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t D, int num_sms,
                                 const norm_rope_plan* plan, size_t* bytes) {
    const Shape s{1, tokens, tokens, D, 0, {q_heads, k_heads}, false, true, NORM_F32};
    const norm_status st = check_counts(s);
    if (st != NORM_OK) return st;
    if (!bytes || (!plan && num_sms < 1) || (plan && plan->ctas < 0)) return NORM_ERR_ARG;
    *bytes = 0;
    if (tokens == 0) return NORM_OK;
    *bytes = static_cast<size_t>(workspace_bytes(plan ? plan->ctas : int64_t(num_sms) * kCtasPerSm, tokens, q_heads + k_heads, D));
    return NORM_OK;
}

}  // extern "C"
