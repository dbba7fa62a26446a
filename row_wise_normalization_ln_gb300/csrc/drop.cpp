// Dropout + add + norm entry points of the C ABI: argument checks, the launch
// planner and dispatch. Every argument error is caught here, before any CUDA
// call.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime_api.h>

#include "drop_args.h"
#include "norm_args.h"

namespace {

using libnorm::DropArgs;
using libnorm::kDropMaxSmem;
using libnorm::kDropMaxStages;
using libnorm::kDropMaxThreads;

constexpr int64_t kMaxN = 65536;
constexpr int64_t kMaxElems = 32768;  // of rows that are not 16-byte aligned
constexpr int64_t kMaxGrid = int64_t(1) << 20;
constexpr int kMaxCluster = 8;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
int elem_size(norm_dtype d) { return d == NORM_F32 ? 4 : 2; }
bool on(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

struct Shape {
    int64_t M, N;
    norm_dtype dtype;
    bool ln, bwd;
    int es() const { return elem_size(dtype); }
};

norm_status check_shape(const Shape& s) {
    if (s.dtype != NORM_F32 && s.dtype != NORM_BF16 && s.dtype != NORM_F16) return NORM_ERR_DTYPE;
    if (s.M < 0 || s.N < 1 || s.N > kMaxN || s.M > (int64_t(1) << 62) / s.N) return NORM_ERR_ARG;
    return NORM_OK;
}

bool known(const Shape& s, bool group, int vec, int per, int rows) { return libnorm::drop_known(s.bwd, group, vec, s.es(), per, rows); }

// Threads that share a row of a CTA.
int team_of(const norm_plan& p) { return p.mapping == NORM_MAP_CTA && p.group > 0 ? p.group : p.threads; }

int teams_of(const norm_plan& p) { return p.threads / (p.mapping == NORM_MAP_GROUP ? p.group : team_of(p)); }

int stat_bytes(const Shape& s, const norm_plan& p) {
    return libnorm::drop_stat_bytes(s.ln, s.bwd, p.vec_elems, p.mapping == NORM_MAP_GROUP ? p.group : 0, p.rounds);
}

int64_t smem_bytes(const Shape& s, const norm_plan& p, int stages) {
    return libnorm::drop_ring_bytes(p.vec_elems, s.es(), p.per_thread, p.threads, p.rounds, stages, s.bwd ? 3 : 2, stat_bytes(s, p)) +
           libnorm::drop_words_bytes(p.vec_elems, p.per_thread, p.threads) +
           (s.bwd ? 0 : libnorm::drop_param_bytes(s.ln, p.vec_elems, p.per_thread, p.threads)) +
           (s.bwd && teams_of(p) > 1 ? libnorm::drop_sums_bytes(s.ln, p.vec_elems, p.per_thread, p.threads) : 0);
}

// Vectors, or pairs of elements, that a row touches.
int64_t accesses(const Shape& s, int vec) { return vec == 1 ? ceil_div(s.N, 2) : libnorm::drop_vectors(s.N, vec); }

// Which threads share a row, from sweeps of the instances (bf16 unless said;
// the other side in brackets):
// - Few vectors a row: lanes of a warp, two accesses a lane and two rows a step.
//   Forward up to 64 vectors: LayerNorm 65536 x 256 23.8 us [a team of a warp,
//   one access, four rows: 27.7], 32768 x 512 24.1 [29.0]. Backward up to 16:
//   131072 x 96 43.8 [60.5]; above, a team's steps of four rows need fewer
//   instructions: 65536 x 256 34.0 [42.6], 32768 x 512 34.6 [43.5].
// - Backward up to 512 vectors: one access a thread, four rows a step: LayerNorm
//   16384 x 1024 35.4 us [two accesses, two rows: 54], 8192 x 4096 66.2 [76.8]. Two
//   teams of 192 or 224 threads would leave much of an SM idle: 16-bit rows of 161
//   to 224 vectors take the other form (RMSNorm 24876 x 1424 53.2 us [60.1],
//   17692 x 1656 62.8 [65.9]). One team of 288 to 448 threads leaves as much idle,
//   yet rows of 257 to 448 vectors stay with the first form, which is right for
//   most fp32 rows alone (LayerNorm with dropout f32 13084 x 1280 62.9 us [62.6],
//   9344 x 1792 58.6 [65.3], RMSNorm 14536 x 1152 64.8 [61.0], 9344 x 1792 56.7 [61.3];
//   bf16 LayerNorm 14536 x 2304 82.2 [71.3], 10064 x 3328 75.9 [70.5], 9344 x 3584 73.7
//   [69.6], RMSNorm 14536 x 2304 79.3 [59.2], 10064 x 3328 72.1 [65.9]; the other form
//   at its best number of teams and CTAs).
//   Above, two accesses and two rows (16-bit), or four and one: more threads do
//   not fit the columns' sums into their registers.
// - Forward: four accesses, one row: LayerNorm 16384 x 2048 46.3 us [one access,
//   four rows: 58.2]; below 128 vectors too few lanes would be busy. Few rows
//   (four per SM): one access, one row, for latency: f32 128 x 1024 2.2 us [3.6].
// CTAs hold several teams, one row each at a time, so that one computes while
// another waits: backward up to 512 threads, one CTA an SM (LayerNorm 16384 x 1024
// 35.4 us, CTAs of one team 39.2; fewer partial rows to add up, too), forward
// up to 128 (LayerNorm 16384 x 1024 23.0 us, of 32 threads 33.2). RMSNorm's
// forward of narrow rows that fill their teams is at its best with two such CTAs
// an SM and three steps in shared memory (65536 x 2048 170 us; four: 177); rows that
// do not, and LayerNorm's, with four and two steps (RMSNorm 16384 x 1500 37.0 us;
// two: 51.9). Few rows forward: the same number of CTAs on every SM, idle ones too,
// so that a following launch finds room (f32 128 x 1024 2.2 us, 128 CTAs 2.6).
norm_status plan_of(const Shape& s, int vec, int num_sms, norm_plan* p) {
    std::memset(p, 0, sizeof *p);
    if (vec == 1 && s.N > kMaxElems) return NORM_ERR_ARG;
    p->vec_elems = vec;
    p->cluster = 1;
    p->stages = vec == 1 ? 3 : 2;
    const int64_t nacc = accesses(s, vec);
    if (vec > 1 && nacc <= (s.bwd ? 16 : 64)) {
        p->mapping = NORM_MAP_GROUP;
        p->per_thread = 2;
        p->group = 1;
        while (p->group * 2 < nacc) p->group *= 2;
        p->threads = 128;
        p->rounds = 2;
    } else if (vec > 1 && nacc <= kDropMaxThreads && (s.bwd ? s.es() == 4 || nacc <= 160 || nacc > 224 : nacc < 128 || s.M <= int64_t(num_sms) * 4)) {
        p->mapping = NORM_MAP_CTA;
        p->per_thread = 1;
        p->rounds = !s.bwd && s.M <= int64_t(num_sms) * 4 ? 1 : 4;
        p->threads = static_cast<int32_t>(round_up(nacc, 32));
    } else {
        p->mapping = NORM_MAP_CTA;
        const int per = vec == 1 ? 8 : s.bwd && s.es() == 2 ? 2 : 4;
        p->per_thread = per;
        p->rounds = per == 2 ? 2 : 1;
        // the smallest cluster whose CTAs' stages fit
        for (;; p->cluster *= 2) {
            if (p->cluster > kMaxCluster) return NORM_ERR_ARG;
            p->threads = static_cast<int32_t>(round_up(ceil_div(nacc, int64_t(p->cluster) * per), 32));
            if (p->threads <= libnorm::drop_max_threads(vec, per) && smem_bytes(s, *p, p->stages) <= kDropMaxSmem) break;
        }
    }
    int64_t per_sm = s.bwd ? 512 : 1024;  // threads
    const int64_t steps = ceil_div(s.M, p->rounds);
    if (p->mapping == NORM_MAP_CTA && vec > 1 && p->cluster == 1) {
        const int most = s.bwd ? kDropMaxThreads : 128;
        const int32_t team = p->threads;
        int64_t teams = std::min<int64_t>(most / team, ceil_div(steps, num_sms));
        for (; teams > 1; --teams) {
            p->group = team;
            p->threads = static_cast<int32_t>(team * teams);
            if (smem_bytes(s, *p, p->stages) <= kDropMaxSmem) break;
        }
        if (teams <= 1) {
            p->group = 0;
            p->threads = team;
        }
        if (!s.bwd && p->per_thread == 4 && p->threads <= 128) {
            per_sm = 512;
            if (!s.ln && nacc == int64_t(4) * team_of(*p)) {
                p->stages = 3;
                per_sm = 256;
            }
        }
    }
    const int teams = teams_of(*p), unit = libnorm::drop_grid_unit(libnorm::drop_phases(s.N, vec), teams);
    const int64_t wanted = std::min<int64_t>(ceil_div(steps, teams), num_sms * std::max<int64_t>(1, per_sm / p->threads) / p->cluster);
    p->grid = std::max<int64_t>(1, ceil_div(wanted, unit)) * unit * p->cluster;
    // few rows forward: every SM the same number of CTAs
    if (!s.bwd && p->per_thread == 1 && p->rounds == 1) p->grid = round_up(round_up(p->grid, num_sms), unit);
    return NORM_OK;
}

norm_status make_plan(const Shape& s, bool aligned, int num_sms, norm_plan* p) {
    if (aligned) {
        const norm_status st = plan_of(s, 16 / s.es(), num_sms, p);
        if (st == NORM_OK) return st;
    }
    return plan_of(s, 1, num_sms, p);
}

norm_status check_plan(const norm_plan& p, const Shape& s, bool aligned) {
    const int es = s.es();
    if (p.vec_elems != 1 && (p.vec_elems != 16 / es || !aligned)) return NORM_ERR_PLAN;
    if (p.vec_elems == 1 && s.N > kMaxElems) return NORM_ERR_PLAN;
    if (p.mapping != NORM_MAP_GROUP && p.mapping != NORM_MAP_CTA) return NORM_ERR_PLAN;
    if (!known(s, p.mapping == NORM_MAP_GROUP, p.vec_elems, p.per_thread, p.rounds)) return NORM_ERR_PLAN;
    if (p.threads < 32 || p.threads > libnorm::drop_max_threads(p.vec_elems, p.per_thread) || p.threads % 32 != 0) return NORM_ERR_PLAN;
    const int64_t nacc = accesses(s, p.vec_elems);
    if (p.mapping == NORM_MAP_GROUP) {
        if (!is_pow2(p.group) || p.group > 32 || int64_t(p.group) * p.per_thread < nacc || p.cluster != 1) return NORM_ERR_PLAN;
    } else {
        if (!is_pow2(p.cluster) || p.cluster > kMaxCluster) return NORM_ERR_PLAN;
        const int team = team_of(p);
        if (team < 32 || team % 32 != 0 || p.threads % team != 0) return NORM_ERR_PLAN;
        if (team < p.threads && (p.cluster > 1 || p.vec_elems == 1)) return NORM_ERR_PLAN;
        if (int64_t(p.cluster) * team * p.per_thread < nacc) return NORM_ERR_PLAN;
    }
    if (p.stages < (p.vec_elems == 1 ? 3 : 2) || p.stages > kDropMaxStages) return NORM_ERR_PLAN;
    if (smem_bytes(s, p, p.stages) > kDropMaxSmem) return NORM_ERR_PLAN;
    const int unit = p.cluster * libnorm::drop_grid_unit(libnorm::drop_phases(s.N, p.vec_elems), teams_of(p));
    if (p.grid < unit || p.grid > kMaxGrid || p.grid % unit != 0) return NORM_ERR_PLAN;
    return NORM_OK;
}

int64_t workspace_bytes(const Shape& s, const norm_plan& p) { return p.grid / p.cluster * libnorm::drop_partial_pitch(static_cast<int32_t>((s.ln ? 2 : 1) * s.N)) * 4; }

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

// The dropout's threshold and scale; rng may be missing where nothing is dropped.
norm_status settle_mask(double p, const norm_rng* rng, DropArgs* a) {
    if (!(p >= 0.0) || !(p < 1.0)) return NORM_ERR_ARG;
    const int64_t t = static_cast<int64_t>(std::floor(p * 65536.0 + 0.5));
    if (t > 65535) return NORM_ERR_ARG;
    if (t > 0 && !rng) return NORM_ERR_ARG;
    a->limit = static_cast<uint32_t>(t) << 16;
    a->scale = static_cast<float>(65536.0 / static_cast<double>(65536 - t));
    if (t > 0) {
        if (!on(rng->device, 8)) return NORM_ERR_ARG;
        a->rng = rng->device;
        a->seed = rng->seed;
        a->offset = rng->offset;
    }
    return NORM_OK;
}

norm_status settle(const Shape& s, bool aligned, const norm_plan* plan, norm_plan* p, DropArgs* a) {
    if (plan) {
        *p = *plan;
        if (p->mapping == NORM_MAP_GROUP) p->cluster = 1;
    } else {
        int sms = 0;
        norm_status st = device_sms(&sms);
        if (st != NORM_OK) return st;
        st = make_plan(s, aligned, sms, p);
        if (st != NORM_OK) return st;
    }
    const norm_status st = check_plan(*p, s, aligned);
    if (st != NORM_OK) return st;
    a->M = s.M;
    a->N = static_cast<int32_t>(s.N);
    a->invN = 1.f / static_cast<float>(s.N);
    a->lanes = p->mapping == NORM_MAP_GROUP ? p->group : 0;
    a->team = team_of(*p);
    a->cluster = p->cluster;
    a->stages = p->stages;
    a->phases = libnorm::drop_phases(s.N, p->vec_elems);
    a->stat_bytes = stat_bytes(s, *p);
    return NORM_OK;
}

}  // namespace

extern "C" {

norm_status drop_fwd_planned(int layer_norm, const void* x, const void* residual, const void* gamma, const void* beta,
                             double prob, const norm_rng* rng, void* h, void* y, float* mean, float* rstd, int64_t M,
                             int64_t N, float eps, norm_dtype dtype, cudaStream_t stream, const norm_plan* plan) {
    const Shape s{M, N, dtype, layer_norm != 0, false};
    norm_status st = check_shape(s);
    if (st != NORM_OK) return st;
    if (!std::isfinite(eps) || eps < 0.f) return NORM_ERR_ARG;
    DropArgs a{};
    st = settle_mask(prob, rng, &a);
    if (st != NORM_OK || M == 0) return st;
    const int es = s.es();
    bool aligned = true;
    for (const void* p : {x, residual, gamma, static_cast<const void*>(h), static_cast<const void*>(y), s.ln ? beta : gamma}) {
        if (!p || !on(p, es)) return NORM_ERR_ARG;
        aligned = aligned && on(p, 16);
    }
    if (h == y || !on(mean, 4) || !on(rstd, 4)) return NORM_ERR_ARG;
    norm_plan p;
    st = settle(s, aligned, plan, &p, &a);
    if (st != NORM_OK) return st;
    a.x = x;
    a.residual = residual;
    a.gamma = gamma;
    a.beta = beta;
    a.h = h;
    a.y = y;
    a.mean = s.ln ? mean : nullptr;
    a.rstd = s.ln ? rstd : nullptr;
    a.eps = eps;
    switch (dtype) {
        case NORM_F32: return done(libnorm::launch_drop_fwd_f32(p, a, s.ln, stream));
        case NORM_BF16: return done(libnorm::launch_drop_fwd_bf16(p, a, s.ln, stream));
        default: return done(libnorm::launch_drop_fwd_f16(p, a, s.ln, stream));
    }
}

norm_status drop_bwd_planned(int layer_norm, const void* dy, const void* dh, const void* h, const void* gamma,
                             const float* mean, const float* rstd, double prob, const norm_rng* rng, void* dx,
                             void* dresidual, float* dgamma, float* dbeta, void* workspace, size_t workspace_size,
                             int64_t M, int64_t N, float eps, norm_dtype dtype, cudaStream_t stream,
                             const norm_plan* plan) {
    const Shape s{M, N, dtype, layer_norm != 0, true};
    norm_status st = check_shape(s);
    if (st != NORM_OK) return st;
    if (!s.ln && (!std::isfinite(eps) || eps < 0.f)) return NORM_ERR_ARG;
    if (!dgamma || !on(dgamma, 4) || (s.ln && (!dbeta || !on(dbeta, 4)))) return NORM_ERR_ARG;
    DropArgs a{};
    st = settle_mask(prob, rng, &a);
    if (st != NORM_OK) return st;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.N = static_cast<int32_t>(N);
    if (M == 0) return done(libnorm::launch_drop_colsum(a, 0, s.ln, stream));
    if (a.limit != 0 && !dx) return NORM_ERR_ARG;
    const int es = s.es();
    bool aligned = on(dh, 16) && on(dx, 16);
    if (!on(dh, es) || !on(dx, es)) return NORM_ERR_ARG;
    for (const void* p : {dy, h, gamma, static_cast<const void*>(dresidual)}) {
        if (!p || !on(p, es)) return NORM_ERR_ARG;
        aligned = aligned && on(p, 16);
    }
    if (dx == dresidual) return NORM_ERR_ARG;
    if (s.ln && (!mean || !rstd || !on(mean, 4) || !on(rstd, 4))) return NORM_ERR_ARG;
    norm_plan p;
    st = settle(s, aligned, plan, &p, &a);
    if (st != NORM_OK) return st;
    if (!workspace || !on(workspace, 16) || workspace_size < static_cast<size_t>(workspace_bytes(s, p))) return NORM_ERR_ARG;
    a.dy = dy;
    a.dh = dh;
    a.hin = h;
    a.gamma = gamma;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dx = dx;
    a.dres = dresidual;
    a.ws = static_cast<float*>(workspace);
    a.eps = eps;
    switch (dtype) {
        case NORM_F32: return done(libnorm::launch_drop_bwd_f32(p, a, s.ln, stream));
        case NORM_BF16: return done(libnorm::launch_drop_bwd_bf16(p, a, s.ln, stream));
        default: return done(libnorm::launch_drop_bwd_f16(p, a, s.ln, stream));
    }
}

norm_status ln_fwd_dropout_add(const void* x, const void* residual, const void* gamma, const void* beta, double p,
                               const norm_rng* rng, void* h, void* y, float* mean, float* rstd, int64_t M, int64_t N,
                               float eps, norm_dtype dtype, cudaStream_t stream) {
    return drop_fwd_planned(1, x, residual, gamma, beta, p, rng, h, y, mean, rstd, M, N, eps, dtype, stream, nullptr);
}

norm_status rms_fwd_dropout_add(const void* x, const void* residual, const void* w, double p, const norm_rng* rng,
                                void* h, void* y, int64_t M, int64_t N, float eps, norm_dtype dtype,
                                cudaStream_t stream) {
    return drop_fwd_planned(0, x, residual, w, nullptr, p, rng, h, y, nullptr, nullptr, M, N, eps, dtype, stream, nullptr);
}

norm_status ln_bwd_dropout_add(const void* dy, const void* dh, const void* h, const void* gamma, const float* mean,
                               const float* rstd, double p, const norm_rng* rng, void* dx, void* dresidual,
                               float* dgamma, float* dbeta, void* workspace, size_t workspace_size, int64_t M,
                               int64_t N, norm_dtype dtype, cudaStream_t stream) {
    if (M > 0 && !dx) return NORM_ERR_ARG;
    return drop_bwd_planned(1, dy, dh, h, gamma, mean, rstd, p, rng, dx, dresidual, dgamma, dbeta, workspace,
                            workspace_size, M, N, 0.f, dtype, stream, nullptr);
}

norm_status rms_bwd_dropout_add(const void* dy, const void* dh, const void* h, const void* w, double p,
                                const norm_rng* rng, void* dx, void* dresidual, float* dw, void* workspace,
                                size_t workspace_size, int64_t M, int64_t N, float eps, norm_dtype dtype,
                                cudaStream_t stream) {
    if (M > 0 && !dx) return NORM_ERR_ARG;
    return drop_bwd_planned(0, dy, dh, h, w, nullptr, nullptr, p, rng, dx, dresidual, dw, nullptr, workspace,
                            workspace_size, M, N, eps, dtype, stream, nullptr);
}

norm_status ln_bwd_add(const void* dy, const void* dh, const void* h, const void* gamma, const float* mean,
                       const float* rstd, void* d, float* dgamma, float* dbeta, void* workspace, size_t workspace_size,
                       int64_t M, int64_t N, norm_dtype dtype, cudaStream_t stream) {
    return drop_bwd_planned(1, dy, dh, h, gamma, mean, rstd, 0.0, nullptr, nullptr, d, dgamma, dbeta, workspace,
                            workspace_size, M, N, 0.f, dtype, stream, nullptr);
}

norm_status rms_bwd_add(const void* dy, const void* dh, const void* h, const void* w, void* d, float* dw,
                        void* workspace, size_t workspace_size, int64_t M, int64_t N, float eps, norm_dtype dtype,
                        cudaStream_t stream) {
    return drop_bwd_planned(0, dy, dh, h, w, nullptr, nullptr, 0.0, nullptr, nullptr, d, dw, nullptr, workspace,
                            workspace_size, M, N, eps, dtype, stream, nullptr);
}

norm_status drop_make_plan(int64_t M, int64_t N, norm_dtype dtype, int layer_norm, int backward, int aligned16,
                           int num_sms, norm_plan* plan) {
    const Shape s{M, N, dtype, layer_norm != 0, backward != 0};
    const norm_status st = check_shape(s);
    if (st != NORM_OK) return st;
    if (!plan || num_sms < 1) return NORM_ERR_ARG;
    return make_plan(s, aligned16 != 0, num_sms, plan);
}

norm_status drop_workspace_bytes(int64_t M, int64_t N, norm_dtype dtype, int layer_norm, int num_sms,
                                 const norm_plan* plan, size_t* bytes) {
    const Shape s{M, N, dtype, layer_norm != 0, true};
    norm_status st = check_shape(s);
    if (st != NORM_OK) return st;
    if (!bytes || (!plan && num_sms < 1)) return NORM_ERR_ARG;
    *bytes = 0;
    if (M == 0) return NORM_OK;
    if (plan) {
        if (plan->cluster < 1 && plan->mapping != NORM_MAP_GROUP) return NORM_ERR_ARG;
        norm_plan p = *plan;
        if (p.mapping == NORM_MAP_GROUP) p.cluster = 1;
        if (p.grid < 0 || p.grid > kMaxGrid) return NORM_ERR_ARG;
        *bytes = static_cast<size_t>(workspace_bytes(s, p));
        return NORM_OK;
    }
    for (bool aligned : {true, false}) {
        norm_plan p;
        st = make_plan(s, aligned, num_sms, &p);
        if (st == NORM_OK) *bytes = std::max(*bytes, static_cast<size_t>(workspace_bytes(s, p)));
        else if (aligned) return st;
    }
    return NORM_OK;
}

}  // extern "C"
