// Group norm entry points of the C ABI: argument checks, the launch planner
// and dispatch. Every argument error is caught here, before any CUDA call.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <numeric>

#include <cuda_runtime_api.h>

#include "gn_args.h"
#include "norm_args.h"

namespace {

using libnorm::GnArgs;
using libnorm::kGnMaxMixedChannels;
using libnorm::kGnMaxThreads;

constexpr int64_t kMaxC = int64_t(1) << 24;
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSmem = 48 * 1024;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxChunk = int64_t(1) << 30;  // values of one access column in a row chunk
constexpr int kFoldRows = 64, kMaxFolds = 256;  // partial rows per folded one, folded rows
constexpr int kSplitFoldFrom = 4096;            // more partial rows than this are folded on the split path
constexpr int kFwdMaxRows = 8, kBwdMaxRows = 4;  // rows a thread of the on-chip kernels can hold

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
int elem_size(norm_dtype d) { return d == NORM_F32 ? 4 : 2; }

struct Shape {
    int64_t B, S, C, G, D;
    norm_dtype dtype;
    bool bwd;
};

norm_status check_shape(int64_t B, int64_t S, int64_t C, int64_t G, norm_dtype dtype, bool bwd, Shape* out) {
    if (dtype != NORM_F32 && dtype != NORM_BF16 && dtype != NORM_F16) return NORM_ERR_DTYPE;
    if (C < 1 || C > kMaxC || G < 1 || G > C || C % G != 0 || B < 0 || S < 0) return NORM_ERR_ARG;
    if (B > (kMaxGrid - 1) / C) return NORM_ERR_ARG;
    if (B > 0 && S > (int64_t(1) << 62) / (B * C)) return NORM_ERR_ARG;
    *out = Shape{B, S, C, G, C / G, dtype, bwd};
    return NORM_OK;
}

// A null pointer or one on a boundary of `bytes`.
bool on(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// One [B, S, C] tensor of a call.
struct Tensor {
    const void* p;
    int64_t batch, row;
};

// Pitches that are not used (one row, one sample) are made those of a
// contiguous tensor.
norm_status check_tensor(const Shape& s, Tensor* t) {
    if (!t->p) return NORM_ERR_ARG;
    if (s.S == 1) t->row = s.C;
    if (t->row < s.C || t->row > (int64_t(1) << 40)) return NORM_ERR_ARG;
    const __int128 span = static_cast<__int128>(s.S - 1) * t->row + s.C;
    if (span >= (static_cast<__int128>(1) << 61)) return NORM_ERR_ARG;
    if (s.B == 1) t->batch = static_cast<int64_t>(span);
    if (t->batch < static_cast<int64_t>(span)) return NORM_ERR_ARG;
    if (static_cast<__int128>(s.B) * t->batch >= (static_cast<__int128>(1) << 61)) return NORM_ERR_ARG;
    if (!on(t->p, elem_size(s.dtype))) return NORM_ERR_ARG;
    return NORM_OK;
}

// The widest access for these tensors and parameters: 16 bytes, two 16-bit
// values, or one element.
int allowed_vec(const Shape& s, const Tensor* ts, int n, const void* gamma, const void* beta) {
    const int es = elem_size(s.dtype);
    for (int vec : {16 / es, 2, 1}) {
        if (vec == 2 && es == 4) continue;
        const int64_t bytes = int64_t(vec) * es;
        bool ok = s.C % vec == 0 && reinterpret_cast<uintptr_t>(gamma) % bytes == 0 &&
                  reinterpret_cast<uintptr_t>(beta) % bytes == 0;
        for (int i = 0; ok && i < n; ++i)
            ok = reinterpret_cast<uintptr_t>(ts[i].p) % bytes == 0 && (s.S == 1 || ts[i].row % vec == 0) &&
                 (s.B == 1 || ts[i].batch % vec == 0);
        if (ok) return vec;
    }
    return 1;
}

// Accesses that make up whole groups: one group when accesses lie within
// groups, otherwise the fewest groups that end on an access boundary.
int64_t group_unit(int64_t D, int vec) { return D / std::gcd(D, int64_t(vec)); }

bool one_group(const Shape& s, int vec) { return s.D % vec == 0; }

int64_t tile_cap(const Shape& s, int vec) {
    return one_group(s, vec) ? kGnMaxThreads : std::max<int64_t>(1, kGnMaxMixedChannels / vec);
}

// Everything a launch needs beyond the plan's own fields; NORM_ERR_PLAN if
// the plan does not fit the call.
norm_status derive(const gn_plan& p, const Shape& s, GnArgs* a) {
    const int es = elem_size(s.dtype);
    const int maxv = s.bwd ? kBwdMaxRows : kFwdMaxRows;
    if (p.path != GN_PATH_CHIP && p.path != GN_PATH_SPLIT) return NORM_ERR_PLAN;
    if (p.vec_elems != 16 / es && p.vec_elems != 1 && !(p.vec_elems == 2 && es == 2)) return NORM_ERR_PLAN;
    if (s.C % p.vec_elems != 0) return NORM_ERR_PLAN;
    if (p.threads < 32 || p.threads > kGnMaxThreads || p.threads % 32 != 0) return NORM_ERR_PLAN;
    const int64_t ncols = s.C / p.vec_elems;
    if (p.tile < 1 || p.tile > p.threads || p.tile > tile_cap(s, p.vec_elems)) return NORM_ERR_PLAN;
    if (!is_pow2(p.cluster) || p.cluster > kMaxCluster) return NORM_ERR_PLAN;
    const int64_t unit = group_unit(s.D, p.vec_elems);
    const bool whole = p.tile % unit == 0 || p.tile >= ncols;
    a->C = static_cast<int32_t>(s.C);
    a->G = static_cast<int32_t>(s.G);
    a->D = static_cast<int32_t>(s.D);
    a->S = s.S;
    a->ncols = static_cast<int32_t>(ncols);
    a->tile = static_cast<int32_t>(std::min<int64_t>(p.tile, ncols));
    a->tiles = static_cast<int32_t>(ceil_div(ncols, a->tile));
    a->par = p.threads / a->tile;
    a->by_tile = libnorm::fast_div(a->tile);
    a->by_tiles = libnorm::fast_div(a->tiles);
    a->by_par = libnorm::fast_div(a->par);
    a->by_D = libnorm::fast_div(s.D);
    a->cluster = p.cluster;
    a->cluster_bits = p.cluster == 8 ? 3 : p.cluster >> 1;
    a->join = 1;
    a->folds = 0;
    a->segs = one_group(s, p.vec_elems) ? 1
                                        : static_cast<int32_t>(std::min<int64_t>(p.vec_elems, (p.vec_elems - 2 + s.D) / s.D + 1));
    const int states = a->tile * (s.bwd ? p.vec_elems : a->segs);
    const int64_t groups = libnorm::gn_tile_groups(int64_t(a->tile) * p.vec_elems, s.D, false);
    const int64_t smem = libnorm::gn_smem_bytes(a->par, states, static_cast<int>(groups), p.threads);
    if (smem > kMaxSmem) return NORM_ERR_PLAN;
    a->ring_at = static_cast<int32_t>(smem / 16);
    if (p.path == GN_PATH_CHIP) {
        if (!whole || !is_pow2(p.per_thread) || p.per_thread > maxv) return NORM_ERR_PLAN;
        a->tpg = 1;
        a->chunks = a->out_chunks = 1;
        a->chunk_rows = a->out_rows = std::max<int64_t>(1, ceil_div(s.S, p.cluster));
        if (a->chunk_rows > int64_t(a->par) * p.per_thread) return NORM_ERR_PLAN;
        // the backward's samples meet in one cluster where they fit
        if (s.bwd && s.B * p.cluster <= kMaxCluster) a->join = static_cast<int32_t>(s.B);
        a->by_cluster = libnorm::fast_div(int64_t(p.cluster) * a->join);
        a->partials = static_cast<int32_t>(a->join > 1 ? 1 : s.B);
        // The column sum is a CTA per 128 channels: beyond some rows they are
        // added over the whole device first (gn_bwd bf16 4096x16x64 21 us
        // instead of 40, 65536x4x64 80 instead of 536).
        if (s.bwd && a->partials > 8 * kFoldRows)
            a->folds = static_cast<int32_t>(std::min<int64_t>(kMaxFolds, ceil_div(a->partials, kFoldRows)));
        if (s.B * a->tiles > kMaxGrid / p.cluster) return NORM_ERR_PLAN;
        return NORM_OK;
    }
    if (p.cluster != 1 || p.chunks < 1 || p.out_chunks < 1) return NORM_ERR_PLAN;
    a->tpg = static_cast<int32_t>(whole ? 1 : ceil_div(s.D - 1, int64_t(a->tile) * p.vec_elems) + 1);
    a->chunks = p.chunks;
    a->out_chunks = p.out_chunks;
    a->by_chunks = libnorm::fast_div(p.chunks);
    a->by_out_chunks = libnorm::fast_div(p.out_chunks);
    a->chunk_rows = std::max<int64_t>(1, ceil_div(s.S, p.chunks));
    a->out_rows = std::max<int64_t>(1, ceil_div(s.S, p.out_chunks));
    // (a thread counts rows times an access's channels in 32 bits)
    if (a->chunk_rows * p.vec_elems > kMaxChunk || a->out_rows > kMaxChunk) return NORM_ERR_PLAN;
    // CTAs of a launch, and partial rows of the column gradients
    const int64_t units = s.B * a->tiles, tall = std::max(p.chunks, p.out_chunks);
    if (tall > kMaxGrid / 4 / std::max<int64_t>(1, units) || s.B > kMaxGrid / p.chunks) return NORM_ERR_PLAN;
    a->partials = static_cast<int32_t>(s.B * p.chunks);
    // The second launch's adders are a CTA per 32 columns: beyond some partial
    // rows they finish after everything else, and the rows are added over the
    // whole device instead, in two more launches. Adders / folds in us: gn_bwd
    // bf16 1030x1100x64 (2060 rows) 121 / 127, 4096x1100x64 420 / 424, f32
    // 16384x1100x8 508 / 454, bf16 65536x1100x8 1531 / 1240.
    if (s.bwd && a->partials > kSplitFoldFrom)
        a->folds = static_cast<int32_t>(std::min<int64_t>(kMaxFolds, ceil_div(a->partials, kFoldRows)));
    return NORM_OK;
}

bool chip_plan(const Shape& s, int vec, int sms, gn_plan* p) {
    const int es = elem_size(s.dtype);
    const int64_t ncols = s.C / vec, unit = group_unit(s.D, vec), cap = tile_cap(s, vec);
    if (unit > cap) return false;
    // at least 64 bytes of a row, so that DRAM accesses are whole
    int64_t tile = std::min(ncols, unit * std::max<int64_t>(1, ceil_div(64, unit * vec * es)));
    if (tile > cap) tile = unit;
    // wider where rows are few and tiles many
    while (tile * 2 <= std::min(ncols, cap) && tile * s.S <= 128 && s.B * ceil_div(ncols, tile * 2) >= 2 * sms)
        tile *= 2;
    const int64_t units = s.B * ceil_div(ncols, tile);
    const int maxv = s.bwd ? kBwdMaxRows : kFwdMaxRows;
    bool found = false;
    for (int cs = 1; cs <= kMaxCluster; cs *= 2) {
        const int64_t rows = ceil_div(s.S, cs);
        int v = 1;
        while (v <= maxv && ceil_div(rows, v) * tile > kGnMaxThreads) v *= 2;
        if (v > maxv) continue;
        // a backward whose samples do not meet in one cluster needs another
        // launch for the column sums, and clusters then lose to the split path
        // (gn_bwd f32 3x1517x180 10.1 us against 8.6)
        if (s.bwd && cs > 1 && s.B * cs > kMaxCluster) break;
        if (found && (rows * tile < 256 || units * cs > 4 * int64_t(sms))) break;
        // The largest clusters lose to the split path where they are many CTAs
        // per SM (gn_fwd f32 16x1024x1280 60 us against 45; in clusters of 4,
        // f32 8x1024x640, 17.0 against 18.9), and, at the most rows per thread,
        // where they leave SMs without one (bf16 1x4096x512 9.6 us against
        // 8.1, 2x2048x320 8.0 against 7.4).
        if (cs == kMaxCluster && (units * cs > 4 * int64_t(sms) || (v == maxv && units * cs < sms))) break;
        p->path = GN_PATH_CHIP;
        p->vec_elems = vec;
        p->tile = static_cast<int32_t>(tile);
        p->threads = static_cast<int32_t>(round_up(std::max<int64_t>(1, ceil_div(rows, v)) * tile, 32));
        p->per_thread = v;
        p->cluster = cs;
        found = true;
        if (units * cs >= sms) break;
    }
    return found;
}

void split_plan(const Shape& s, int vec, int sms, gn_plan* p) {
    const int es = elem_size(s.dtype);
    const int64_t ncols = s.C / vec, unit = group_unit(s.D, vec), cap = tile_cap(s, vec);
    // tiles of at least 128 bytes of a row, whole groups
    int64_t tile = std::min(ncols, cap);
    if (unit <= cap) tile = std::min(tile, unit * std::max<int64_t>(1, ceil_div(128, unit * vec * es)));
    if (tile > cap) tile = unit;
    p->path = GN_PATH_SPLIT;
    p->vec_elems = vec;
    p->tile = static_cast<int32_t>(tile);
    p->threads = static_cast<int32_t>(round_up(std::max<int64_t>(1, 256 / tile) * tile, 32));
    p->cluster = 1;
    const int64_t units = std::max<int64_t>(1, s.B * ceil_div(ncols, tile));
    const int64_t rows = p->threads / tile;
    // One CTA per SM while a thread has few rows, two per SM otherwise (four of
    // narrower accesses, which have fewer bytes in flight each: f16 5x363654x25
    // gn_fwd 97 us instead of 146, gn_bwd 150 instead of 215); counts between
    // leave some SMs with twice the rows of others. Measured in us with
    // one / two per SM, at the rows per thread that one gives: gn_fwd bf16
    // 2x4096x320 (9 rows) 9.4 / 11.8, 1x16384x256 (14) 10.0 / 10.4, 2x8192x320
    // (18) 12.1 / 14.7, f32 2x4096x320 (19) 12.4 / 12.2, bf16 8x4096x320 (41)
    // 23.3 / 20.4; gn_bwd f32 3x1517x180 (6) 8.7 / 9.8, bf16 1x4096x512 (7)
    // 11.7 / 10.2, 2x4096x320 (9) 13.9 / 12.7, 4x4096x320 (19) 19.6 / 16.2. With
    // narrower accesses, one / four per SM: gn_bwd f32 2x10000x30 (17) 9.5 /
    // 12.5, gn_fwd f32 10x445x175 (22) 8.3 / 9.5, f16 8x1500x75 (56) 11.9 / 9.9.
    const int64_t once = std::max<int64_t>(1, sms / units);
    const bool whole = vec * es == 16;  // 16-byte accesses
    const int64_t slots = int64_t(sms) * (whole ? 2 : 4);
    const int64_t few = whole ? (s.bwd ? 6 : 18) : (s.bwd ? 24 : 36);
    int64_t chunks = once;
    if (ceil_div(ceil_div(s.S, once), rows) > few) {
        // Where whole chunks of every sample and tile leave a tenth of the two
        // CTAs per SM without work, up to 8 rounds of them, the first that
        // leave less or the fullest, while a thread has 16 rows or more (gn_bwd
        // f16 14x5390x768, 154 tiles: 112 us with 9 chunks each, 164 with 1;
        // gn_fwd bf16 10x2897x1024 36 with 5, 45 with 1).
        double best = 0.0;
        for (int64_t round = 1; round <= 8 && best < 0.9; ++round) {
            const int64_t c = std::max<int64_t>(1, round * slots / units);
            if (round > 1 && s.S / (c * rows) < 16) break;
            const double used = static_cast<double>(c * units) / static_cast<double>(round_up(c * units, slots));
            if (used > best) {
                best = used;
                chunks = c;
            }
        }
    }
    const int64_t most = std::max<int64_t>(1, ceil_div(s.S, rows));
    p->chunks = static_cast<int32_t>(std::max(std::min(std::max<int64_t>(1, chunks), most), ceil_div(s.S * vec, kMaxChunk)));
    p->out_chunks = p->chunks;
}

// The plan for accesses of `vec` elements.
norm_status make_plan(const Shape& s, int vec, int sms, gn_plan* p) {
    std::memset(p, 0, sizeof *p);
    GnArgs a;
    p->chunks = p->out_chunks = 1;
    if (!chip_plan(s, vec, sms, p) || derive(*p, s, &a) != NORM_OK) {
        std::memset(p, 0, sizeof *p);
        p->per_thread = 1;
        split_plan(s, vec, sms, p);
    }
    return derive(*p, s, &a) == NORM_OK ? NORM_OK : NORM_ERR_ARG;
}

// The parts of the workspace, in order; each starts on a 16-byte boundary.
struct Workspace {
    int64_t shift, part, cols, fold, bytes;
};
Workspace layout(const gn_plan& p, const Shape& s, const GnArgs& a) {
    Workspace w{0, 0, 0, 0, 0};
    if (s.B == 0 || s.S == 0) return w;
    if (p.path != GN_PATH_CHIP) {
        w.part = w.shift + (s.bwd ? 0 : round_up(s.B * s.G * 4, 16));
        w.cols = w.part + s.B * s.G * a.tpg * a.chunks * 16;
    }
    w.fold = w.cols + (s.bwd && a.partials > 1 ? round_up(int64_t(a.partials) * 2 * s.C * 4, 16) : 0);
    w.bytes = w.fold + int64_t(a.folds) * 2 * s.C * 4;
    return w;
}

// SM count of the current device, asked once per device.
int device_sms() {
    static std::atomic<int> cache[64];
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= 0 && dev < 64) n = cache[dev].load(std::memory_order_relaxed);
    if (e == cudaSuccess && n <= 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    }
    if (e != cudaSuccess || n <= 0) {
        libnorm::note_cuda_error(static_cast<int>(e));
        return -1;
    }
    return n;
}

// The plan of a call (the caller's, or the planner's) and its workspace.
norm_status settle(const Shape& s, int vec, const gn_plan* user, void* ws, size_t ws_bytes, gn_plan* p, GnArgs* a) {
    if (user) {
        *p = *user;
        if (p->vec_elems > vec) return NORM_ERR_PLAN;
        const norm_status st = derive(*p, s, a);
        if (st != NORM_OK) return st;
    } else {
        const int sms = device_sms();
        if (sms <= 0) return NORM_ERR_CUDA;
        norm_status st = make_plan(s, vec, sms, p);
        if (st != NORM_OK) return st;
        st = derive(*p, s, a);
        if (st != NORM_OK) return st;
    }
    const Workspace w = layout(*p, s, *a);
    if (w.bytes > 0) {
        if (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0 || ws_bytes < static_cast<size_t>(w.bytes)) return NORM_ERR_ARG;
        char* base = static_cast<char*>(ws);
        a->shift = reinterpret_cast<float*>(base + w.shift);
        a->part = base + w.part;
        a->colg = reinterpret_cast<float*>(base + w.cols);
        a->fold = reinterpret_cast<float*>(base + w.fold);
    }
    return NORM_OK;
}

norm_status done(cudaError_t e) {
    if (e == cudaSuccess) return NORM_OK;
    libnorm::note_cuda_error(static_cast<int>(e));
    return NORM_ERR_CUDA;
}

bool act_ok(norm_act act) { return act == NORM_ACT_NONE || act == NORM_ACT_SILU || act == NORM_ACT_GELU; }

bool same_or_apart(const Tensor& out, const Tensor& in) {
    return out.p != in.p || (out.batch == in.batch && out.row == in.row);
}

}  // namespace

extern "C" {

norm_status gn_fwd_planned(const void* x, int64_t x_batch, int64_t x_row, const void* gamma, const void* beta,
                           void* y, int64_t y_batch, int64_t y_row, float* mean, float* rstd, void* workspace,
                           size_t workspace_bytes, int64_t B, int64_t S, int64_t C, int64_t G, float eps,
                           norm_act act, norm_dtype dtype, cudaStream_t stream, const gn_plan* plan) {
    Shape s;
    norm_status st = check_shape(B, S, C, G, dtype, false, &s);
    if (st != NORM_OK) return st;
    if (!std::isfinite(eps) || eps < 0.f || !act_ok(act)) return NORM_ERR_ARG;
    if (B == 0 || S == 0) return NORM_OK;
    const int es = elem_size(dtype);
    if (!gamma || !beta || !on(gamma, es) || !on(beta, es) || !on(mean, 4) || !on(rstd, 4)) return NORM_ERR_ARG;
    Tensor t[2] = {{x, x_batch, x_row}, {y, y_batch, y_row}};
    for (Tensor& i : t)
        if ((st = check_tensor(s, &i)) != NORM_OK) return st;
    if (!same_or_apart(t[1], t[0])) return NORM_ERR_ARG;
    gn_plan p;
    GnArgs a{};
    st = settle(s, allowed_vec(s, t, 2, gamma, beta), plan, workspace, workspace_bytes, &p, &a);
    if (st != NORM_OK) return st;
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.xb = t[0].batch;
    a.xr = t[0].row;
    a.yb = t[1].batch;
    a.yr = t[1].row;
    a.eps = eps;
    switch (dtype) {
        case NORM_F32: return done(libnorm::launch_gn_fwd_f32(p, a, act, B, stream));
        case NORM_BF16: return done(libnorm::launch_gn_fwd_bf16(p, a, act, B, stream));
        default: return done(libnorm::launch_gn_fwd_f16(p, a, act, B, stream));
    }
}

norm_status gn_fwd(const void* x, int64_t x_batch, int64_t x_row, const void* gamma, const void* beta, void* y,
                   int64_t y_batch, int64_t y_row, float* mean, float* rstd, void* workspace, size_t workspace_bytes,
                   int64_t B, int64_t S, int64_t C, int64_t G, float eps, norm_act act, norm_dtype dtype,
                   cudaStream_t stream) {
    return gn_fwd_planned(x, x_batch, x_row, gamma, beta, y, y_batch, y_row, mean, rstd, workspace, workspace_bytes,
                          B, S, C, G, eps, act, dtype, stream, nullptr);
}

norm_status gn_bwd_planned(const void* dy, int64_t dy_batch, int64_t dy_row, const void* x, int64_t x_batch,
                           int64_t x_row, const void* gamma, const void* beta, const float* mean, const float* rstd,
                           void* dx, int64_t dx_batch, int64_t dx_row, float* dgamma, float* dbeta, void* workspace,
                           size_t workspace_bytes, int64_t B, int64_t S, int64_t C, int64_t G, norm_act act,
                           norm_dtype dtype, cudaStream_t stream, const gn_plan* plan) {
    Shape s;
    norm_status st = check_shape(B, S, C, G, dtype, true, &s);
    if (st != NORM_OK) return st;
    if (!act_ok(act) || !dgamma || !dbeta || !on(dgamma, 4) || !on(dbeta, 4)) return NORM_ERR_ARG;
    gn_plan p{};
    GnArgs a{};
    a.C = static_cast<int32_t>(C);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    if (B > 0 && S > 0) {
        const int es = elem_size(dtype);
        if (!gamma || !beta || !mean || !rstd) return NORM_ERR_ARG;
        if (!on(gamma, es) || !on(beta, es) || !on(mean, 4) || !on(rstd, 4)) return NORM_ERR_ARG;
        Tensor t[3] = {{dy, dy_batch, dy_row}, {x, x_batch, x_row}, {dx, dx_batch, dx_row}};
        for (Tensor& i : t)
            if ((st = check_tensor(s, &i)) != NORM_OK) return st;
        if (!same_or_apart(t[2], t[0]) || !same_or_apart(t[2], t[1])) return NORM_ERR_ARG;
        st = settle(s, allowed_vec(s, t, 3, gamma, beta), plan, workspace, workspace_bytes, &p, &a);
        if (st != NORM_OK) return st;
        a.dy = dy;
        a.x = x;
        a.gamma = gamma;
        a.beta = beta;
        a.mean = const_cast<float*>(mean);
        a.rstd = const_cast<float*>(rstd);
        a.y = dx;
        a.dyb = t[0].batch;
        a.dyr = t[0].row;
        a.xb = t[1].batch;
        a.xr = t[1].row;
        a.yb = t[2].batch;
        a.yr = t[2].row;
        if (a.partials == 1) {  // dgamma and dbeta are written without partial rows
            a.colg = dgamma;
            a.colb = dbeta;
        } else {
            a.colb = a.colg + C;
            a.col_pitch = 2 * C;
        }
    }
    switch (dtype) {
        case NORM_F32: return done(libnorm::launch_gn_bwd_f32(p, a, act, B, stream));
        case NORM_BF16: return done(libnorm::launch_gn_bwd_bf16(p, a, act, B, stream));
        default: return done(libnorm::launch_gn_bwd_f16(p, a, act, B, stream));
    }
}

norm_status gn_bwd(const void* dy, int64_t dy_batch, int64_t dy_row, const void* x, int64_t x_batch, int64_t x_row,
                   const void* gamma, const void* beta, const float* mean, const float* rstd, void* dx,
                   int64_t dx_batch, int64_t dx_row, float* dgamma, float* dbeta, void* workspace,
                   size_t workspace_bytes, int64_t B, int64_t S, int64_t C, int64_t G, norm_act act, norm_dtype dtype,
                   cudaStream_t stream) {
    return gn_bwd_planned(dy, dy_batch, dy_row, x, x_batch, x_row, gamma, beta, mean, rstd, dx, dx_batch, dx_row,
                          dgamma, dbeta, workspace, workspace_bytes, B, S, C, G, act, dtype, stream, nullptr);
}

norm_status gn_make_plan(int64_t B, int64_t S, int64_t C, int64_t G, norm_dtype dtype, int backward, int vec_elems,
                         int num_sms, gn_plan* plan) {
    Shape s;
    const norm_status st = check_shape(B, S, C, G, dtype, backward != 0, &s);
    if (st != NORM_OK) return st;
    if (!plan || num_sms < 1 || B == 0 || S == 0) return NORM_ERR_ARG;
    const int es = elem_size(dtype);
    if ((vec_elems != 16 / es && vec_elems != 1 && !(vec_elems == 2 && es == 2)) || C % vec_elems != 0) return NORM_ERR_ARG;
    return make_plan(s, vec_elems, num_sms, plan);
}

norm_status gn_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G, norm_dtype dtype, int backward,
                               int num_sms, const gn_plan* plan, size_t* bytes) {
    Shape s;
    norm_status st = check_shape(B, S, C, G, dtype, backward != 0, &s);
    if (st != NORM_OK) return st;
    if (!bytes || (!plan && num_sms < 1)) return NORM_ERR_ARG;
    *bytes = 0;
    if (B == 0 || S == 0) return NORM_OK;
    GnArgs a{};
    if (plan) {
        st = derive(*plan, s, &a);
        if (st != NORM_OK) return st;
        *bytes = static_cast<size_t>(layout(*plan, s, a).bytes);
        return NORM_OK;
    }
    const int es = elem_size(dtype);
    for (int vec : {16 / es, 2, 1}) {
        if ((vec == 2 && es == 4) || C % vec != 0) continue;
        gn_plan p;
        st = make_plan(s, vec, num_sms, &p);
        if (st != NORM_OK) return st;
        derive(p, s, &a);
        *bytes = std::max(*bytes, static_cast<size_t>(layout(p, s, a).bytes));
    }
    return NORM_OK;
}

}  // extern "C"
