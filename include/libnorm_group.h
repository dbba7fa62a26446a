/*
 * libnorm - group norm over channels-last tensors, with an activation,
 * forward and backward, for NVIDIA GB300 (sm_103a). Part of the same library
 * as libnorm.h, whose conventions hold here too (device pointers owned by the
 * caller, asynchronous work on `stream`, argument errors detected on the host
 * before any CUDA call, fp32 arithmetic, nearest-even output rounding).
 *
 * A tensor is [B, S, C]: B samples, S positions (height x width, frames, or
 * time x height x width), C channels, channels innermost. The C channels form
 * G groups of D = C / G neighbours; statistics run over the S * D values of a
 * sample's group. Rows (positions) may have a pitch of their own and samples
 * too: element (b, s, c) of x is x[b * x_batch + s * x_row + c], pitches in
 * elements, x_row >= C, x_batch >= (S - 1) * x_row + C (ignored where S or B
 * is 1). Every pointer needs its element's alignment (others are refused); 16-byte
 * accesses are used when every tensor and parameter is 16-byte aligned and
 * C and all pitches are whole 16-byte vectors, 4-byte accesses of 16-bit
 * pairs when the same holds for 4 bytes, element accesses otherwise.
 *
 * Limits: 1 <= C <= 2^24, 1 <= G <= C, G divides C, B, S >= 0,
 * B * S * C < 2^62, B * C < 2^31, eps finite and >= 0. B == 0 or S == 0:
 * nothing is normalised (dgamma and dbeta are still written, as zeros; mean
 * and rstd of empty groups are left as they were).
 */
#ifndef LIBNORM_GROUP_H
#define LIBNORM_GROUP_H

#include "libnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NORM_ACT_NONE = 0,
    NORM_ACT_SILU = 1, /* z / (1 + exp(-z)) */
    NORM_ACT_GELU = 2  /* z * (1 + erf(z / sqrt 2)) / 2 */
} norm_act;

typedef enum {
    GN_PATH_CHIP = 0, /* a CTA or a cluster holds a sample's tile on chip: x (and dy) is read once */
    GN_PATH_SPLIT = 1 /* one launch sums row chunks into the workspace, a second reads the rows again and writes */
} gn_path;

/* A launch plan of gn_fwd / gn_bwd. Every CTA works on a tile of `tile`
 * neighbouring accesses (of `vec_elems` channels each) of a run of rows. */
typedef struct {
    int32_t path;       /* gn_path */
    int32_t vec_elems;  /* channels per access: 16 / sizeof(element), 2 (16-bit types) or 1 */
    int32_t tile;       /* accesses per row a CTA covers: whole groups for GN_PATH_CHIP */
    int32_t threads;    /* threads per CTA, a multiple of 32, tile <= threads <= 256 */
    int32_t per_thread; /* CHIP: rows each thread holds, 1, 2, 4 or 8 (backward: up to 4) */
    int32_t cluster;    /* CHIP: the CTAs that share a sample's tile, 1, 2, 4 or 8; otherwise 1 */
    int32_t chunks;     /* SPLIT: row chunks per sample and tile that are summed */
    int32_t out_chunks; /* SPLIT: row chunks per sample and tile that are written */
} gn_plan;

/*
 * Group norm forward:
 *   mean_bg = sum x / (S D),  var_bg = sum (x - mean_bg)^2 / (S D)  (biased)
 *   rstd_bg = 1 / sqrt(var_bg + eps)
 *   y = act((x - mean_bg) * rstd_bg * gamma_c + beta_c)
 * x, gamma, beta, y of `dtype`; mean, rstd fp32 [B, G], each may be NULL.
 * A group that holds an infinity or a NaN has NaN for mean, rstd and y.
 * y may be x itself (same pitches); any other overlap is undefined.
 * `workspace`: device memory of the caller, 16-byte aligned, of at least
 * gn_workspace_bytes() (may be NULL when that is 0); nothing in it needs a
 * value before the call. Calls that share a workspace must not overlap on
 * the GPU (two captured graphs that were given the same one included).
 */
norm_status gn_fwd(const void* x, int64_t x_batch, int64_t x_row, const void* gamma, const void* beta, void* y,
                   int64_t y_batch, int64_t y_row, float* mean, float* rstd, void* workspace, size_t workspace_bytes,
                   int64_t B, int64_t S, int64_t C, int64_t G, float eps, norm_act act, norm_dtype dtype,
                   cudaStream_t stream);

/*
 * Group norm backward, from gn_fwd's statistics (fp32 [B, G]):
 *   xhat = (x - mean_bg) * rstd_bg,  z = xhat * gamma_c + beta_c,  dz = dy * act'(z),  g = dz * gamma_c
 *   dx = rstd_bg * (g - mean(g) - xhat * mean(g * xhat)), means over the S D values of the group
 *   dgamma_c = sum_bs dz * xhat,  dbeta_c = sum_bs dz          (fp32 [C], always written)
 * dx may be dy or x itself (same pitches); any other overlap is undefined.
 * The sums are added in a fixed order: results are deterministic for a plan.
 */
norm_status gn_bwd(const void* dy, int64_t dy_batch, int64_t dy_row, const void* x, int64_t x_batch, int64_t x_row,
                   const void* gamma, const void* beta, const float* mean, const float* rstd, void* dx,
                   int64_t dx_batch, int64_t dx_row, float* dgamma, float* dbeta, void* workspace,
                   size_t workspace_bytes, int64_t B, int64_t S, int64_t C, int64_t G, norm_act act, norm_dtype dtype,
                   cudaStream_t stream);

/* The plan gn_fwd (backward == 0) or gn_bwd would choose on a device with
 * `num_sms` SMs; vec_elems: the widest access the call's tensors allow (see
 * above). Host only: makes no CUDA call. */
norm_status gn_make_plan(int64_t B, int64_t S, int64_t C, int64_t G, norm_dtype dtype, int backward, int vec_elems,
                         int num_sms, gn_plan* plan);

/* Workspace bytes of a plan; plan == NULL: enough for whichever plan the
 * calls choose on a device with `num_sms` SMs, at any alignment. Host only. */
norm_status gn_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G, norm_dtype dtype, int backward,
                               int num_sms, const gn_plan* plan, size_t* bytes);

/* The calls with an explicit plan (NULL: choose), checked against the call
 * on the host; NORM_ERR_PLAN if it does not fit. */
norm_status gn_fwd_planned(const void* x, int64_t x_batch, int64_t x_row, const void* gamma, const void* beta,
                           void* y, int64_t y_batch, int64_t y_row, float* mean, float* rstd, void* workspace,
                           size_t workspace_bytes, int64_t B, int64_t S, int64_t C, int64_t G, float eps,
                           norm_act act, norm_dtype dtype, cudaStream_t stream, const gn_plan* plan);

norm_status gn_bwd_planned(const void* dy, int64_t dy_batch, int64_t dy_row, const void* x, int64_t x_batch,
                           int64_t x_row, const void* gamma, const void* beta, const float* mean, const float* rstd,
                           void* dx, int64_t dx_batch, int64_t dx_row, float* dgamma, float* dbeta, void* workspace,
                           size_t workspace_bytes, int64_t B, int64_t S, int64_t C, int64_t G, norm_act act,
                           norm_dtype dtype, cudaStream_t stream, const gn_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* LIBNORM_GROUP_H */
