/*
 * libnorm - dropout, residual add and norm in one pass, forward and backward,
 * and the backward of the fused residual add + norm, for NVIDIA GB300
 * (sm_103a). Part of the same library as libnorm.h, whose conventions hold
 * here too (contiguous [M, N] rows, device pointers owned by the caller,
 * asynchronous work on `stream`, argument errors detected on the host before
 * any CUDA call, fp32 arithmetic, nearest-even output rounding).
 *
 * The mask. Value e = row * N + column of the flattened [M, N] tensor has the
 * 16-bit word e % 8 (word 2 i the low half of output i, word 2 i + 1 its high
 * half) of Philox4x32-7 with the counter (e / 8, offset), 64 bits each, and
 * the key `seed` (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
 * easy as 1, 2, 3", 2011: the counter-based generator with the 7 rounds that
 * they find to pass every test). With t = round(65536 p) it is dropped where
 * its word is below t; what is kept is multiplied by 65536 / (65536 - t), the
 * inverse of the exact probability of being kept. The mask depends on seed,
 * offset, p, e and nothing else (not on the type, the alignment or the launch),
 * and is never stored: the backward makes it again from the same arguments. A
 * program gives every call of a step, and every step, an offset of its own.
 */
#ifndef LIBNORM_DROPOUT_H
#define LIBNORM_DROPOUT_H

#include "libnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Where a call's random numbers come from. `device`: two 64-bit words (seed,
 * offset) in device memory, 8-byte aligned, read when the kernel runs, so that
 * a captured graph takes a new mask for each replay; NULL: the two values
 * here. */
typedef struct {
    uint64_t seed, offset;
    const uint64_t* device;
} norm_rng;

/*
 * Forward:
 *   h = residual + x * keep / P(keep), rounded to `dtype` (one rounding after
 *       an fp32 fused multiply-add); a dropped x is not looked at
 *   y (and mean, rstd fp32 [M], each may be NULL) = ln_fwd / rms_fwd of h
 * x, residual, h, y: [M, N] of `dtype`; gamma, beta, w: [N] of `dtype`.
 * h and y may each be x or residual itself; h and y must differ; any other
 * overlap is undefined. 0 <= p and round(65536 p) < 65536; with p = 0 rng is
 * not looked at and h, y are those of the plain fused add, to the rounding of
 * the statistics.
 * Limits: 1 <= N <= 65536 where every pointer is 16-byte aligned and the rows
 * are whole 16-byte vectors, N <= 65520 where they are not, N <= 32768 where a
 * pointer is not 16-byte aligned; longer rows return NORM_ERR_ARG.
 * Every pointer needs its element's alignment.
 */
norm_status ln_fwd_dropout_add(const void* x, const void* residual, const void* gamma, const void* beta, double p,
                               const norm_rng* rng, void* h, void* y, float* mean, float* rstd, int64_t M, int64_t N,
                               float eps, norm_dtype dtype, cudaStream_t stream);

norm_status rms_fwd_dropout_add(const void* x, const void* residual, const void* w, double p, const norm_rng* rng,
                                void* h, void* y, int64_t M, int64_t N, float eps, norm_dtype dtype,
                                cudaStream_t stream);

/*
 * Backward, from h (the forward's output), the gradients dy of y and dh of h
 * (what reaches the sum from elsewhere; NULL: nothing does), and, for
 * LayerNorm, mean and rstd:
 *   d         = dh + the norm's gradient of its input (as ln_bwd / rms_bwd)
 *   dresidual = d
 *   dx        = d * keep / P(keep)
 *   dgamma, dbeta, dw: fp32 [N], always written, as ln_bwd / rms_bwd
 * dx and dresidual are each rounded once from fp32. Each may be dy, dh or h
 * itself; the two must differ; any other overlap is undefined. `workspace`:
 * 16-byte aligned device memory of at least drop_workspace_bytes() (may be
 * NULL when that is 0); nothing in it needs a value before the call; calls
 * that share it must not overlap on the GPU (two captured graphs that were
 * given the same one included). The column sums are added in a fixed order:
 * results are deterministic for a plan. Limits as above.
 */
norm_status ln_bwd_dropout_add(const void* dy, const void* dh, const void* h, const void* gamma, const float* mean,
                               const float* rstd, double p, const norm_rng* rng, void* dx, void* dresidual,
                               float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes, int64_t M,
                               int64_t N, norm_dtype dtype, cudaStream_t stream);

norm_status rms_bwd_dropout_add(const void* dy, const void* dh, const void* h, const void* w, double p,
                                const norm_rng* rng, void* dx, void* dresidual, float* dw, void* workspace,
                                size_t workspace_bytes, int64_t M, int64_t N, float eps, norm_dtype dtype,
                                cudaStream_t stream);

/* The backward of ln_fwd_add / rms_fwd_add: the same without dropout, one
 * gradient d for x and the residual alike. */
norm_status ln_bwd_add(const void* dy, const void* dh, const void* h, const void* gamma, const float* mean,
                       const float* rstd, void* d, float* dgamma, float* dbeta, void* workspace,
                       size_t workspace_bytes, int64_t M, int64_t N, norm_dtype dtype, cudaStream_t stream);

norm_status rms_bwd_add(const void* dy, const void* dh, const void* h, const void* w, void* d, float* dw,
                        void* workspace, size_t workspace_bytes, int64_t M, int64_t N, float eps, norm_dtype dtype,
                        cudaStream_t stream);

/* The plan the calls would choose for M rows of N elements on a device with
 * `num_sms` SMs (fields of norm_plan: `mapping` NORM_MAP_GROUP with `group`
 * lanes of a warp per row, or NORM_MAP_CTA with `cluster` CTAs per row, or
 * teams of `group` threads of a CTA (0: all `threads` of it); `per_thread`
 * accesses of `vec_elems` elements per thread (vec_elems 1: of two elements),
 * which cover the row and, where rows are no whole number of vectors, up to
 * vec_elems - 1 elements before it; `rounds` rows at a time; `stages` steps of
 * them in shared memory, up to 4, from 2 on 16-byte vectors, from 3 on
 * elements; `grid` CTAs at most, persistent, whose teams are a multiple of the
 * 1, 2, 4 or 8 rows after which one begins at the same place of a vector).
 * `aligned16`: every pointer is 16-byte aligned. Host only: makes no CUDA
 * call. NORM_ERR_ARG for rows beyond the limits. */
norm_status drop_make_plan(int64_t M, int64_t N, norm_dtype dtype, int layer_norm, int backward, int aligned16,
                           int num_sms, norm_plan* plan);

/* Workspace bytes of the backward: with a plan, its own; plan == NULL: enough
 * for whichever plan the call chooses on a device with `num_sms` SMs, at any
 * alignment. Host only. */
norm_status drop_workspace_bytes(int64_t M, int64_t N, norm_dtype dtype, int layer_norm, int num_sms,
                                 const norm_plan* plan, size_t* bytes);

/* The calls with an explicit plan (NULL: choose), checked against the call on
 * the host; NORM_ERR_PLAN if it does not fit. gamma is the RMSNorm's w where
 * layer_norm is 0 (beta, mean, rstd, dbeta are then not looked at, and eps not
 * by the LayerNorm's backward). With p = 0 rng may be NULL, and dx too: it is
 * then not written. */
norm_status drop_fwd_planned(int layer_norm, const void* x, const void* residual, const void* gamma, const void* beta,
                             double p, const norm_rng* rng, void* h, void* y, float* mean, float* rstd, int64_t M,
                             int64_t N, float eps, norm_dtype dtype, cudaStream_t stream, const norm_plan* plan);

norm_status drop_bwd_planned(int layer_norm, const void* dy, const void* dh, const void* h, const void* gamma,
                             const float* mean, const float* rstd, double p, const norm_rng* rng, void* dx,
                             void* dresidual, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                             int64_t M, int64_t N, float eps, norm_dtype dtype, cudaStream_t stream,
                             const norm_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* LIBNORM_DROPOUT_H */
