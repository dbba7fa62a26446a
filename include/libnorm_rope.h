/*
 * libnorm - RMSNorm of every query and key head with the rotary position
 * rotation in the same pass, forward and backward, for NVIDIA GB300
 * (sm_103a). Part of the same library as libnorm.h, whose conventions hold
 * here too (device pointers owned by the caller, asynchronous work on
 * `stream`, argument errors detected on the host before any CUDA call, fp32
 * arithmetic, nearest-even output rounding, once, at the end).
 *
 * Per token t with position p and per head (D values x, weight w of D):
 *   r = 1 / sqrt(sum_i x_i^2 / D + eps),   z_i = x_i r w_i
 * and the first R values of z are rotated in R / 2 pairs (a, b) by the angle
 * whose cosine and sine are cos[p][i], sin[p][i] for pair i:
 *   y_a = z_a cos - z_b sin,   y_b = z_b cos + z_a sin
 * with (a, b) = (i, i + R / 2), or, `interleaved`, (2 i, 2 i + 1); y = z
 * elsewhere. Queries have their own heads and weight, keys theirs; both share
 * tokens, positions and tables.
 */
#ifndef LIBNORM_ROPE_H
#define LIBNORM_ROPE_H

#include "libnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of heads [B, S, heads, D]: element (b, s, h, i) is
 * data[b * batch + s * token + h * head + i], pitches in elements, of either
 * sign or 0 (outputs: no two elements may share an address). */
typedef struct {
    void* data; /* inputs are not written */
    int64_t batch, token, head;
} norm_heads;

/* Queries or keys of a call. The other one's tensors are not looked at where
 * heads is 0 (queries or keys alone). */
typedef struct {
    int64_t heads;
    const void* w;  /* [D] */
    norm_heads x;   /* [B, S, heads, D] */
    norm_heads dy;  /* backward: the gradient of the rotated heads */
    norm_heads y;   /* forward: the rotated heads; backward: dx */
    float* dw;      /* backward: [D], always written */
} norm_rope_side;

/* The angles: fp32 tables [P, R / 2] with rows `table_pitch` elements apart
 * (>= R / 2), and the token's positions. */
typedef struct {
    const float *cos, *sin;
    int64_t table_pitch, P; /* P >= 1 where R > 0 */
    const void* positions; /* [B * S] whole numbers of position_bytes each; NULL: token s of a sequence has position s */
    int32_t position_bytes; /* 8 or 4 (signed); ignored without positions */
    int32_t R;              /* values that rotate: even, 0 <= R <= D */
    int32_t interleaved;
    int32_t reserved;       /* 0 */
} norm_rope_angles;

/* A launch plan. A warp works on `heads` heads of each of 32 / lanes tokens. */
typedef struct {
    int32_t vec_elems; /* values per access: 16 / sizeof(element), 4 or 2 (16-bit types) or 1 */
    int32_t pairs;     /* pairs of accesses per lane */
    int32_t lanes;     /* lanes per head, a power of two, <= 32 */
    int32_t heads;     /* heads per warp and token, >= 1 */
    int32_t warps;     /* warps per CTA, 1..8 */
    int32_t few;       /* forward: 1: a warp has one task, without shared memory; 0: persistent, heads streamed */
    int64_t ctas;      /* persistent: CTAs of queries and keys together at most (fewer if fewer fit), >= 2 */
} norm_rope_plan;

/*
 * Forward. A token whose position is negative is padding: its outputs are
 * zeros, whatever its heads (which may be read all the same), the weight and
 * the tables hold, and for every eps. One whose position is P or beyond has no
 * angle: its outputs are NaN (nothing beyond the tables is read). Outputs
 * may be the inputs themselves (same data and pitches); any other overlap is
 * undefined. Limits: 1 <= D <= 512, B, S, heads >= 0, B * S < 2^31,
 * heads < 2^20, pitches below 2^40 in magnitude, B * S * heads * D < 2^62,
 * eps finite and >= 0. Every pointer needs its element's alignment. 16-byte
 * accesses are used when every tensor, weight and pitch is a multiple of 16
 * bytes, as are D and, not interleaved, R / 2, or, interleaved, R; 8- or 4-byte
 * accesses of 16-bit values when the same holds for 8 or 4 bytes; element
 * accesses otherwise.
 */
norm_status rms_fwd_rope(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles, int64_t B,
                         int64_t S, int64_t D, float eps, norm_dtype dtype, cudaStream_t stream);

/*
 * Backward, from the forward's inputs (r is recomputed: no statistics are
 * saved). With dz = dy rotated back by the same angle and g = dz w:
 *   dx_i = r (g_i - x_i r^2 sum_j g_j x_j / D),   dw_i = sum over tokens and heads of dz_i x_i r
 * Padding tokens get dx = 0 and add nothing to dw; positions of P or beyond
 * give NaN in dx and dw. dx may be dy or x itself (same data and pitches);
 * any other overlap is undefined. `workspace`: 16-byte aligned device memory
 * of at least rope_workspace_bytes() (may be NULL when that is 0); nothing in
 * it needs a value before the call; calls that share it must not overlap on
 * the GPU (two captured graphs that were given the same one included). The
 * sums are added in a fixed order: results are deterministic for a plan.
 */
norm_status rms_bwd_rope(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles,
                         void* workspace, size_t workspace_bytes, int64_t B, int64_t S, int64_t D, float eps,
                         norm_dtype dtype, cudaStream_t stream);

/* The plan the calls would choose on a device with `num_sms` SMs for
 * `q_heads` and `k_heads` heads of D values, R of them rotating; vec_elems:
 * the widest access the call's tensors allow (see above). Host only: makes no
 * CUDA call. */
norm_status rope_make_plan(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t D, int64_t R, int interleaved,
                           norm_dtype dtype, int backward, int vec_elems, int num_sms, norm_rope_plan* plan);

/* Workspace bytes of the backward: with a plan, its own; plan == NULL: enough
 * for whichever plan the call chooses on a device with `num_sms` SMs. */
norm_status rope_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t D, int num_sms,
                                 const norm_rope_plan* plan, size_t* bytes);

/* The calls with an explicit plan (NULL: choose), checked against the call on
 * the host; NORM_ERR_PLAN if it does not fit. */
norm_status rms_fwd_rope_planned(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles,
                                 int64_t B, int64_t S, int64_t D, float eps, norm_dtype dtype, cudaStream_t stream,
                                 const norm_rope_plan* plan);

norm_status rms_bwd_rope_planned(const norm_rope_side* q, const norm_rope_side* k, const norm_rope_angles* angles,
                                 void* workspace, size_t workspace_bytes, int64_t B, int64_t S, int64_t D, float eps,
                                 norm_dtype dtype, cudaStream_t stream, const norm_rope_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* LIBNORM_ROPE_H */
