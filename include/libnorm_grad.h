/*
 * libnorm - the global norm of a list of gradients, and clipping by it, for
 * NVIDIA GB300 (sm_103a). Part of the same library as libnorm.h, whose
 * conventions hold here too.
 */
#ifndef LIBNORM_GRAD_H
#define LIBNORM_GRAD_H

#include "libnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One gradient: `numel` values of `dtype` one after the other in device
 * memory (any order of the dimensions: nothing but the values counts). The
 * array of these is host memory, read during the call only. */
typedef struct {
    const void* data;  /* may be NULL where numel is 0 */
    void* out;         /* grad_clip: where the clipped values go (data itself: in place); unused by grad_norm */
    int64_t numel;     /* >= 0, < 2^46 */
    int32_t dtype;     /* norm_dtype */
    int32_t reserved;  /* 0 */
} norm_tensor;

/*
 * norm = sqrt(sum over all tensors of v^2), one fp32 value in device memory.
 * Squares are added in fp32 over at most 64 values of a thread (short lists:
 * over a warp's), and beyond in fp64 or in pairs of fp32 numbers that keep
 * every addition's error; where fp32 squares leave the range (values above
 * 2^60 or sums below 2^-80) that part is summed again in fp64, so the norm is
 * right wherever it fits fp32, infinite or NaN where a value is. A tensor that
 * is listed twice counts twice. No tensors (or only empty ones): 0.
 * `workspace`: 8-byte aligned device memory of the caller, at least
 * grad_workspace_bytes() (may be NULL when that is 0); nothing in it needs a
 * value before the call. Calls that share a workspace must not overlap on the
 * GPU. The sums are added in a
 * fixed order: the same tensors give the same bits on one device.
 */
norm_status grad_norm(const norm_tensor* tensors, int64_t count, float* norm, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream);

/*
 * norm as above; coef = max_norm / (norm + 1e-6), 1 where that is above 1;
 * out = v * coef, formed in fp32 and rounded once to the tensor's type. A
 * norm that is infinite gives coef 0, and a NaN norm NaN, as the formula
 * says: the caller who wants to skip such a step reads `norm`. With coef 1,
 * tensors clipped in place are not touched. Each `out` is its tensor's `data`
 * itself or apart from every other data and out of the list, and `norm` is
 * apart from all of them; overlaps return NORM_ERR_ARG. max_norm: finite and
 * >= 0.
 */
norm_status grad_clip(const norm_tensor* tensors, int64_t count, float max_norm, float* norm, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes for these tensors on a device with `num_sms` SMs, by their
 * sizes, types and number (a short list needs none). Host only: makes no CUDA
 * call. */
norm_status grad_workspace_bytes(const norm_tensor* tensors, int64_t count, int num_sms, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* LIBNORM_GRAD_H */
