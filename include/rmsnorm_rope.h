/*
 * rmsnorm_rope.h -- C ABI of librmsnorm.so, continued: the per-head QK norm
 * with a position rotation in the same pass, the same with keys and values
 * appended to a paged cache, and the gradients of the norms.
 *
 * Contexts, statuses, element types, asynchrony and threads are those of
 * rmsnorm.h.  Structures are read during the call only.
 */
#ifndef RMSNORM_ROPE_H
#define RMSNORM_ROPE_H

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further status (rmsnorm_status_t): a position outside the rotation table
 * or a slot outside the cache, found on the device (device status word). */
enum { RMSNORM_ERR_BAD_INDEX = 11 };

/* The heads of one tensor: head h of token t is the head_dim contiguous
 * elements from element t * token_stride + h * head_stride of `data` (a
 * DEVICE pointer).  A stride of 0 stands for the contiguous layout [tokens,
 * heads, head_dim]: head_stride = head_dim, token_stride = heads *
 * head_stride.  Strides let the heads be views into a fused QKV buffer (by
 * tensor, or head by head) or lie head-major ([heads, tokens, head_dim]).
 * They are >= 0, and no two heads of a tensor may share an element. */
typedef struct {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} rmsnorm_heads_t;

/* The position rotation.  Row p of the table `cos_sin` (DEVICE, fp32,
 * [max_position, rotary_dim], contiguous) holds the cosines of position p's
 * rotary_dim / 2 angles, then their sines; token t takes row positions[t]
 * (DEVICE, int64).  The first rotary_dim elements of a head are rotated (an
 * even number from 0 to head_dim; 0: no rotation, both pointers unused):
 * element i with element i + rotary_dim / 2, or, with `interleaved`, element
 * 2i with element 2i + 1:
 *   y_a = u_a cos_i - u_b sin_i,   y_b = u_b cos_i + u_a sin_i.
 * A position outside [0, max_position) is found on the device: the token is
 * left out (nothing of it is written, and it adds nothing to a weight's
 * gradient) and RMSNORM_ERR_BAD_INDEX is recorded in the device
 * status word (rmsnorm_get_device_status). */
typedef struct {
    const float *cos_sin;
    const int64_t *positions;
    int64_t max_position;
    int32_t rotary_dim;
    int32_t interleaved; /* 0 or 1 */
} rmsnorm_rope_t;

/* Per-head QK norm and rotation in one pass: for every head of q and of k
 *   u[d] = (x[d] * rsqrt(sum_e x[e]^2 / head_dim + eps)) * (w[d] + weight_bias)
 *   y    = round(rotate(u))                     (fp32 inside, one rounding)
 * with q_weight for q and k_weight for k, q and k in one launch.
 *   q, k          inputs; with no heads (q_heads or k_heads 0) NULL is allowed
 *   q_out, k_out  outputs; NULL writes in place.  An output may be exactly its
 *                 input (same data and strides); any other overlap of an output
 *                 with an input or output is RMSNORM_ERR_ALIASING (layouts that
 *                 interleave with different strides count as overlapping).
 *   q_weight, k_weight  DEVICE, [head_dim] of `dtype`; may be equal
 *   head_dim      1 .. 1024;  tokens >= 0;  weight_bias finite;  eps >= 0, finite
 * Heads that can be read in vectors of 16, 8 or 4 bytes (data, weights,
 * strides and the table on such boundaries, head_dim and rotary_dim multiples of
 * two vectors' elements) take a vector kernel, others a scalar one.
 * Enqueues one kernel on `stream`; does not synchronise.  Returns RMSNORM_OK,
 * RMSNORM_ERR_INVALID_ARG, RMSNORM_ERR_UNSUPPORTED_DTYPE,
 * RMSNORM_ERR_MISALIGNED (a pointer that is not on an element's boundary),
 * RMSNORM_ERR_ALIASING, RMSNORM_ERR_NOT_INITIALIZED or RMSNORM_ERR_CUDA. */
int rmsnorm_qk_norm_rope(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k,
                         const rmsnorm_heads_t *q_out, const rmsnorm_heads_t *k_out,
                         const void *q_weight, const void *k_weight, const rmsnorm_rope_t *rope,
                         int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                         float weight_bias, float eps, int dtype, void *stream);

/* The gradient of rmsnorm_qk_norm_rope.  With dy the gradient of an output
 * head, x its input, r = rsqrt(mean(x^2) + eps), g = w + weight_bias, n =
 * head_dim:
 *   du = rotate back(dy),  xh = x * r
 *   dx = round( r * (du * g - xh * sum_e(du[e] g[e] xh[e]) / n) )
 *   dw = sum over tokens and heads of du * xh
 * in fp32, dw in a fixed order (the same inputs give the same bits).
 *   dq_out, dk_out  gradients of the outputs, of `dtype`
 *   q, k            the inputs the forward call was given (not its outputs)
 *   dq, dk          gradients of the inputs, of `dtype`; may be exactly dq_out /
 *                   dk_out or exactly q / k, else may overlap nothing
 *   dq_weight, dk_weight  DEVICE, fp32 [head_dim]; NULL (both) skips them
 *   workspace       DEVICE, 16-byte aligned, the caller's; at least the bytes
 *                   rmsnorm_qk_norm_rope_bwd_workspace gives; unused (may be
 *                   NULL) when the weights' gradients are skipped.  Calls that may
 *                   run at the same time need a workspace each.
 * A tensor with no heads gets a zero weight gradient.  Enqueues one kernel,
 * and a second small one for the weights' gradients.  Otherwise as
 * rmsnorm_qk_norm_rope; RMSNORM_ERR_MISALIGNED for the workspace, too. */
int rmsnorm_qk_norm_rope_bwd(const rmsnorm_heads_t *dq_out, const rmsnorm_heads_t *dk_out,
                             const rmsnorm_heads_t *q, const rmsnorm_heads_t *k,
                             const rmsnorm_heads_t *dq, const rmsnorm_heads_t *dk,
                             const void *q_weight, const void *k_weight, float *dq_weight,
                             float *dk_weight, const rmsnorm_rope_t *rope, void *workspace,
                             size_t workspace_bytes, int64_t tokens, int64_t q_heads,
                             int64_t k_heads, int64_t head_dim, float weight_bias, float eps,
                             int dtype, void *stream);

/* Workspace bytes rmsnorm_qk_norm_rope_bwd needs for a head size on a device
 * with `sm_count` SMs, whatever the other sizes (host only). */
int rmsnorm_qk_norm_rope_bwd_workspace(int64_t head_dim, int sm_count, size_t *bytes);

/* A paged cache of keys and values: element d of head h in slot s of page p is
 * element p * page_stride + s * slot_stride + h * head_stride + d of `k`
 * (and of `v`), both DEVICE pointers, so that pages may hold their slots
 * head by head or slot by slot.  Strides of 0 (all three) stand for the
 * contiguous [pages, page_size, k_heads, head_dim]. */
typedef struct {
    void *k;
    void *v;
    int64_t pages;
    int64_t page_size;
    int64_t page_stride;
    int64_t slot_stride;
    int64_t head_stride;
    int32_t e4m3;  /* 0: elements of the call's dtype; 1: E4M3 bytes */
    float k_scale; /* E4M3: a value is stored as E4M3(value * (1 / scale)), 1 / scale in fp32, */
    float v_scale; /* nearest-even, saturating at +-448 (NaN stays NaN); scale and its
                    * reciprocal positive and finite */
} rmsnorm_paged_cache_t;

/* rmsnorm_qk_norm_rope with the keys and values appended to a paged cache in
 * the same launch: q is normalised and rotated into q_out (NULL: in place),
 * k is normalised and rotated into the cache (one rounding, to the cache's
 * type; k itself is left as it was), v is copied there (or rounded to E4M3).
 * Token t goes to slot slots[t] % page_size of page slots[t] / page_size
 * (DEVICE, int64).  A negative slot marks padding: nothing of the token is
 * written, its q_out row included, and its values and position have no effect.  A slot
 * beyond the cache leaves the token out and records RMSNORM_ERR_BAD_INDEX, as
 * a position outside the table does.  The non-negative slots of one call must
 * differ: which of two tokens in one slot remains is not defined, byte by
 * byte.
 *   q_weight, k_weight  both NULL: no norm, the rotation alone
 *   q may have no heads (q_heads 0, q NULL); k_heads >= 1
 * Cache bytes may overlap none of the other arguments.  Otherwise as
 * rmsnorm_qk_norm_rope. */
int rmsnorm_qk_norm_rope_append(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k,
                                const rmsnorm_heads_t *v, const rmsnorm_heads_t *q_out,
                                const void *q_weight, const void *k_weight,
                                const rmsnorm_rope_t *rope, const rmsnorm_paged_cache_t *cache,
                                const int64_t *slots, int64_t tokens, int64_t q_heads,
                                int64_t k_heads, int64_t head_dim, float weight_bias, float eps,
                                int dtype, void *stream);

/* The gradient of rmsnorm_fwd_bias (of rmsnorm_fwd with weight_bias -0 or 0).
 * With g = w + weight_bias, r = rsqrt(mean(x^2) + eps) and xh = x * r per row:
 *   dx = round( r * (dy * g - xh * sum_j(dy[j] g[j] xh[j]) / hidden) )
 *   dw = sum over rows of dy * xh
 * in fp32, dw in a fixed order (the same inputs give the same bits).
 *   dy, x, dx  DEVICE, [rows, hidden] of `dtype`, contiguous; dx may be exactly
 *              dy or exactly x, else may overlap nothing
 *   weight     DEVICE, [hidden] of `dtype`
 *   dweight    DEVICE, fp32 [hidden] (zeroed when rows is 0); NULL skips it
 *   workspace  DEVICE, 16-byte aligned, the caller's; at least the bytes
 *              rmsnorm_bwd_workspace gives.  Calls that may run at the same time
 *              need a workspace each.
 * The statistic is formed as in rmsnorm_fwd, over the types' whole range.
 * Enqueues one kernel on `stream`, and a second small one for dweight (rows too
 * long for the registers, of more than 8192 or 16384 elements: up to four); does
 * not synchronise.  Returns the statuses of rmsnorm_fwd; RMSNORM_ERR_INVALID_ARG
 * for a workspace that is too small, RMSNORM_ERR_MISALIGNED for one that is not
 * 16-byte aligned. */
int rmsnorm_bwd(const void *dy, const void *x, const void *weight, void *dx, float *dweight,
                void *workspace, size_t workspace_bytes, int64_t rows, int64_t hidden,
                float weight_bias, float eps, int dtype, void *stream);

/* Workspace bytes rmsnorm_bwd needs on a device with `sm_count` SMs (host
 * only). */
int rmsnorm_bwd_workspace(int64_t rows, int64_t hidden, int dtype, int sm_count, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_ROPE_H */
