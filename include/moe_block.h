/*
 * moe_block.h -- what stands around the Mixture-of-Experts layer of
 * moe_layer.h in a transformer block on one MI355X (gfx950): the norm of the
 * residual stream in front of the router and the dispatch, with its gradient,
 * and the experts' products with weights of 4 bits for serving.  Same library,
 * plans, statuses and conventions.
 *
 *   moe_norm               residual addition, then layer norm or RMS norm
 *   moe_norm_backward      its gradient
 *   moe_weights4_pack      4-bit codes and scales -> packed weights
 *   moe_weights4_quantize  bf16 weights -> packed weights
 *   moe_weights4_unpack    the values that packed weights stand for
 *   moe_expert_linear4     moe_expert_linear with packed weights
 *
 * A decoding step calls moe_norm, moe_router on the gate's logits,
 * moe_route_plan, moe_dispatch, moe_expert_linear4 (once for each product) and
 * moe_combine, whose output is the residual of the next block's moe_norm.
 * Arguments, streams and errors as in moe_layer.h: contiguous device buffers
 * of the caller, 16-byte aligned unless said otherwise, distinct from those
 * the call writes; asynchronous, nothing is allocated, no atomics on floating
 * values.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- norm ------------------------------------------------------------------ */

typedef enum moe_norm_kind {
  MOE_NORM_LAYER = 0, /* the mean is taken off      */
  MOE_NORM_RMS = 1    /* mean = 0 in the formulas   */
} moe_norm_kind;

typedef struct moe_norm_config {
  int32_t kind;    /* moe_norm_kind                                       */
  float eps;       /* >= 0, finite; added to the variance                 */
  int32_t x_dtype; /* moe_out_dtype of x, residual, total and grad_x      */
  int32_t y_dtype; /* moe_out_dtype of y and grad_y                       */
} moe_norm_config;

/* Norm of the plan's T rows of H columns:
 *   total = x + residual             float32 sum, rounded to x_dtype
 *   mean  = sum(total) / H           (RMS: 0)
 *   rstd  = 1 / sqrt(sum((total - mean)^2) / H + eps)
 *   y     = (total - mean) * rstd * gamma + beta
 * in float32 from the rounded total, y rounded to y_dtype (nearest even).
 * x, residual, total: [T, H]; residual NULL: total = x, and total has to be
 * NULL.  total may be NULL with a residual too (not wanted).  gamma, beta: [H]
 * float32, NULL for ones and zeros.  y: [T, H].  stats: [T, 2] float32, mean
 * and rstd, as the gradient takes them, 8-byte aligned, or NULL.
 * A row whose sum of squares passes float32's range has rstd 0.  The plan need
 * not be routed; its experts take no part.  Limit: H <= 16384.
 * Errors: INVALID_ARGUMENT (null or misaligned pointers, unknown kind or
 * dtype, eps negative or not finite, a total without a residual), UNSUPPORTED
 * (H beyond the limit), HIP. */
moe_status moe_norm(moe_plan* plan, const moe_norm_config* cfg, const void* x, const void* residual,
                    const float* gamma, const float* beta, void* y, void* total, float* stats,
                    void* stream);

/* Device workspace of moe_norm_backward (bytes, a multiple of 256; it may be
 * 0): the partial sums of the weights' gradients.  Its contents need no
 * initialisation.  0 for a cfg that the call refuses. */
size_t moe_norm_backward_workspace_bytes(const moe_plan* plan, const moe_norm_config* cfg);

/* Gradient of moe_norm.  With h = (total - mean) * rstd and g = grad_y * gamma:
 *   grad_x = rstd * (g - mean_H(g) - h * mean_H(g * h)) + grad_total
 *            (RMS: without mean_H(g)), rounded to x_dtype
 *   grad_gamma = sum over the rows of grad_y * h        float32 [H]
 *   grad_beta  = sum over the rows of grad_y            float32 [H]
 * Each may be NULL (not wanted); without rows the sums are zeros.  grad_x is
 * the gradient of x and of the residual.  total: what was normed (x without a
 * residual); stats: as moe_norm stored them; grad_total: [T, H] of x_dtype,
 * the gradient that reaches total by other ways, or NULL; workspace: 256-byte
 * aligned, may be NULL where its size is 0.  cfg->eps is only checked.
 * Errors as moe_norm. */
moe_status moe_norm_backward(moe_plan* plan, const moe_norm_config* cfg, const void* grad_y,
                             const void* total, const float* stats, const float* gamma,
                             const void* grad_total, void* grad_x, float* grad_gamma,
                             float* grad_beta, void* workspace, void* stream);

/* Kernels of these calls, as moe_plan_timing_read names them (moe_kernel_name
 * takes their ids too). */
typedef enum moe_block_kernel {
  MOE_KERNEL_NORM = 64,
  MOE_KERNEL_NORM_GRAD,
  MOE_KERNEL_NORM_SUM,         /* partial sums of the weights' gradients added up */
  MOE_BLOCK_KERNEL_END
} moe_block_kernel;

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
