/*
 * moe_layer.h -- the operators around the shuffle of moe_shuffle.h that a
 * Mixture-of-Experts layer computes on one MI355X (gfx950), and the gradients
 * of the layer.  Same library, plans, statuses and conventions.
 *
 *   moe_router                  gate logits -> topk_idx, topk_w of a plan
 *   moe_expert_linear           every expert's matrix product on its rows of
 *                               the receive layout, with bias, activation and
 *                               residual in its epilogue
 *   moe_combine_backward        gradient of moe_combine (and moe_combine_hier)
 *   moe_expert_linear_backward  gradient of moe_expert_linear
 *   moe_dispatch_backward       gradient of moe_dispatch
 *   moe_router_backward         gradient of moe_router
 *
 * A training step calls moe_router, moe_route_plan, moe_dispatch,
 * moe_expert_linear (once for each product), moe_combine, then the backward
 * calls in the order above.  Arguments are device buffers owned by the caller,
 * row-major and contiguous, 16-byte aligned unless said otherwise; calls are
 * asynchronous on the stream, allocate nothing and never synchronise.  Nothing
 * uses atomics on floating values: the same inputs give the same bits.  Every
 * buffer that a call reads or writes is distinct from those it writes.
 * Host-detectable errors return before anything is launched.  An empty batch
 * (T = 0) launches nothing, except that gradients of weights and biases are
 * then filled with zeros.
 *
 * Slots dropped for bad routing (moe_shuffle.h, "Errors") add nothing here
 * either; receive rows that no slot owns are neither read nor written.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_shuffle.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- router -------------------------------------------------------------- */

typedef enum moe_score {
  MOE_SCORE_SOFTMAX = 0, /* p = softmax of the token's E logits */
  MOE_SCORE_SIGMOID = 1  /* p = 1 / (1 + exp(-logit))           */
} moe_score;

typedef enum moe_router_key {
  MOE_KEY_LOGIT = 0, /* experts are chosen by their logits             */
  MOE_KEY_SCORE = 1  /* by their scores p, as float32 computes them    */
} moe_router_key;

typedef struct moe_router_config {
  int32_t score;           /* moe_score                                                  */
  int32_t renormalise;     /* nonzero: the k selected scores are divided by their sum    */
  int32_t nodes_per_token; /* 0: any expert.  m > 0: only experts of the token's m best
                              nodes (the plan's N = R / G nodes), a node's worth being the
                              float32 sum of its two largest keys; ties to the lower node */
  float scale;             /* the weights are multiplied by this                         */
  int32_t key;             /* moe_router_key                                             */
} moe_router_config;

/* Router: key[e] = logit[e] or p[e] (+ bias[e], added in float32); the experts
 * of the k largest keys, in descending order, ties to the lower id, are
 * topk_idx[t]; topk_w[t, j] = scale * p[id_j] (/ sum over the k selected p).
 * The bias only takes part in the choice; p is of the logits alone.
 * Scores rise with the logits, so that without a bias and a limit of the nodes
 * both keys choose alike, up to scores that float32 rounds to one value.  With
 * either they do not: a bias is added to what it was adjusted for.  Balancing
 * without an auxiliary loss adjusts it for the scores, and the node-limited
 * routing of DeepSeek-V3 sums a node's two largest biased sigmoid scores:
 * MOE_SCORE_SIGMOID with MOE_KEY_SCORE.
 * With either key a logit of -infinity has the key -infinity.
 * A NaN key ranks below -infinity, and a NaN logit has p = 0.  Where all the
 * scores of a sum are 0 (all logits -infinity), the weights are 0.  An
 * infinite maximum logit stands for the limit: p is shared by the logits that
 * are +infinity.
 * logits: [T, E] float32 or bf16 (logits_dtype: moe_out_dtype), aligned to its
 * element; bias: [E] float32 or NULL; topk_idx [T, k] int32 and topk_w [T, k]
 * float32, 4-byte aligned, as moe_route_plan and moe_combine take them.  The
 * plan need not be routed.  Limits: with nodes_per_token m > 0, N <= 64 nodes.
 * Errors: INVALID_ARGUMENT (null or misaligned pointers, unknown score, key or
 * dtype, m < 0 or m > N, fewer than k experts on the m smallest nodes, a scale
 * that is not finite), UNSUPPORTED (N > 64 with m > 0), HIP. */
moe_status moe_router(moe_plan* plan, const moe_router_config* cfg, const void* logits,
                      int32_t logits_dtype, const float* bias, int32_t* topk_idx, float* topk_w,
                      void* stream);

/* Gradient of the weights with respect to the logits, the choice being fixed:
 * grad_w [T, k] float32 -> grad_logits [T, E] of logits_dtype, every entry
 * written.  topk_idx: the ids moe_router chose (an id outside [0, E) adds
 * nothing, a repeated one adds its gradients).  The bias and the nodes have no
 * gradient.  Errors as moe_router. */
moe_status moe_router_backward(moe_plan* plan, const moe_router_config* cfg, const void* logits,
                               int32_t logits_dtype, const int32_t* topk_idx, const float* grad_w,
                               void* grad_logits, void* stream);

/* ---- gradients of the shuffle --------------------------------------------- */

/* Gradient of the dispatch: grad_x[t] = sum_j grad_recv[slot_of[t, j]], added
 * in float32 in ascending j, then rounded to bf16 (nearest even) or stored as
 * float32.  grad_recv: [T*k, H] bf16 in the receive layout; grad_x: [T, H] of
 * out_dtype.  Any plan (banded and node-deduplicated ones too: the staging hop
 * copies).  Errors: PLAN_NOT_ROUTED, INVALID_ARGUMENT, HIP. */
moe_status moe_dispatch_backward(moe_plan* plan, const uint16_t* grad_recv, void* grad_x,
                                 int32_t out_dtype, void* stream);

/* Gradient of moe_combine (and of moe_combine_hier, the same function):
 *   grad_y[slot_of[t, j]] = topk_w[t, j] * grad_out[t], rounded to bf16;
 *   grad_w[t, j] = sum_h grad_out[t, h] * y[slot_of[t, j], h], float32 fused
 *                  multiply-adds in a fixed order (0 for a dropped slot).
 * grad_out: [T, H] of grad_dtype (moe_out_dtype); y, grad_y: [T*k, H] bf16 in
 * the receive layout; topk_w, grad_w: [T, k] float32, 4-byte aligned.
 * Errors: PLAN_NOT_ROUTED, INVALID_ARGUMENT, HIP. */
moe_status moe_combine_backward(moe_plan* plan, const void* grad_out, int32_t grad_dtype,
                                const uint16_t* y, const float* topk_w, uint16_t* grad_y,
                                float* grad_w, void* stream);

/* ---- the experts' products -------------------------------------------------- */

typedef enum moe_activation {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_SILU = 2,   /* z / (1 + exp(-z))                          */
  MOE_ACT_GELU = 3,   /* z * Phi(z), Phi the normal distribution    */
  MOE_ACT_SWIGLU = 4, /* silu(z[:N]) * z[N:], a product of width 2N */
  MOE_ACT_GEGLU = 5   /* gelu(z[:N]) * z[N:]                        */
} moe_activation;

typedef struct moe_expert_config {
  int32_t in_features;  /* K > 0, multiple of 8: width of x                          */
  int32_t out_features; /* N > 0, multiple of 8: width of y                          */
  int32_t activation;   /* moe_activation.  Z = 2N for the gated ones, else N        */
} moe_expert_config;

/* Expert product: for every receive row r of expert e,
 *   z[r] = x[r] . w[e]^T + bias[e]        (float32 accumulation)
 *   y[r] = act(z[r]) + residual[r]        rounded to bf16 (nearest even)
 *   pre[r] = z[r] rounded to bf16         (kept for the gradient)
 * x: [T*k, K] bf16; w: [E, Z, K] bf16; bias: [E, Z] float32 or NULL; residual:
 * [T*k, N] bf16 or NULL; y: [T*k, N] bf16; pre: [T*k, Z] bf16 or NULL.
 * K and N are the product's own (not the plan's H).  Banded plans are computed
 * band by band, a launch each.  Limits: Z * K < 2^30, K and Z <= 2^20.
 * Errors: PLAN_NOT_ROUTED, INVALID_ARGUMENT, UNSUPPORTED (sizes beyond the
 * limits), HIP. */
moe_status moe_expert_linear(moe_plan* plan, const moe_expert_config* cfg, const uint16_t* x,
                             const uint16_t* w, const float* bias, const uint16_t* residual,
                             uint16_t* y, uint16_t* pre, void* stream);

/* Device workspace of moe_expert_linear_backward (bytes, a multiple of 256; 0
 * for a cfg that the call refuses): the gradient of z in bf16 with an
 * activation, and the partial sums of the bias gradient.  Its contents need no
 * initialisation. */
size_t moe_expert_backward_workspace_bytes(const moe_plan* plan, const moe_expert_config* cfg);

/* Gradient of moe_expert_linear, with grad_z = grad_y * act'(pre) (gated:
 * [grad_y * up * act'(gate), grad_y * act(gate)]):
 *   grad_x[r] = grad_z[r] . w[e]                       bf16 [T*k, K]
 *   grad_w[e] = sum over e's rows of grad_z[r]^T x[r]  [E, Z, K] of w_dtype
 *   grad_bias[e] = sum over e's rows of grad_z[r]      float32 [E, Z]
 * Each may be NULL (not wanted); an expert without rows gets zeros.  With an
 * activation grad_z is rounded to bf16 for the two products, which the matrix
 * cores take as bf16 (grad_bias sums it unrounded).  The residual's gradient is
 * grad_y.  grad_y: [T*k, N] bf16; pre: [T*k, Z] bf16 as moe_expert_linear
 * stored it (ignored without an activation); x is read for grad_w only and w
 * for grad_x only, and may be NULL without it; w_dtype: moe_out_dtype of
 * grad_w; workspace: 256-byte aligned.
 * Errors as moe_expert_linear. */
moe_status moe_expert_linear_backward(moe_plan* plan, const moe_expert_config* cfg,
                                      const uint16_t* grad_y, const uint16_t* x, const uint16_t* w,
                                      const uint16_t* pre, uint16_t* grad_x, void* grad_w,
                                      int32_t w_dtype, float* grad_bias, void* workspace,
                                      void* stream);

/* Kernels of these calls, as moe_plan_timing_read names them (ids after those
 * of moe_kernel; moe_kernel_name takes both). */
typedef enum moe_layer_kernel {
  MOE_KERNEL_ROUTER = MOE_KERNEL_COUNT,
  MOE_KERNEL_ROUTER_GRAD,
  MOE_KERNEL_DISPATCH_GRAD,
  MOE_KERNEL_COMBINE_GRAD,
  MOE_KERNEL_EXPERT_ROWS,      /* product of receive rows with expert weights            */
  MOE_KERNEL_EXPERT_FEW_ROWS,  /* the same for batches of few rows an expert             */
  MOE_KERNEL_EXPERT_ROWS_GRAD, /* product of grad_z with expert weights: grad_x          */
  MOE_KERNEL_EXPERT_WGRAD,     /* product over an expert's rows: grad_w                  */
  MOE_KERNEL_EXPERT_GRADS,     /* both of them, and few bias sums, where both are wanted */
  MOE_KERNEL_EXPERT_ACT_GRAD,  /* grad_z, and partial sums of the bias gradient          */
  MOE_KERNEL_EXPERT_BIAS_SUM,  /* the partial sums added up                              */
  MOE_LAYER_KERNEL_END
} moe_layer_kernel;

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
