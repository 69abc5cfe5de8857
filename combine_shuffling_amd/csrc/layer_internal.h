// Internal declarations of the layer's operators (moe_layer_api.cpp and
// router.hip, shuffle_grad.hip, expert.hip).  Not part of the public ABI.
#pragma once

#include "moe_internal.h"
#include "moe_layer.h"

namespace moe {

// Nodes a node-limited router chooses among: one lane holds one node's worth.
constexpr int kRouterMaxNodes = 64;

// router.hip
hipError_t launch_router(const Dims& d, const moe_router_config& c, const void* logits, bool f32,
                         const float* bias, int32_t* topk_idx, float* topk_w, hipStream_t s);
hipError_t launch_router_grad(const Dims& d, const moe_router_config& c, const void* logits,
                              bool f32, const int32_t* topk_idx, const float* grad_w,
                              void* grad_logits, hipStream_t s);

// shuffle_grad.hip.  slot_of must be final.
hipError_t launch_dispatch_grad(const Dims& d, const uint16_t* grad_recv, void* grad_x, bool f32,
                                const Work& w, hipStream_t s);
hipError_t launch_combine_grad(const Dims& d, const void* grad_out, bool f32, const uint16_t* y,
                               const float* wts, uint16_t* grad_y, float* grad_w, const Work& w,
                               hipStream_t s);

// expert.hip.  Sizes of one expert product: `rows` receive rows (T * k), sorted
// by expert inside each band, off[b * (E + 1) + e] the experts' first rows (of
// all bands together, in order); K in, N out, Z = the width of the product
// itself.
struct ExpertDims {
  int32_t rows, E, K, N, Z;
  int32_t T;              // tokens: no expert has more rows
  int32_t act;            // moe_activation
  int32_t bands;          // 1: not banded
  int32_t band_tokens;    // tokens a band (the last may have fewer)
};
inline bool gated(int32_t act) { return act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU; }

// Rows per slot of the partial bias sums, and the slots: expert e's of band b
// start at off / kBiasRows + e + b * E (off: its first row), which leaves room
// for the rows of every expert without knowing their counts on the host.  A
// block of the activation's gradient takes one slot.  Against 64 rows, 32 took
// 14% off it for 4084 rows of 1000 columns (11 us) and 6% for 32768 of 2 x 1024 (70
// us), and added half to the bias sums of a Zipf batch (one expert of 8192 rows: 12.6
// to 19.5 us); 16 rows 25%, 8%, and 34.9 us.
constexpr int kBiasRows = 32;
inline int64_t bias_slots(const ExpertDims& x) {
  return x.rows / kBiasRows + (int64_t)x.bands * x.E;
}

hipError_t launch_expert_rows(const ExpertDims& x, const int32_t* off, const uint16_t* a,
                              const uint16_t* w, const float* bias, const uint16_t* residual,
                              uint16_t* y, uint16_t* pre, hipStream_t s);
hipError_t launch_expert_rows_grad(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                                   const uint16_t* w, uint16_t* gx, hipStream_t s);
hipError_t launch_expert_wgrad(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                               const uint16_t* a, void* gw, bool f32, hipStream_t s);
// Both, in one launch on a plan of one band, and the bias gradient from its
// partial sums (gb null: not wanted).
hipError_t launch_expert_grads(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                               const uint16_t* w, uint16_t* gx, const uint16_t* a, void* gw,
                               bool f32, const float* partial, float* gb, hipStream_t s);
// gz (bf16, null: not wanted) and partial (float32 [bias_slots, Z], null: not wanted).
hipError_t launch_expert_act_grad(const ExpertDims& x, const int32_t* off, const uint16_t* gy,
                                  const uint16_t* pre, uint16_t* gz, float* partial,
                                  hipStream_t s);
hipError_t launch_expert_bias_sum(const ExpertDims& x, const int32_t* off, const float* partial,
                                  float* gb, hipStream_t s);

}  // namespace moe
