// The plan object and the host helpers shared by the two API files
// (moe_api.cpp: the shuffle, moe_layer_api.cpp: the layer's operators).
#pragma once

#include <cstdint>
#include <vector>

#include "moe_internal.h"

namespace moe {
typedef unsigned long long CaptureId;

// Event pairs of moe_plan_timing and the kernel of each recorded launch.
struct LaunchTimer {
  std::vector<hipEvent_t> start, stop;
  std::vector<int32_t> ids;
  int used = 0;
};
}  // namespace moe

struct moe_plan {
  moe_config cfg;
  moe::Dims d;
  moe::Layout layout;
  int64_t staging_rows_max;
  // Bound by moe_route_plan.
  const int32_t* idx;
  void* ws;
  moe::Work work;
  bool routed;     // route_count has been launched for the bound routing
  bool scanned;    // route_scan has been launched for it (tile bases, offsets, status)
  bool assigned;   // slot_of / row_src (and stage_of / stage_src) are final
  // The stream captures that recorded these (0: none, they were launched).
  moe::CaptureId route_capture, scan_capture, assign_capture;
  moe::LaunchTimer* timer;  // per-launch timing, or null
};

namespace moe {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// The timer of the plan whose call is running on this thread (moe_api.cpp).
extern thread_local LaunchTimer* tl_timer;

// Makes `plan`'s timer the active one for the lifetime of the scope (each
// API call that launches kernels opens one).
struct TimerScope {
  LaunchTimer* prev;
  explicit TimerScope(const moe_plan* plan) : prev(tl_timer) { tl_timer = plan->timer; }
  ~TimerScope() { tl_timer = prev; }
};

// The capture that stream s records into (0: none).
moe_status capture_of(hipStream_t s, CaptureId* id);

// A scan or an assign recorded into a graph counts in that capture only.  A
// capture on a plan that was routed outside of it records its own, so that a
// graph replayed after another route of the plan computes with that route.
// And where the route itself was recorded, every replay routes anew, so that
// each call outside of the graph does again what the graph does not hold.
//
// Launches the plan's scan if the route left it to the gather (small plans).
moe_status ensure_scanned(moe_plan* plan, hipStream_t s);
// Makes slot_of / row_src (and the staging arrays) final when no dispatch
// has done it since the last route.
moe_status ensure_assigned(moe_plan* plan, hipStream_t s);

}  // namespace moe
