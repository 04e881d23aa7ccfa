// Internal declarations of the forward step, the router and the gradient clipping: workspace
// layouts and kernel launchers (see lrm_internal.hpp for the backward path's).
#pragma once

#include "lrm_internal.hpp"

namespace lrm {

// Router workspace.  A workgroup of the routing kernel writes one row of partial sums; the grid is
// at most kRouteBlocks workgroups, so the reduction over workgroups stays small.
constexpr int kRouteBlocks = 256;

struct RouteWs {
  size_t err;      // int32 error word of the last lrm_route
  size_t tokens;   // int32 [kRouteBlocks][2] valid tokens, error bits
  size_t counts;   // int32 [kRouteBlocks][pitch] pairs per expert
  size_t prob;     // float [kRouteBlocks][pitch] sums of probabilities
  size_t total;
  int pitch;       // E rounded up to 4
};

inline RouteWs route_ws(int E) {
  RouteWs w{};
  w.pitch = (E + 3) / 4 * 4;
  size_t off = 256;
  w.tokens = off;
  off = align_up(off + (size_t)kRouteBlocks * 8, 256);
  w.counts = off;
  off = align_up(off + (size_t)kRouteBlocks * w.pitch * 4, 256);
  w.prob = off;
  off = align_up(off + (size_t)kRouteBlocks * w.pitch * 4, 256);
  w.total = off;
  return w;
}

// Workspace of the forward calls and lrm_gate_dots: the error word's 256 bytes, then the pair ->
// row map int32 [T*k] (validated on use, never cleared).
constexpr size_t kForwardMap = 256;
inline size_t forward_ws_bytes(const lrm_problem& p) {
  return align_up(kForwardMap + (size_t)p.T * p.k * 4, 256);
}

// Gradient clipping: a launch takes up to kTensorsPerLaunch list entries in its kernel arguments
// and writes kGradBlocks partial sums.
constexpr int kTensorsPerLaunch = 64;
constexpr int kGradBlocks = 1024;
constexpr size_t kGradPartials = 256;  // byte offset of double [launches][kGradBlocks]
inline int64_t grad_launches(int32_t n) { return n <= 0 ? 1 : (n + kTensorsPerLaunch - 1) / kTensorsPerLaunch; }
inline size_t grad_ws_bytes(int32_t n) {
  return kGradPartials + (size_t)grad_launches(n) * kGradBlocks * 8;
}

hipError_t launch_route(const lrm_router& r, const void* logits, const uint8_t* mask,
                        int32_t* topk_idx, float* topk_w, float* lse, int32_t* counts, float* prob,
                        float* loss, char* ws, hipStream_t s);
hipError_t launch_route_backward(const lrm_router& r, const void* logits, const int32_t* topk_idx,
                                 const float* topk_w, const int32_t* counts,
                                 const float* adot, float* dlogits, hipStream_t s);
hipError_t launch_gate_dots(const lrm_problem& p, const int32_t* sel_pair, const int32_t* cmp_off,
                            const float* dphi, const void* Phic, float* adot, char* ws,
                            hipStream_t s);
hipError_t launch_fc1_swiglu(const lrm_problem& p, const int32_t* row_pair, const int32_t* fwd_off,
                             const void* x, const void* W1, void* ac, void* phi, char* ws,
                             hipStream_t s);
// wide: y in float32 for a bf16 layer too
hipError_t launch_fc2(const lrm_problem& p, const int32_t* fwd_off, const void* phi, const void* W,
                      void* y, bool wide, hipStream_t s);
hipError_t launch_combine(const lrm_problem& p, const int32_t* row_pair, const int32_t* fwd_off,
                          const float* topk_w, const void* y, bool wide, const void* residual,
                          void* out, char* ws, hipStream_t s);
hipError_t launch_grad_norm(const lrm_tensor* list, int32_t n, float* norm, char* ws,
                            hipStream_t s);
hipError_t launch_clip(const lrm_tensor* list, int32_t n, float max_norm, float* norm, char* ws,
                       hipStream_t s);

}  // namespace lrm
