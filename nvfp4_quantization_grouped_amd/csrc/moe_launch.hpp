// Host-side launchers of the routed-expert layer's kernels (internal; the
// public ABI is include/mxq_moe.h).  Each launcher enqueues on `st` and
// returns the HIP error of the launch.  Arguments are validated by the ABI
// layer before these run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxGroups = 64;

// A launch's threads in one dimension are counted in 32 bits.
inline bool launchable(int64_t blocks, int64_t threads) { return blocks > 0 && blocks <= 0xFFFFFFFFll / threads; }

struct RouteArgs {
  const void* logits;
  const float* bias;          // NULL: none
  const uint8_t* token_mask;  // NULL: every token counts
  float* weights;
  int32_t* index;
  int64_t tokens;
  int experts, top_k, groups, group_size, top_groups, group_best;
  bool sigmoid, renormalize;
  double scale;
};
hipError_t launch_moe_route(const RouteArgs& a, int dt, hipStream_t st);
hipError_t launch_moe_route_bwd(const void* logits, int dt, int64_t tokens, int experts, int top_k, bool sigmoid,
                                bool renormalize, double scale, const int32_t* index, const float* grad_weights,
                                void* grad_logits, hipStream_t st);

int64_t plan_workspace_bytes(int64_t slots, int local);
hipError_t launch_moe_plan(const int32_t* index, int64_t slots, int first, int local, int32_t* offs, int32_t* rows,
                           int32_t* slot_of_row, int32_t* workspace, hipStream_t st);
// x [tokens, hidden] -> out [tokens * top_k, hidden] at rows.
hipError_t launch_moe_dispatch(const void* x, int dt, int64_t tokens, int64_t hidden, int top_k, const int32_t* rows,
                               void* out, hipStream_t st);
hipError_t launch_moe_dispatch_quantized(const void* x, int dt, int64_t tokens, int64_t hidden, int top_k,
                                         const int32_t* rows, int fmt, uint8_t* codes, uint8_t* scales,
                                         hipStream_t st);
// weights NULL: all 1.
hipError_t launch_moe_combine(const void* y, int dt, int64_t tokens, int64_t hidden, int top_k, const int32_t* rows,
                              const float* weights, void* out, hipStream_t st);
hipError_t launch_moe_combine_bwd(const void* grad_out, const void* y, int dt, int64_t tokens, int64_t hidden,
                                  int top_k, const int32_t* rows, const float* weights, void* grad_y,
                                  float* grad_weights, hipStream_t st);
// total: the count of rows that count, in device memory (NULL: all of them).
hipError_t launch_swiglu_fwd(const void* gate_up, int dt, int64_t rows, int64_t inter, const int32_t* total, void* h,
                             uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_swiglu_quantized(const void* gate_up, int dt, int64_t rows, int64_t inter, const int32_t* total,
                                   int fmt, uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_swiglu_bwd(const void* grad_h, const void* gate_up, const uint8_t* codes, const uint8_t* scales,
                             int dt, int64_t rows, int64_t inter, const int32_t* total, void* grad_gate_up,
                             hipStream_t st);

}  // namespace mxq
