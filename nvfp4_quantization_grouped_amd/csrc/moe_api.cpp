// C ABI of the routed-expert layer (declared in include/mxq_moe.h): host-side
// validation, then asynchronous launches on the caller's stream.  No
// allocation, no sync.
#include "../../include/mxq.h"
#include "../../include/mxq_moe.h"
#include "abi_checks.hpp"
#include "moe_launch.hpp"

namespace {

using namespace mxq;

constexpr int64_t kMaxSlots = (int64_t(1) << 31) - (1 << 16);   // rows, and a workgroup past them, fit int32
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxElems = int64_t(1) << 40;

int route_shape(int64_t tokens, int64_t experts, int64_t top_k) {
  if (tokens < 0 || experts < 1 || experts > mxq::kMaxExperts || top_k < 1 || top_k > mxq::kMaxTopK || top_k > experts)
    return MXQ_ERR_SHAPE;
  return product_below(tokens, experts, kMaxElems) < 0 ? MXQ_ERR_SHAPE : MXQ_OK;
}

int rows_shape(int64_t tokens, int64_t hidden, int64_t top_k) {
  if (tokens < 0 || hidden < 0 || hidden > kMaxWidth || top_k < 1) return MXQ_ERR_SHAPE;
  return product_below(tokens, top_k, kMaxSlots) < 0 ? MXQ_ERR_SHAPE : MXQ_OK;
}

}  // namespace

extern "C" {

int moe_route(const void* logits, int t, int64_t tokens, int64_t experts, int64_t top_k, int score, const float* bias,
              int64_t groups, int64_t top_groups, int group_best, int renormalize, double scale,
              const uint8_t* token_mask, float* weights, int32_t* index, void* stream) {
  const int st = route_shape(tokens, experts, top_k);
  if (st != MXQ_OK) return st;
  if (groups < 1 || groups > mxq::kMaxGroups || experts % groups != 0 || top_groups < 1 || top_groups > groups ||
      (group_best != 1 && group_best != 2))
    return MXQ_ERR_SHAPE;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (score != MXQ_SCORE_SOFTMAX && score != MXQ_SCORE_SIGMOID) return MXQ_ERR_FORMAT;
  if (tokens == 0) return MXQ_OK;
  if (!logits || !weights || !index) return MXQ_ERR_NULL;
  if (misaligned4(bias) || misaligned4(weights) || misaligned4(index)) return MXQ_ERR_ALIGN;
  const Span in[] = {{logits, tokens * experts * dtype_bytes(t)}, {bias, experts * 4}, {token_mask, tokens},
                     {weights, tokens * top_k * 4}};
  if (overlaps_any({weights, tokens * top_k * 4}, in, 3) || overlaps_any({index, tokens * top_k * 4}, in, 4))
    return MXQ_ERR_ALIAS;
  const mxq::RouteArgs a = {logits, bias, token_mask, weights, index, tokens, (int)experts, (int)top_k, (int)groups,
                            (int)(experts / groups), (int)top_groups, group_best, score == MXQ_SCORE_SIGMOID,
                            renormalize != 0, scale};
  return from_hip(mxq::launch_moe_route(a, t, (hipStream_t)stream));
}

int moe_route_bwd(const void* logits, int t, int64_t tokens, int64_t experts, int64_t top_k, int score,
                  int renormalize, double scale, const int32_t* index, const float* grad_weights, void* grad_logits,
                  void* stream) {
  const int st = route_shape(tokens, experts, top_k);
  if (st != MXQ_OK) return st;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (score != MXQ_SCORE_SOFTMAX && score != MXQ_SCORE_SIGMOID) return MXQ_ERR_FORMAT;
  if (tokens == 0) return MXQ_OK;
  if (!logits || !index || !grad_weights || !grad_logits) return MXQ_ERR_NULL;
  if (misaligned4(index) || misaligned4(grad_weights)) return MXQ_ERR_ALIGN;
  const int64_t bytes = tokens * experts * dtype_bytes(t), slots = tokens * top_k * 4;
  const Span in[] = {{logits, bytes}, {index, slots}, {grad_weights, slots}};
  if (overlaps_any({grad_logits, bytes}, in, 3)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_moe_route_bwd(logits, t, tokens, (int)experts, (int)top_k, score == MXQ_SCORE_SIGMOID,
                                            renormalize != 0, scale, index, grad_weights, grad_logits,
                                            (hipStream_t)stream));
}

int64_t moe_plan_workspace(int64_t tokens, int64_t top_k, int64_t local) {
  if (tokens < 0 || top_k < 1 || local < 1 || local > mxq::kMaxExperts) return MXQ_ERR_SHAPE;
  const int64_t n = product_below(tokens, top_k, kMaxSlots);
  return n < 0 ? (int64_t)MXQ_ERR_SHAPE : mxq::plan_workspace_bytes(n, (int)local);
}

int moe_plan(const int32_t* index, int64_t tokens, int64_t top_k, int64_t first, int64_t local, int32_t* offs,
             int32_t* rows, int32_t* slots, void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t need = moe_plan_workspace(tokens, top_k, local);
  if (need < 0 || first < 0 || first >= (int64_t(1) << 31) - local || workspace_bytes < need) return MXQ_ERR_SHAPE;
  const int64_t n = tokens * top_k;
  if (!offs || (n > 0 && (!index || !rows || !slots)) || (need > 0 && !workspace)) return MXQ_ERR_NULL;
  if (misaligned4(index) || misaligned4(offs) || misaligned4(rows) || misaligned4(slots) || misaligned4(workspace))
    return MXQ_ERR_ALIGN;
  const Span all[] = {{index, n * 4}, {offs, local * 4}, {rows, n * 4}, {slots, n * 4}, {workspace, need}};
  for (int i = 1; i < 5; ++i)
    if (overlaps_any(all[i], all, i)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_moe_plan(index, n, (int)first, (int)local, offs, rows, slots, (int32_t*)workspace,
                                       (hipStream_t)stream));
}

int moe_dispatch(const void* x, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows, void* out,
                 void* stream) {
  const int st = rows_shape(tokens, hidden, top_k);
  if (st != MXQ_OK) return st;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (tokens == 0 || hidden == 0) return MXQ_OK;
  if (!x || !rows || !out) return MXQ_ERR_NULL;
  if (misaligned4(rows)) return MXQ_ERR_ALIGN;
  const int64_t row = hidden * dtype_bytes(t), n = tokens * top_k;
  const Span in[] = {{x, tokens * row}, {rows, n * 4}};
  if (overlaps_any({out, n * row}, in, 2)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_moe_dispatch(x, t, tokens, hidden, (int)top_k, rows, out, (hipStream_t)stream));
}

static int combine_rows(const void* y, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows,
                        const float* weights, bool weighted, void* out, void* stream) {
  const int st = rows_shape(tokens, hidden, top_k);
  if (st != MXQ_OK) return st;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (tokens == 0 || hidden == 0) return MXQ_OK;
  if (!y || !rows || !out || (weighted && !weights)) return MXQ_ERR_NULL;
  if (misaligned4(rows) || misaligned4(weights)) return MXQ_ERR_ALIGN;
  const int64_t row = hidden * dtype_bytes(t), n = tokens * top_k;
  const Span in[] = {{y, n * row}, {rows, n * 4}, {weights, n * 4}};
  if (overlaps_any({out, tokens * row}, in, 3)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_moe_combine(y, t, tokens, hidden, (int)top_k, rows, weights, out, (hipStream_t)stream));
}

int moe_dispatch_bwd(const void* grad_out, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows,
                     void* grad_x, void* stream) {
  return combine_rows(grad_out, t, tokens, hidden, top_k, rows, nullptr, false, grad_x, stream);
}

int moe_combine(const void* y, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows,
                const float* weights, void* out, void* stream) {
  return combine_rows(y, t, tokens, hidden, top_k, rows, weights, true, out, stream);
}

int moe_dispatch_quantized(const void* x, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows,
                           int fmt, uint8_t* codes, uint8_t* scales, void* stream) {
  const int st = rows_shape(tokens, hidden, top_k);
  if (st != MXQ_OK) return st;
  if (hidden % 32 != 0) return MXQ_ERR_SHAPE;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (fmt != MXQ_FMT_FP8 && fmt != MXQ_FMT_MXFP4) return MXQ_ERR_FORMAT;
  if (tokens == 0 || hidden == 0) return MXQ_OK;
  if (!x || !rows || !codes || !scales) return MXQ_ERR_NULL;
  if (misaligned4(rows)) return MXQ_ERR_ALIGN;
  const int64_t n = tokens * top_k, nc = n * (fmt == MXQ_FMT_FP8 ? hidden : hidden / 2);
  const Span in[] = {{x, tokens * hidden * dtype_bytes(t)}, {rows, n * 4}, {codes, nc}};
  if (overlaps_any({codes, nc}, in, 2) || overlaps_any({scales, n * (hidden / 32)}, in, 3)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_moe_dispatch_quantized(x, t, tokens, hidden, (int)top_k, rows, fmt, codes, scales,
                                                     (hipStream_t)stream));
}

int moe_combine_bwd(const void* grad_out, const void* y, int t, int64_t tokens, int64_t hidden, int64_t top_k,
                    const int32_t* rows, const float* weights, void* grad_y, float* grad_weights, void* stream) {
  const int st = rows_shape(tokens, hidden, top_k);
  if (st != MXQ_OK) return st;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (tokens == 0 || (!grad_y && !grad_weights)) return MXQ_OK;
  if (!rows || (hidden > 0 && (!grad_out || (grad_weights && !y) || (grad_y && !weights)))) return MXQ_ERR_NULL;
  if (misaligned4(rows) || misaligned4(weights) || misaligned4(grad_weights)) return MXQ_ERR_ALIGN;
  const int64_t row = hidden * dtype_bytes(t), n = tokens * top_k;
  const Span in[] = {{grad_out, tokens * row}, {y, n * row}, {rows, n * 4}, {weights, n * 4}, {grad_y, n * row}};
  if (overlaps_any({grad_y, n * row}, in, 4) || overlaps_any({grad_weights, n * 4}, in, 5)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_moe_combine_bwd(grad_out, y, t, tokens, hidden, (int)top_k, rows, weights, grad_y,
                                              grad_weights, (hipStream_t)stream));
}

// Checks that the two directions of swiglu share.
static int swiglu_shape(int t, int64_t rows, int64_t inter, const int32_t* offs, int64_t experts) {
  if (rows < 0 || inter < 0 || inter % 32 != 0 || inter > kMaxWidth || (offs && experts < 1)) return MXQ_ERR_SHAPE;
  if (product_below(rows, inter, kMaxElems) < 0) return MXQ_ERR_SHAPE;
  return dtype_ok(t) ? MXQ_OK : MXQ_ERR_DTYPE;
}

int swiglu_fwd(const void* gate_up, int t, int64_t rows, int64_t inter, const int32_t* offs, int64_t experts, void* h,
               uint8_t* codes, uint8_t* scales, void* stream) {
  const int st = swiglu_shape(t, rows, inter, offs, experts);
  if (st != MXQ_OK) return st;
  if (rows == 0 || inter == 0) return MXQ_OK;
  if (!gate_up || !h || !codes != !scales) return MXQ_ERR_NULL;
  if (misaligned4(offs)) return MXQ_ERR_ALIGN;
  const int64_t n = rows * inter;
  const Span in[] = {{gate_up, 2 * n * dtype_bytes(t)}, {offs, experts * 4}, {h, n * dtype_bytes(t)}, {codes, 2 * n}};
  if (overlaps_any({h, n * dtype_bytes(t)}, in, 2) || overlaps_any({codes, 2 * n}, in, 3) ||
      overlaps_any({scales, n / 16}, in, 4))
    return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_swiglu_fwd(gate_up, t, rows, inter, offs ? offs + experts - 1 : nullptr, h, codes,
                                         scales, (hipStream_t)stream));
}

int swiglu_quantized(const void* gate_up, int t, int64_t rows, int64_t inter, const int32_t* offs, int64_t experts,
                     int fmt, uint8_t* codes, uint8_t* scales, void* stream) {
  const int st = swiglu_shape(t, rows, inter, offs, experts);
  if (st != MXQ_OK) return st;
  if (fmt != MXQ_FMT_FP8 && fmt != MXQ_FMT_MXFP4) return MXQ_ERR_FORMAT;
  if (rows == 0 || inter == 0) return MXQ_OK;
  if (!gate_up || !codes || !scales) return MXQ_ERR_NULL;
  if (misaligned4(offs)) return MXQ_ERR_ALIGN;
  const int64_t n = rows * inter, nc = fmt == MXQ_FMT_FP8 ? n : n / 2;
  const Span in[] = {{gate_up, 2 * n * dtype_bytes(t)}, {offs, experts * 4}, {codes, nc}};
  if (overlaps_any({codes, nc}, in, 2) || overlaps_any({scales, n / 32}, in, 3)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_swiglu_quantized(gate_up, t, rows, inter, offs ? offs + experts - 1 : nullptr, fmt, codes,
                                               scales, (hipStream_t)stream));
}

int swiglu_bwd(const void* grad_h, const void* gate_up, const uint8_t* codes, const uint8_t* scales, int t,
               int64_t rows, int64_t inter, const int32_t* offs, int64_t experts, void* grad_gate_up, void* stream) {
  const int st = swiglu_shape(t, rows, inter, offs, experts);
  if (st != MXQ_OK) return st;
  if (rows == 0 || inter == 0) return MXQ_OK;
  if (!grad_h || !grad_gate_up || !codes != !scales || !codes == !gate_up) return MXQ_ERR_NULL;
  if (misaligned4(offs)) return MXQ_ERR_ALIGN;
  const int64_t n = rows * inter, wide = 2 * n * dtype_bytes(t);
  const Span in[] = {{grad_h, n * dtype_bytes(t)}, {gate_up, wide}, {codes, 2 * n}, {scales, n / 16},
                     {offs, experts * 4}};
  if (overlaps_any({grad_gate_up, wide}, in, 5)) return MXQ_ERR_ALIAS;
  return from_hip(mxq::launch_swiglu_bwd(grad_h, gate_up, codes, scales, t, rows, inter,
                                         offs ? offs + experts - 1 : nullptr, grad_gate_up, (hipStream_t)stream));
}

}  // extern "C"
