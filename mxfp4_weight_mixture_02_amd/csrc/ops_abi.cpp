// C ABI of the operators beside the expert block (include/mxmoe_ops.h):
// host-side validation, workspace layout and launches.  Every check runs
// before the first enqueue.
#include "mxmoe_ops.h"

#include <hip/hip_runtime.h>

#include "abi_util.hpp"
#include "gate.hpp"

namespace {

using mxmoe::aligned;
using mxmoe::fail;
using mxmoe::ok;

constexpr size_t ALIGN = 256;
size_t up(size_t v, size_t m) { return (v + m - 1) / m * m; }

bool finite(float v) { return v - v == 0.0f; }

int check_workspace(const void* ws, size_t given, size_t needed) {
  if (!ws || given < needed)
    return fail(MXFP4_EWORKSPACE, "workspace of %zu bytes given, %zu needed", given, needed);
  if (!aligned(ws, ALIGN)) return fail(MXFP4_EINVAL, "workspace must be 256-byte aligned");
  return MXFP4_OK;
}

int check_route_sizes(int64_t T, int32_t E, int32_t k) {
  if (T < 1 || E < 1 || k < 1)
    return fail(MXFP4_EINVAL, "T, E and k must be >= 1 (T=%lld E=%d k=%d)", (long long)T, E, k);
  if (E > 256) return fail(MXFP4_EUNSUPPORTED, "E=%d > 256", E);
  if (k > E || k > 8) return fail(MXFP4_EUNSUPPORTED, "k=%d must be <= min(E, 8)", k);
  if (T >= (int64_t(1) << 31) || T * k >= (int64_t(1) << 31))
    return fail(MXFP4_EUNSUPPORTED, "T*k routed rows exceed int32 (T=%lld k=%d)", (long long)T, k);
  return MXFP4_OK;
}

int check_route(const mxmoe_route_opts* o, int64_t T, int32_t E, int32_t k) {
  if (!o) return fail(MXFP4_EINVAL, "opts is NULL");
  const int rc = check_route_sizes(T, E, k);
  if (rc) return rc;
  if (o->score != MXMOE_SCORE_SOFTMAX && o->score != MXMOE_SCORE_SIGMOID)
    return fail(MXFP4_EINVAL, "score=%d unknown", o->score);
  if (o->group_score != MXMOE_GROUP_MAX && o->group_score != MXMOE_GROUP_TOP2)
    return fail(MXFP4_EINVAL, "group_score=%d unknown", o->group_score);
  if (o->groups < 1 || o->top_groups < 1 || o->top_groups > o->groups)
    return fail(MXFP4_EINVAL, "groups must be >= 1 and top_groups in 1..groups (groups=%d top_groups=%d)",
                o->groups, o->top_groups);
  if (o->groups > 64 || E % o->groups)
    return fail(MXFP4_EUNSUPPORTED, "groups=%d must divide E=%d and be <= 64", o->groups, E);
  if (k > o->top_groups * (E / o->groups))
    return fail(MXFP4_EUNSUPPORTED, "k=%d experts do not fit %d groups of %d", k, o->top_groups,
                E / o->groups);
  if (!finite(o->scale)) return fail(MXFP4_EINVAL, "scale must be finite");
  return MXFP4_OK;
}

mxmoe::RouteArgs route_args(const mxmoe_route_opts& o, int64_t T, int32_t E, int32_t k,
                            const float* logits, const float* bias) {
  mxmoe::RouteArgs a{};
  a.T = T;
  a.E = E;
  a.k = k;
  a.groups = o.groups;
  a.top_groups = o.top_groups;
  a.sigmoid = o.score == MXMOE_SCORE_SIGMOID;
  a.top2 = o.group_score == MXMOE_GROUP_TOP2;
  a.renorm = o.renorm != 0;
  a.scale = o.scale;
  a.logits = logits;
  a.bias = bias;
  return a;
}

}  // namespace

extern "C" {

size_t mxmoe_route_workspace_bytes(int64_t T, int32_t E, int32_t k) {
  if (check_route_sizes(T, E, k) != MXFP4_OK) return 0;
  ok();
  return up((size_t)mxmoe::gate_blocks(T) * E * 4, ALIGN) + up((size_t)E * 4, ALIGN);
}

int mxmoe_route(const mxmoe_route_opts* opts, int64_t T, int32_t E, int32_t k, const float* logits,
                const float* bias, int32_t* topk_idx, float* topk_w, int32_t* expert_offsets,
                int32_t* sorted_rows, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_route(opts, T, E, k);
  if (rc) return rc;
  if (!logits || !topk_idx || !topk_w || !expert_offsets || !sorted_rows)
    return fail(MXFP4_EINVAL, "logits, topk_idx, topk_w, expert_offsets and sorted_rows are required");
  if (!aligned(logits, 4) || (bias && !aligned(bias, 4)) || !aligned(topk_idx, 4) ||
      !aligned(topk_w, 4) || !aligned(expert_offsets, 4) || !aligned(sorted_rows, 4))
    return fail(MXFP4_EINVAL, "tensors must be 4-byte aligned");
  rc = check_workspace(workspace, workspace_bytes, mxmoe_route_workspace_bytes(T, E, k));
  if (rc) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  mxmoe::RouteArgs a = route_args(*opts, T, E, k, logits, bias);
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.offsets = expert_offsets;
  a.sorted_rows = sorted_rows;
  int32_t* hist = static_cast<int32_t*>(workspace);
  int32_t* total = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) +
                                              up((size_t)mxmoe::gate_blocks(T) * E * 4, ALIGN));
  LAUNCH(mxmoe::launch_gate(a, hist, s), "gate");
  LAUNCH(mxmoe::launch_gate_prefix(a, hist, total, s), "gate_prefix");
  LAUNCH(mxmoe::launch_gate_scatter(a, hist, total, s), "gate_scatter");
  return ok();
}

int mxmoe_route_backward(const mxmoe_route_opts* opts, int64_t T, int32_t E, int32_t k,
                         const float* logits, const int32_t* topk_idx, const float* dw,
                         float* dlogits, void* stream) {
  const int rc = check_route(opts, T, E, k);
  if (rc) return rc;
  if (!logits || !topk_idx || !dw || !dlogits)
    return fail(MXFP4_EINVAL, "logits, topk_idx, dw and dlogits are required");
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(dw, 4) || !aligned(dlogits, 4))
    return fail(MXFP4_EINVAL, "tensors must be 4-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  LAUNCH(mxmoe::launch_gate_bwd(route_args(*opts, T, E, k, logits, nullptr), topk_idx, dw, dlogits, s),
         "gate_bwd");
  return ok();
}

}  // extern "C"
