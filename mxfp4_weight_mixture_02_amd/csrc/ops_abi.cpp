// C ABI of the operators beside the expert block (include/mxmoe_ops.h):
// host-side validation, workspace layout and launches.  Every check runs
// before the first enqueue.
#include "mxmoe_ops.h"

#include <hip/hip_runtime.h>

#include "abi_util.hpp"
#include "fp8.hpp"
#include "gate.hpp"
#include "swiglu8.hpp"

namespace {

using mxmoe::aligned;
using mxmoe::fail;
using mxmoe::launchable;
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
  if (T >= (int64_t(1) << 26))
    return fail(MXFP4_EUNSUPPORTED, "T=%lld tokens (must be < 2^26)", (long long)T);
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
                            const float* logits, const float* bias, const float* dlogits = nullptr) {
  mxmoe::RouteArgs a{};
  a.T = T;
  a.E = E;
  a.k = k;
  a.groups = o.groups;
  a.top_groups = o.top_groups;
  a.share = 1;
  while (2 * a.share * o.groups <= 64) a.share *= 2;
  // the choice gives a lane ceil(E / 64) experts, as 1, 2 or 4
  const int each = E <= 64 ? 1 : E <= 128 ? 2 : 4, per = E / o.groups;
  const int lanes = per % each == 0 ? per / each : 0;
  a.group_lanes = (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const int row_each = 4 * each, row_of = per % row_each == 0 ? per / row_each : 0;
  a.row_lanes = o.top_groups == o.groups ? 16 : (row_of & (row_of - 1)) == 0 ? row_of : 0;
  a.rows = E % 4 == 0 && aligned(logits, 16) && aligned(dlogits, 16);
  if (!a.rows) a.row_lanes = 0;
  a.wide = E % each == 0 && aligned(logits, 4 * each) && aligned(dlogits, 4 * each);
  a.sigmoid = o.score == MXMOE_SCORE_SIGMOID;
  a.top2 = o.group_score == MXMOE_GROUP_TOP2;
  a.renorm = o.renorm != 0;
  a.scale = o.scale;
  a.logits = logits;
  a.bias = bias;
  return a;
}

constexpr int64_t FP8_MAX_K = int64_t(1) << 22;

// An 8-bit matrix of `rows` rows and K columns: sizes that the kernels'
// 32-bit offsets within a tile and block counts hold.
int check_fp8(int64_t rows, int64_t K, const char* what) {
  if (rows < 1 || K < 1)
    return fail(MXFP4_EINVAL, "%s: sizes must be >= 1 (%lld x %lld)", what, (long long)rows,
                (long long)K);
  if (rows >= (int64_t(1) << 27) || K > FP8_MAX_K)
    return fail(MXFP4_EUNSUPPORTED, "%s: %lld x %lld (rows must be < 2^27, K <= 2^22)", what,
                (long long)rows, (long long)K);
  // the quantizers launch a thread for 8 elements, and a launch has 2^32
  if ((rows + 127) * mxmoe::fp8_pitch(K) >= (int64_t(1) << 35))
    return fail(MXFP4_EUNSUPPORTED, "%s: %lld x %lld elements (must be < 2^35)", what,
                (long long)rows, (long long)K);
  return MXFP4_OK;
}

int check_dtype(int dtype, const void* p, const char* what) {
  if (dtype != MXMOE_F32 && dtype != MXMOE_BF16)
    return fail(MXFP4_EINVAL, "%s: dtype %d unknown", what, dtype);
  if (!aligned(p, dtype == MXMOE_F32 ? 4 : 2)) return fail(MXFP4_EINVAL, "%s is misaligned", what);
  return MXFP4_OK;
}

int check_product(int64_t M, int64_t N, int64_t K) {
  int rc = check_fp8(M, K, "X");
  if (!rc) rc = check_fp8(N, K, "W");
  if (!rc && ((M + 127) / 128) * ((N + 127) / 128) >= (int64_t(1) << 23))
    rc = fail(MXFP4_EUNSUPPORTED, "M=%lld N=%lld: too many tiles", (long long)M, (long long)N);
  // few rows: a workgroup of 512 threads for 16 rows of W
  if (!rc && M <= 16 && !launchable((N + 15) / 16, 512))
    rc = fail(MXFP4_EUNSUPPORTED, "M=%lld N=%lld: N must be <= 2^27 - 16 for up to 16 rows", (long long)M,
              (long long)N);
  return rc;
}

// Workspace of a product: X's codes and scales, then (dw) W's, then the
// product's own.
struct Fp8Layout {
  size_t xs, w, ws, part, total;
};
Fp8Layout fp8_layout(int64_t M, int64_t N, int64_t K, bool w, int out_f32) {
  Fp8Layout L{};
  if (!w && mxmoe::fp8_fused_fits(M, N, K)) {   // X never leaves the product's launch
    L.total = ALIGN;
    return L;
  }
  const size_t kb = (size_t)mxmoe::fp8_pitch(K) / 128;
  L.xs = up((size_t)M * mxmoe::fp8_pitch(K), ALIGN);
  L.w = L.xs + up(kb * mxmoe::fp8_scale_pitch(M), ALIGN);
  L.ws = L.w + (w ? up((size_t)N * mxmoe::fp8_pitch(K), ALIGN) : 0);
  L.part = L.ws + (w ? up(kb * mxmoe::fp8_scale_pitch(N), ALIGN) : 0);
  L.total = L.part + up(mxmoe::fp8_part_bytes(M, N, K, out_f32), ALIGN);
  return L;
}

size_t matmul_bytes(int64_t M, int64_t N, int64_t K, int out_dtype) {
  return up(mxmoe::fp8_part_bytes(M, N, K, out_dtype == MXMOE_F32), ALIGN) + ALIGN;
}

int check_swiglu8(int64_t R, int64_t I, float alpha, float limit) {
  if (R < 1 || I < 1)
    return fail(MXFP4_EINVAL, "R and I must be >= 1 (R=%lld I=%lld)", (long long)R, (long long)I);
  if (I % 16) return fail(MXFP4_EUNSUPPORTED, "I=%lld is not a multiple of 16", (long long)I);
  // a thread for 8 elements of h
  if (I >= (int64_t(1) << 32) || R >= (int64_t(1) << 34) / I || !launchable((R * I / 4 + 255) / 256, 256))
    return fail(MXFP4_EUNSUPPORTED, "R=%lld I=%lld: R * 2I elements must be <= 2^35 - 2048", (long long)R,
                (long long)I);
  if (!finite(alpha) || !finite(limit) || !(limit > 0.0f))
    return fail(MXFP4_EINVAL, "alpha must be finite and limit finite and > 0");
  return MXFP4_OK;
}

}  // namespace

extern "C" {

size_t mxmoe_route_workspace_bytes(int64_t T, int32_t E, int32_t k) {
  if (check_route_sizes(T, E, k) != MXFP4_OK) return 0;
  ok();
  if (mxmoe::gate_in_one(T)) return ALIGN;
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
  if (mxmoe::gate_in_one(T)) {
    LAUNCH(mxmoe::launch_gate_one(a, s), "gate");
    return ok();
  }
  LAUNCH(mxmoe::launch_gate(a, hist, s), "gate");
  if (mxmoe::gate_adds(T))
    total = nullptr;
  else
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
  LAUNCH(mxmoe::launch_gate_bwd(route_args(*opts, T, E, k, logits, nullptr, dlogits), topk_idx, dw, dlogits, s),
         "gate_bwd");
  return ok();
}

int mxmoe_fp8_quantize(const void* x, int dtype, int64_t rows, int64_t K, int block_rows,
                       uint8_t* codes, uint8_t* scales, void* stream) {
  int rc = check_fp8(rows, K, "x");
  if (rc) return rc;
  if (!x || !codes || !scales) return fail(MXFP4_EINVAL, "x, codes and scales are required");
  rc = check_dtype(dtype, x, "x");
  if (rc) return rc;
  if (block_rows != 1 && block_rows != 128)
    return fail(MXFP4_EINVAL, "block_rows=%d must be 1 or 128", block_rows);
  if (!aligned(codes, 16) || !aligned(scales, 16))
    return fail(MXFP4_EINVAL, "codes and scales must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (block_rows == 1)
    LAUNCH(mxmoe::launch_fp8_quantize_rows(x, dtype == MXMOE_F32, rows, K, codes, scales, s),
           "fp8_quantize_rows");
  else
    LAUNCH(mxmoe::launch_fp8_quantize_blocks(x, dtype == MXMOE_F32, rows, K, codes, scales, s),
           "fp8_quantize_blocks");
  return ok();
}

int mxmoe_fp8_quantize_t(const void* x, int dtype, int64_t rows, int64_t K, uint8_t* codes,
                         uint8_t* scales, void* stream) {
  int rc = check_fp8(K, rows, "x transposed");
  if (rc) return rc;
  if (!x || !codes || !scales) return fail(MXFP4_EINVAL, "x, codes and scales are required");
  rc = check_dtype(dtype, x, "x");
  if (rc) return rc;
  if (!aligned(codes, 16) || !aligned(scales, 16))
    return fail(MXFP4_EINVAL, "codes and scales must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  LAUNCH(mxmoe::launch_fp8_quantize_cols(x, dtype == MXMOE_F32, rows, K, codes, scales, s),
         "fp8_quantize_cols");
  return ok();
}

int mxmoe_fp8_transpose(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                        uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  int rc = check_fp8(rows, K, "w");
  if (!rc) rc = check_fp8(K, rows, "w transposed");
  if (rc) return rc;
  if (!codes || !scales || !codes_t || !scales_t)
    return fail(MXFP4_EINVAL, "codes, scales, codes_t and scales_t are required");
  if (!aligned(codes, 16) || !aligned(codes_t, 16))
    return fail(MXFP4_EINVAL, "codes and codes_t must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  LAUNCH(mxmoe::launch_fp8_transpose(codes, scales, rows, K, codes_t, scales_t, s), "fp8_transpose");
  return ok();
}

int mxmoe_fp8_matmul(int64_t M, int64_t N, int64_t K, const uint8_t* x_codes,
                     const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                     int w_block_rows, const uint16_t* bias, int out_dtype, void* out,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_product(M, N, K);
  if (rc) return rc;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !out)
    return fail(MXFP4_EINVAL, "codes, scales and out are required");
  if (w_block_rows != 1 && w_block_rows != 128)
    return fail(MXFP4_EINVAL, "w_block_rows=%d must be 1 or 128", w_block_rows);
  rc = check_dtype(out_dtype, out, "out");
  if (rc) return rc;
  if (!aligned(x_codes, 16) || !aligned(x_scales, 16) || !aligned(w_codes, 16) ||
      (w_block_rows == 1 && !aligned(w_scales, 16)) || !aligned(out, 16) || !aligned(bias, 2))
    return fail(MXFP4_EINVAL, "codes, scales of rows and out must be 16-byte aligned");
  rc = check_workspace(workspace, workspace_bytes, matmul_bytes(M, N, K, out_dtype));
  if (rc) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const mxmoe::Fp8Gemm g{M, N, K, x_codes, x_scales, w_codes, w_scales, w_block_rows == 1, bias,
                         out, out_dtype == MXMOE_F32, static_cast<float*>(workspace)};
  LAUNCH(mxmoe::launch_fp8_gemm(g, s), "fp8_matmul");
  return ok();
}

size_t mxmoe_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype) {
  if (check_product(M, N, K) != MXFP4_OK || check_dtype(out_dtype, nullptr, "out") != MXFP4_OK) return 0;
  ok();
  return matmul_bytes(M, N, K, out_dtype);
}

size_t mxmoe_fp8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype) {
  if (check_product(M, N, K) != MXFP4_OK || check_dtype(out_dtype, nullptr, "out") != MXFP4_OK) return 0;
  ok();
  return fp8_layout(M, N, K, false, out_dtype == MXMOE_F32).total;
}

size_t mxmoe_fp8_linear_dw_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (check_product(N, K, M) != MXFP4_OK) return 0;
  ok();
  return fp8_layout(N, K, M, true, 1).total;
}

int mxmoe_fp8_linear(int64_t M, int64_t N, int64_t K, const uint16_t* x, const uint8_t* w_codes,
                     const uint8_t* w_scales, const uint16_t* bias, int out_dtype, void* out,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_product(M, N, K);
  if (rc) return rc;
  if (!x || !w_codes || !w_scales || !out)
    return fail(MXFP4_EINVAL, "x, w_codes, w_scales and out are required");
  rc = check_dtype(out_dtype, out, "out");
  if (!rc) rc = check_dtype(MXMOE_BF16, x, "x");
  if (rc) return rc;
  if (!aligned(w_codes, 16) || !aligned(out, 16) || !aligned(bias, 2))
    return fail(MXFP4_EINVAL, "w_codes and out must be 16-byte aligned");
  const Fp8Layout L = fp8_layout(M, N, K, false, out_dtype == MXMOE_F32);
  rc = check_workspace(workspace, workspace_bytes, L.total);
  if (rc) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const mxmoe::Fp8Gemm g{M, N, K, ws, ws + L.xs, w_codes, w_scales, 0, bias, out,
                         out_dtype == MXMOE_F32, reinterpret_cast<float*>(ws + L.part)};
  if (mxmoe::fp8_fused_fits(M, N, K)) {
    LAUNCH(mxmoe::launch_fp8_fused(g, x, s), "fp8_linear");
    return ok();
  }
  LAUNCH(mxmoe::launch_fp8_quantize_rows(x, 0, M, K, ws, ws + L.xs, s), "fp8_quantize_rows");
  LAUNCH(mxmoe::launch_fp8_gemm(g, s), "fp8_matmul");
  return ok();
}

int mxmoe_fp8_linear_dw(int64_t M, int64_t N, int64_t K, const uint16_t* dy, const uint16_t* x,
                        float* dw, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_product(N, K, M);
  if (rc) return rc;
  if (!dy || !x || !dw) return fail(MXFP4_EINVAL, "dy, x and dw are required");
  if (!aligned(dy, 2) || !aligned(x, 2) || !aligned(dw, 16))
    return fail(MXFP4_EINVAL, "dw must be 16-byte, dy and x 2-byte aligned");
  const Fp8Layout L = fp8_layout(N, K, M, true, 1);
  rc = check_workspace(workspace, workspace_bytes, L.total);
  if (rc) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LAUNCH(mxmoe::launch_fp8_quantize_cols_pair(dy, N, ws, ws + L.xs, x, K, ws + L.w, ws + L.ws, M, s),
         "fp8_quantize_cols");
  const mxmoe::Fp8Gemm g{N, K, M, ws, ws + L.xs, ws + L.w, ws + L.ws, 1, nullptr, dw, 1,
                         reinterpret_cast<float*>(ws + L.part)};
  LAUNCH(mxmoe::launch_fp8_gemm(g, s), "fp8_matmul");
  return ok();
}

int mxmoe_swiglu8_forward(const uint16_t* h, int64_t R, int64_t I, float alpha, float limit,
                          uint16_t* a, uint8_t* codes, uint8_t* scales, void* stream) {
  const int rc = check_swiglu8(R, I, alpha, limit);
  if (rc) return rc;
  if (!h || !codes || !scales) return fail(MXFP4_EINVAL, "h, codes and scales are required");
  if (!aligned(h, 16) || !aligned(a, 16) || !aligned(codes, 16))
    return fail(MXFP4_EINVAL, "h, a and codes must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  LAUNCH(mxmoe::launch_swiglu8_fwd(h, R * I / 4, alpha, limit, a, codes, scales, s), "swiglu8_fwd");
  return ok();
}

int mxmoe_swiglu8_backward(const uint8_t* codes, const uint8_t* scales, const uint16_t* da,
                           int64_t R, int64_t I, float alpha, float limit, uint16_t* dh,
                           uint16_t* a, void* stream) {
  const int rc = check_swiglu8(R, I, alpha, limit);
  if (rc) return rc;
  if (!codes || !scales || !da || !dh)
    return fail(MXFP4_EINVAL, "codes, scales, da and dh are required");
  if (!aligned(codes, 16) || !aligned(da, 16) || !aligned(dh, 16) || !aligned(a, 16))
    return fail(MXFP4_EINVAL, "codes, da, dh and a must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  LAUNCH(mxmoe::launch_swiglu8_bwd(codes, scales, da, R * I / 4, alpha, limit, dh, a, s), "swiglu8_bwd");
  return ok();
}

int mxmoe_swiglu8_restore(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t I,
                          float alpha, float limit, uint16_t* h, uint16_t* a, void* stream) {
  const int rc = check_swiglu8(R, I, alpha, limit);
  if (rc) return rc;
  if (!codes || !scales || (!h && !a))
    return fail(MXFP4_EINVAL, "codes, scales and one of h and a are required");
  if (!aligned(codes, 16) || !aligned(h, 16) || !aligned(a, 16))
    return fail(MXFP4_EINVAL, "codes, h and a must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  LAUNCH(mxmoe::launch_swiglu8_restore(codes, scales, R * I / 4, alpha, limit, h, a, s), "swiglu8_restore");
  return ok();
}

}  // extern "C"
