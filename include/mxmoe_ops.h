/*
 * mxmoe_ops.h -- C ABI of the operators beside the MXFP4 expert block of
 * mxfp4_moe.h: routing with its gradient and the block on a given routing,
 * dense products in 8-bit floating point, and 8-bit activation checkpoints.
 *
 * Conventions as in mxfp4_moe.h: dense row-major tensors in device memory
 * owned by the caller, bf16 as uint16_t bit patterns, `stream` a
 * hipStream_t of the current device, all validation on the host before
 * anything is enqueued, the same return codes and mxfp4_last_error().  No
 * call allocates, synchronises or records a memset, so every call can be
 * captured into a HIP graph.  Scratch comes in through `workspace` (256-byte
 * aligned); calls that may overlap need workspaces of their own.
 */
#ifndef MXMOE_OPS_H
#define MXMOE_OPS_H

#include "mxfp4_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------- routing */

#define MXMOE_SCORE_SOFTMAX 0
#define MXMOE_SCORE_SIGMOID 1
#define MXMOE_GROUP_MAX 0
#define MXMOE_GROUP_TOP2 1

/* How logits become a routing.
 *  score        s = softmax or sigmoid of the logits, in fp64
 *  groups       E / groups consecutive experts form a group; 1 = no groups.
 *               groups divides E and is at most 64
 *  top_groups   experts of this many groups may be chosen (1..groups)
 *  group_score  a group's value: the largest choice value in it, or the
 *               fp32 sum of its two largest (of its one, if it has one)
 *  renorm       nonzero: weights are divided by the sum of the chosen scores
 *  scale        weights are multiplied by it; finite
 * Choice value of an expert: c = fp32(s + bias), the fp64 sum rounded once.
 * The groups, then the k experts, with the largest values are chosen, ties
 * to the lower index, a NaN below every number.  Without renorm the weight
 * is scale * s (the bias takes part in the choice alone); with it, weights
 * of a token whose chosen scores are all 0 are 0.  A token whose logits are
 * all -inf has scores 0.  A token's routing and gradient have the same bits
 * whatever the other tokens and T are (a NaN is 0x7FC00000). */
typedef struct mxmoe_route_opts {
  int32_t score;
  int32_t groups;
  int32_t top_groups;
  int32_t group_score;
  int32_t renorm;
  float scale;
} mxmoe_route_opts;

/* Routing of T tokens over E experts (E <= 256, 1 <= k <= 8, k at most the
 * experts of top_groups groups, T < 2^26).
 *  logits fp32 [T, E] in; bias fp32 [E] in or NULL
 *  topk_idx int32 [T, k], topk_w fp32 [T, k]: slots in descending choice
 *  value; expert_offsets int32 [E + 1] and sorted_rows int32 [T * k]: the
 *  plan of mxfp4_moe_saved (flat rows grouped by expert, ascending within
 *  an expert).  workspace: mxmoe_route_workspace_bytes. */
int mxmoe_route(const mxmoe_route_opts* opts, int64_t T, int32_t E, int32_t k, const float* logits,
                const float* bias, int32_t* topk_idx, float* topk_w, int32_t* expert_offsets,
                int32_t* sorted_rows, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace mxmoe_route needs (0 if T, E or k is out of range). */
size_t mxmoe_route_workspace_bytes(int64_t T, int32_t E, int32_t k);

/* Gradient of the weights: dlogits fp32 [T, E] (every element written) from
 * dw fp32 [T, k], the gradient of topk_w, with the choice topk_idx held
 * fixed.  The bias gets no gradient.  A topk_idx outside [0, E) is skipped;
 * a token whose chosen scores are all 0 under renorm has gradient 0. */
int mxmoe_route_backward(const mxmoe_route_opts* opts, int64_t T, int32_t E, int32_t k,
                         const float* logits, const int32_t* topk_idx, const float* dw,
                         float* dlogits, void* stream);

/* Router logits as the expert block forms them: fp32 [T, E] = x W_r^T + b_r
 * with x bf16 [T, H], router_w fp32 [E, H], router_b fp32 [E] or NULL,
 * products summed in fp64 and rounded once.  H % 32 == 0, H <= 5120, E <=
 * 256, T * H < 2^31, ceil(T / 16) * ceil(E / 16) < 2^22; x and router_w 16-byte
 * aligned. */
int mxmoe_router_logits(int64_t T, int64_t H, int32_t E, const uint16_t* x, const float* router_w,
                        const float* router_b, float* logits, void* stream);

/* The expert block (mxfp4_moe_forward) on a given routing: `saved` names
 * its topk_idx, topk_w, expert_offsets and sorted_rows as mxmoe_route fills
 * them (inputs, read as they are: offsets must end at T * k, sorted_rows
 * must be a permutation grouped by expert); h, a (and lora_v, lora_vg with
 * the adapters) are outputs, or all NULL for inference.  router_w may be
 * NULL.  workspace: mxfp4_moe_workspace_bytes of MXFP4_WS_FORWARD_SAVED or
 * (without h) MXFP4_WS_FORWARD. */
int mxmoe_forward_routed(const mxfp4_moe_dims* dims, const mxfp4_moe_weights* w, const uint16_t* x,
                         uint16_t* out, const mxfp4_moe_saved* saved, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Its backward: everything mxfp4_moe_backward computes for the gradients
 * that grads names, except that dX holds no router term; dw fp32 [T, k] is
 * the gradient of topk_w instead (the input of mxmoe_route_backward).
 * router_w may be NULL.  workspace: MXFP4_WS_BACKWARD, or
 * MXFP4_WS_BACKWARD_FULL if grads names dW_gu, dW_dn, db_gu or db_dn. */
int mxmoe_backward_routed(const mxfp4_moe_dims* dims, const mxfp4_moe_weights* w,
                          const mxfp4_moe_saved* saved, const uint16_t* x, const uint16_t* dy,
                          const mxfp4_moe_grads* grads, float* dw, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ------------------------------------------------- 8-bit dense products */

/* An 8-bit matrix of `rows` rows and K columns:
 *  codes   uint8 [rows, Kp], Kp = K rounded up to 128: OCP E4M3, the bytes
 *          past K zero; 16-byte aligned
 *  scales  uint8 UE8M0 (value 2^(s - 127)), K block by K block of 128:
 *          block_rows == 1:   [Kp / 128, rows rounded up to 16], one scale
 *                             for 1 x 128 elements, 16-byte aligned; the
 *                             bytes past `rows` are not used
 *          block_rows == 128: [Kp / 128, ceil(rows / 128)], one scale for
 *                             128 x 128 elements
 * Scales are powers of two alone: a matrix with fp32 scales has to be
 * dequantized and quantized here again.
 * Scale of a block: the smallest 2^e with its largest finite magnitude at
 * most 448 * 2^e, e in [-127, 127] (all zeros: -127).  Element: the nearest
 * E4M3 value to x / 2^e, ties to even; a non-finite x has the NaN code.
 * rows and K are >= 1, K <= 2^22, rows < 2^27, (rows + 127) * Kp < 2^35; a
 * product's M * N < 2^37 (both rounded up to 128), and N <= 2^27 - 16 where
 * M <= 16. */

/* Quantizers.  x [rows, K], dtype MXMOE_F32 or MXMOE_BF16 (any alignment of
 * the dtype's; 16 bytes and K % 8 == 0 run faster).  block_rows 1 or 128. */
#define MXMOE_F32 0
#define MXMOE_BF16 1
int mxmoe_fp8_quantize(const void* x, int dtype, int64_t rows, int64_t K, int block_rows,
                       uint8_t* codes, uint8_t* scales, void* stream);
/* The transpose of x as an 8-bit matrix of K rows and `rows` columns with
 * block_rows 1 (blocks run along x's rows); rows <= 2^22. */
int mxmoe_fp8_quantize_t(const void* x, int dtype, int64_t rows, int64_t K, uint8_t* codes,
                         uint8_t* scales, void* stream);
/* The transpose of an 8-bit matrix with block_rows 128, exactly: codes_t
 * [K, rows rounded up to 128], scales_t [ceil(rows / 128), Kp / 128]. */
int mxmoe_fp8_transpose(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                        uint8_t* codes_t, uint8_t* scales_t, void* stream);

/* out [M, N] = X W^T + bias for 8-bit X [M, K] (block_rows 1) and W [N, K]
 * (block_rows w_block_rows); bias bf16 [N] or NULL; out bf16 or fp32
 * (out_dtype), 16-byte aligned, rounded once.  fp32 results: products and
 * sums in fp32 (values below 2^-126 may count as 0).  bf16 results: fp32
 * sums over K blocks, but within a K block the block-scaled matrix core
 * drops what lies below 2^-13 of its largest product (about 1.5e-5 of a
 * result over random values, a hundredth of its rounding to bf16).  A NaN in
 * a row of X or W stays in that row of the result.  The order of the sums,
 * and so the result's last bits, depend on M, N and K alone. */
int mxmoe_fp8_matmul(int64_t M, int64_t N, int64_t K, const uint8_t* x_codes,
                     const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                     int w_block_rows, const uint16_t* bias, int out_dtype, void* out,
                     void* workspace, size_t workspace_bytes, void* stream);
/* The same from bf16 rows x [M, K], which are quantized with block_rows 1
 * (in the product's own launch for few rows, else into the workspace), and
 * W with block_rows 128.  A linear layer's input gradient is this product
 * of dy [M, N] with the transposed W. */
int mxmoe_fp8_linear(int64_t M, int64_t N, int64_t K, const uint16_t* x, const uint8_t* w_codes,
                     const uint8_t* w_scales, const uint16_t* bias, int out_dtype, void* out,
                     void* workspace, size_t workspace_bytes, void* stream);
/* The weights' gradient of a linear layer: dw fp32 [N, K] = dy^T x with dy
 * bf16 [M, N] and x bf16 [M, K], both quantized in blocks of 128 tokens of
 * one column.  M <= 2^22. */
int mxmoe_fp8_linear_dw(int64_t M, int64_t N, int64_t K, const uint16_t* dy, const uint16_t* x,
                        float* dw, void* workspace, size_t workspace_bytes, void* stream);
/* Bytes of workspace of the three products; 0 if a size is out of range. */
size_t mxmoe_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype);
size_t mxmoe_fp8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype);
size_t mxmoe_fp8_linear_dw_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* ------------------------------------------- 8-bit activation checkpoints */

/* The clamped SwiGLU of mxfp4_moe.h on rows h bf16 [R, 2I] (gate 2j, up
 * 2j + 1), with an 8-bit checkpoint of h: codes uint8 [R, 2I] (OCP E4M3) and
 * scales uint8 [R, 2I / 32] (UE8M0, scale rule as above with blocks of 32).
 * A code is the nearest whose value lies on the same side of the clamp
 * bounds as the element (gate: above limit or not; up: above limit, below
 * -limit or neither), so a backward pass from the checkpoint takes the
 * forward's clamp decisions.  Non-finite elements have the NaN code.
 * R >= 1, I % 16 == 0, alpha finite, limit > 0 and finite; tensors 16-byte
 * aligned; R * 2I <= 2^35 - 2048. */

/* a bf16 [R, I] out (NULL: the checkpoint alone). */
int mxmoe_swiglu8_forward(const uint16_t* h, int64_t R, int64_t I, float alpha, float limit,
                          uint16_t* a, uint8_t* codes, uint8_t* scales, void* stream);
/* dh bf16 [R, 2I] = the derivative at the checkpoint's values times da bf16
 * [R, I] (no gradient beyond a clamp bound); a bf16 [R, I], the activation
 * of the checkpoint's values, or NULL. */
int mxmoe_swiglu8_backward(const uint8_t* codes, const uint8_t* scales, const uint16_t* da,
                           int64_t R, int64_t I, float alpha, float limit, uint16_t* dh,
                           uint16_t* a, void* stream);
/* h bf16 [R, 2I], the checkpoint's values (exact unless below bf16's
 * subnormals; a magnitude from 2^128 - 2^123 on has rounded to 2^128 and is an
 * infinity), and their activation a bf16 [R, I]; either may be NULL. */
int mxmoe_swiglu8_restore(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t I,
                          float alpha, float limit, uint16_t* h, uint16_t* a, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXMOE_OPS_H */
