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
 * all -inf has scores 0. */
typedef struct mxmoe_route_opts {
  int32_t score;
  int32_t groups;
  int32_t top_groups;
  int32_t group_score;
  int32_t renorm;
  float scale;
} mxmoe_route_opts;

/* Routing of T tokens over E experts (E <= 256, 1 <= k <= 8, k at most the
 * experts of top_groups groups, T * k < 2^31).
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

#ifdef __cplusplus
}
#endif

#endif /* MXMOE_OPS_H */
