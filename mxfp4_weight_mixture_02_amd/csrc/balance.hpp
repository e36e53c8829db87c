// Launchers of the router's balance losses (balance.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxmoe {

struct BalanceArgs {
  int64_t T;
  int E, k, S;
  int sigmoid;
  const float* logits;      // [T, E]
  const int32_t* topk_idx;  // [T, k]
  const uint8_t* mask;      // [T] or nullptr: nonzero counts
  const int32_t* offsets;   // [S + 1] or nullptr: one sequence of all tokens
  float* losses;            // [2]
  int32_t* counts;          // [S, E]
  float* prob;              // [S, E]
  int32_t* tokens;          // [S]
};
size_t balance_ws_bytes(int64_t T, int E, int S);
// all launches of a forward: balance_launches of them, numbered from 0
int balance_launches(int64_t T, int E, int S);
hipError_t launch_balance(const BalanceArgs& a, int which, void* ws, hipStream_t s);
// dlogits [T, E] from counts, tokens and dlosses [2], plus add [T, E] or nullptr
hipError_t launch_balance_bwd(const BalanceArgs& a, const float* dlosses, const float* add, float* dlogits,
                              hipStream_t s);

}  // namespace mxmoe
