// Launchers of the routing kernels (gate.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxmoe {

struct RouteArgs {
  int64_t T;
  int E, k;
  int groups, top_groups;   // top_groups == groups: no groups
  int share;                // lanes that value a group: a power of two, share * groups <= 64
  int group_lanes;          // lanes whose experts are a whole group, if a power of two, else 0
  int rows;                 // rows of 16 lanes can read (and write) four experts at a time
  int row_lanes;            // group_lanes of 16 lanes (16 without groups), or 0: not in rows of 16
  int wide;                 // a lane's experts exist together, at their vector's alignment
  int sigmoid, top2, renorm;
  float scale;
  const float* logits;      // [T, E]
  const float* bias;        // [E] or nullptr
  int32_t* topk_idx;        // [T, k]
  float* topk_w;            // [T, k]
  int32_t* offsets;         // [E + 1]
  int32_t* sorted_rows;     // [T * k]
};

// Few tokens (gate_in_one): all in one launch, without workspace.  Else: the
// choice and each workgroup's histogram [gate_blocks(T), E]; then in
// place the rows of earlier workgroups, with the totals [E]; then offsets
// and permutation.
bool gate_in_one(int64_t T);
bool gate_adds(int64_t T);   // few workgroups: the scatter adds up their histograms itself
int64_t gate_blocks(int64_t T);
hipError_t launch_gate_one(const RouteArgs& a, hipStream_t s);
hipError_t launch_gate(const RouteArgs& a, int32_t* hist, hipStream_t s);
hipError_t launch_gate_prefix(const RouteArgs& a, int32_t* hist, int32_t* total, hipStream_t s);
hipError_t launch_gate_scatter(const RouteArgs& a, const int32_t* base, const int32_t* total,
                               hipStream_t s);
hipError_t launch_gate_bwd(const RouteArgs& a, const int32_t* idx, const float* dw, float* dlogits,
                           hipStream_t s);

}  // namespace mxmoe
