// Launchers of the root-mean-square norm (norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxmoe {

constexpr int64_t NORM_MAX_H = 32768;   // a row stays in one workgroup's registers

struct NormArgs {
  int64_t T, H;
  int f32;                  // x, residual, sum, dsum and dx: fp32, else bf16
  int w_f32;                // weight: fp32, else bf16
  float eps;
  const void* x;            // [T, H]; backward: the sum that was normed
  const void* residual;     // [T, H] or nullptr; backward: the sum's own gradient
  const void* w;            // [H]
  void* sum;                // x + residual, with a residual; backward: dx
  uint16_t* y;              // bf16 [T, H] or nullptr
  uint8_t *codes, *scales;  // 8-bit y (blocks of 1 x 128) or nullptr
  float* rstd;              // [T]
  const uint16_t* dy;       // backward: bf16 [T, H]
  float* dw;                // backward: fp32 [H]
  float* part;              // norm_part_bytes of scratch
};
// workgroups of a forward launch and their threads (a backward one has at most
// 1024 workgroups)
int64_t norm_blocks(int64_t T, int64_t H);
int norm_threads(int64_t T, int64_t H);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
size_t norm_part_bytes(int64_t T, int64_t H);   // 0: one workgroup, no scratch
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_join(const NormArgs& a, hipStream_t s);

}  // namespace mxmoe
