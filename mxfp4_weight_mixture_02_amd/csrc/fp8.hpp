// Launchers of the 8-bit floating point products (fp8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxmoe {

constexpr int64_t fp8_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
// Bytes of a row of codes for K elements, and of a K block's row of scales
// for `rows` rows with a scale each.
constexpr int64_t fp8_pitch(int64_t K) { return fp8_up(K, 128); }
constexpr int64_t fp8_scale_pitch(int64_t rows) { return fp8_up(rows, 16); }

// x [rows, K] (bf16, or fp32 with x_f32) in blocks of 1 x 128 -> codes
// [rows, pitch(K)], scales [K blocks, scale_pitch(rows)]
hipError_t launch_fp8_quantize_rows(const void* x, int x_f32, int64_t rows, int64_t K,
                                    uint8_t* codes, uint8_t* scales, hipStream_t s);
// the same of x's transpose: blocks of 128 rows of one column -> codes [K,
// pitch(rows)], scales [row blocks, scale_pitch(K)]
hipError_t launch_fp8_quantize_cols(const void* x, int x_f32, int64_t rows, int64_t K,
                                    uint8_t* codes, uint8_t* scales, hipStream_t s);
// the same of two bf16 matrices of as many rows
hipError_t launch_fp8_quantize_cols_pair(const uint16_t* x, int64_t K, uint8_t* codes, uint8_t* scales,
                                         const uint16_t* x2, int64_t K2, uint8_t* codes2,
                                         uint8_t* scales2, int64_t rows, hipStream_t s);
// blocks of 128 x 128 -> codes [rows, pitch(K)], scales [K blocks, row blocks]
hipError_t launch_fp8_quantize_blocks(const void* x, int x_f32, int64_t rows, int64_t K,
                                      uint8_t* codes, uint8_t* scales, hipStream_t s);
// 128 x 128-block codes and scales of w [rows, K] -> those of its transpose
hipError_t launch_fp8_transpose(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t K, uint8_t* codes_t, uint8_t* scales_t, hipStream_t s);

struct Fp8Gemm {
  int64_t M, N, K;
  const uint8_t *x, *sx;    // codes and scales of X [M, K], blocks of 1 x 128
  const uint8_t *w, *sw;    // of W [N, K]: blocks of 128 x 128, or 1 x 128 with w_rows
  int w_rows;
  const uint16_t* bias;     // bf16 [N] or nullptr
  void* out;                // [M, N], bf16 or fp32 with out_f32
  int out_f32;
  float* part;              // fp8_part_bytes of scratch
};
// out = X W^T + bias
size_t fp8_part_bytes(int64_t M, int64_t N, int64_t K, int out_f32);
hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t s);
// the same from bf16 rows x (rounded inside) for few rows
bool fp8_fused_fits(int64_t M, int64_t N, int64_t K);
hipError_t launch_fp8_fused(const Fp8Gemm& g, const uint16_t* x, hipStream_t s);

}  // namespace mxmoe
