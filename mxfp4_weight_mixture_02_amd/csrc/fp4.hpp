// Launchers of the 4-bit products (fp4.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.hpp"

namespace mxmoe {

// Bytes of a padded row of codes for K elements; blocks of 256 of K, and rows
// of scales of one.
constexpr int64_t fp4_pitch(int64_t K) { return fp8_up(K, 256) / 2; }
constexpr int64_t fp4_kblocks(int64_t K) { return fp8_up(K, 256) / 256; }
constexpr int64_t fp4_scale_rows(int64_t rows) { return fp8_up(rows, 16); }
constexpr int64_t fp4_scale_bytes(int64_t rows, int64_t K) { return fp4_kblocks(K) * 8 * fp4_scale_rows(rows); }

// x [rows, K] (bf16, or fp32 with x_f32) -> codes [rows, fp4_pitch(K)] and
// scales [K blocks, 4, scale_rows(rows), 2]
hipError_t launch_fp4_quantize(const void* x, int x_f32, int64_t rows, int64_t K, uint8_t* codes, uint8_t* scales,
                               hipStream_t s);
// scales [rows, K / 32] -> the same order
hipError_t launch_fp4_scales(const uint8_t* scales, int64_t rows, int64_t K, uint8_t* ordered, hipStream_t s);

struct Fp4Gemm {
  int64_t M, N, K;
  const uint8_t *x, *sx;   // codes [M, fp4_pitch(K)] and scales of X
  const uint8_t *w, *sw;   // codes [N, wp] and scales of W
  int64_t wp;              // bytes of a row of W's codes: K / 2 or fp4_pitch(K)
  const uint16_t* bias;    // bf16 [N] or nullptr
  void* out;               // [M, N], bf16 or fp32 with out_f32
  int out_f32;
  float* part;             // fp4_part_bytes of scratch
};
// out = X W^T + bias
size_t fp4_part_bytes(int64_t M, int64_t N, int64_t K, int out_f32);
hipError_t launch_fp4_gemm(const Fp4Gemm& g, hipStream_t s);
// the same from bf16 rows x (rounded inside) for few rows
bool fp4_fused_fits(int64_t M, int64_t N, int64_t K);
hipError_t launch_fp4_fused(const Fp4Gemm& g, const uint16_t* x, hipStream_t s);

// out [M, K] = X W for bf16 rows x [M, N] (of g: N and K of W, w, wp, sw, out,
// out_f32, part of fp4_dx_few_bytes), where that is the faster way
bool fp4_dx_few(int64_t M, int64_t N, int64_t K, int out_f32);
size_t fp4_dx_few_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_fp4_dx_few(const Fp4Gemm& g, const uint16_t* x, hipStream_t s);
// W [N, K] -> its transpose in bf16 [K, N rounded up to 64], zeros past N
hipError_t launch_fp4_dequant_t(const uint8_t* w, int64_t wp, const uint8_t* sw, int64_t N, int64_t K, uint16_t* wt,
                                hipStream_t s);
// x [rows, K] -> [rows, K rounded up to 64], zeros past K
hipError_t launch_bf16_pad(const uint16_t* x, int64_t rows, int64_t K, uint16_t* out, hipStream_t s);
// out = X W^T for bf16 X [M, K] and W [N, K], K % 64 == 0 (of g: sizes, x, w
// as bf16 rows, out, out_f32, part)
size_t bf16_part_bytes(int64_t M, int64_t N, int64_t K, int out_f32);
hipError_t launch_bf16_gemm(const Fp4Gemm& g, hipStream_t s);

}  // namespace mxmoe
