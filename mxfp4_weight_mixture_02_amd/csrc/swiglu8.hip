// The clamped SwiGLU with an 8-bit checkpoint of its input (gfx950): forward
// with the checkpoint, backward from the checkpoint, and the restoration of
// the bf16 input and activation.
//
// The checkpoint is MXFP8 of h along a row (E4M3, one power-of-two scale for
// each 32 elements: 16 gates and their 16 ups), 1.03 bytes an element
// against 2 for h and 3 for h with the activation a.  A code is the nearest
// one that lies on its value's side of the clamp bounds (a gate at most
// `limit` stays at most `limit`, an up within +-limit stays within), so the
// backward takes the forward's clamp decisions; a value rounded across a
// bound takes the neighbouring code.
//
// All three are streaming kernels bound by HBM: a lane owns 8 elements of h
// (16 bytes), four lanes a scale block.  With I = 2880 and 65536 rows the
// forward takes 312 us (4.9 TB/s; a copy reaches 4.7), the backward with a
// again 294 us (6.5 TB/s, the last-level cache helping); with 8192 rows 41 and
// 36 us, and the restoration of h and a 30 us; with 64 rows 3 us, a launch.
#include "common.hpp"
#include "swiglu8.hpp"

namespace mxmoe {

// 2^e for e in [-127, 127]
__device__ __forceinline__ float ck_two(int e) {
  return e == -127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

// The values of 8 codes (two words) of a block with exponent e.
__device__ __forceinline__ void ck_values(u32x2 c, int e, float (&v)[8]) {
  const float f = ck_two(e);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], true);
    v[4 * w] = lo[0] * f;
    v[4 * w + 1] = lo[1] * f;
    v[4 * w + 2] = hi[0] * f;
    v[4 * w + 3] = hi[1] * f;
  }
}

// 8 values (4 gate/up pairs) to codes, with the clamp sides kept.  The four
// lanes of a block call it together; e returns the block's exponent.
__device__ __forceinline__ u32x2 ck_encode(const float (&v)[8], float limit, int* e_out) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[i]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  const int e = e4m3_exponent(m);
  const float f = e4m3_inverse(e);
  u32x2 c;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float* x = v + 4 * w;
    c[w] = e4m3_pack4(nan_unless_finite(x[0]) * f, nan_unless_finite(x[1]) * f,
                      nan_unless_finite(x[2]) * f, nan_unless_finite(x[3]) * f);
  }
  // The next code up is the next magnitude.  It cannot reach the NaN code: a
  // value above the bound whose rounding is not is below the block's largest
  // value 448 * 2^e; and a code that is lowered is above 0.
  float r[8];
  ck_values(c, e, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int d = (int)(v[i] > limit) - (int)(r[i] > limit);
    if (i & 1) d += (int)(v[i] < -limit) - (int)(r[i] < -limit);
    if (non_finite(v[i])) d = 0;
    c[i >> 2] += (uint32_t)d << (8 * (i & 3));
  }
  *e_out = e;
  return c;
}

__device__ __forceinline__ void bf16x8_values(u32x4 a, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}

// swiglu() with NaN inputs kept (its clamps drop them), and 0 for a gate of
// -inf (whose sigmoid 0 would be multiplied by an infinity).
__device__ __forceinline__ float act(float g, float u, float alpha, float limit) {
  const float a = swiglu(fmaxf(g, -3.402823466e38f), u, alpha, limit);
  return g != g || u != u ? __uint_as_float(0x7FC00000u) : a;
}

__global__ __launch_bounds__(256) void swiglu8_fwd_kernel(const u32x4* __restrict__ h, int64_t n8,
                                                          float alpha, float limit,
                                                          u32x2* __restrict__ a,
                                                          u32x2* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;   // whole groups of 4 lanes: n8 is a multiple of 4
  float v[8];
  bf16x8_values(h[i], v);
  int e;
  const u32x2 c = ck_encode(v, limit, &e);
  codes[i] = c;
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)(e + 127);
  if (a)
    a[i] = u32x2{pack_bf16x2(act(v[0], v[1], alpha, limit), act(v[2], v[3], alpha, limit)),
                 pack_bf16x2(act(v[4], v[5], alpha, limit), act(v[6], v[7], alpha, limit))};
}

__global__ __launch_bounds__(256) void swiglu8_bwd_kernel(const u32x2* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          const u32x2* __restrict__ da, int64_t n8,
                                                          float alpha, float limit,
                                                          u32x4* __restrict__ dh,
                                                          u32x2* __restrict__ a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  ck_values(codes[i], (int)scales[i >> 2] - 127, v);
  const u32x2 d = da[i];
  u32x4 o;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float x = __uint_as_float((p & 1) ? (d[p >> 1] & 0xFFFF0000u) : (d[p >> 1] << 16));
    float dg, du;
    swiglu_grad<true>(v[2 * p], v[2 * p + 1], x, alpha, limit, &dg, &du);
    o[p] = pack_bf16x2(dg, du);
  }
  dh[i] = o;
  if (a)
    a[i] = u32x2{pack_bf16x2(act(v[0], v[1], alpha, limit), act(v[2], v[3], alpha, limit)),
                 pack_bf16x2(act(v[4], v[5], alpha, limit), act(v[6], v[7], alpha, limit))};
}

__global__ __launch_bounds__(256) void swiglu8_restore_kernel(const u32x2* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              int64_t n8, float alpha, float limit,
                                                              u32x4* __restrict__ h,
                                                              u32x2* __restrict__ a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  ck_values(codes[i], (int)scales[i >> 2] - 127, v);
  if (h)   // exact: 4 significant bits and a power of two
    h[i] = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7])};
  if (a)
    a[i] = u32x2{pack_bf16x2(act(v[0], v[1], alpha, limit), act(v[2], v[3], alpha, limit)),
                 pack_bf16x2(act(v[4], v[5], alpha, limit), act(v[6], v[7], alpha, limit))};
}

hipError_t launch_swiglu8_fwd(const uint16_t* h, int64_t n8, float alpha, float limit, uint16_t* a,
                              uint8_t* codes, uint8_t* scales, hipStream_t s) {
  hipLaunchKernelGGL(swiglu8_fwd_kernel, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s,
                     reinterpret_cast<const u32x4*>(h), n8, alpha, limit,
                     reinterpret_cast<u32x2*>(a), reinterpret_cast<u32x2*>(codes), scales);
  return hipGetLastError();
}

hipError_t launch_swiglu8_bwd(const uint8_t* codes, const uint8_t* scales, const uint16_t* da,
                              int64_t n8, float alpha, float limit, uint16_t* dh, uint16_t* a,
                              hipStream_t s) {
  hipLaunchKernelGGL(swiglu8_bwd_kernel, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s,
                     reinterpret_cast<const u32x2*>(codes), scales,
                     reinterpret_cast<const u32x2*>(da), n8, alpha, limit,
                     reinterpret_cast<u32x4*>(dh), reinterpret_cast<u32x2*>(a));
  return hipGetLastError();
}

hipError_t launch_swiglu8_restore(const uint8_t* codes, const uint8_t* scales, int64_t n8,
                                  float alpha, float limit, uint16_t* h, uint16_t* a, hipStream_t s) {
  hipLaunchKernelGGL(swiglu8_restore_kernel, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s,
                     reinterpret_cast<const u32x2*>(codes), scales, n8, alpha, limit,
                     reinterpret_cast<u32x4*>(h), reinterpret_cast<u32x2*>(a));
  return hipGetLastError();
}

}  // namespace mxmoe
