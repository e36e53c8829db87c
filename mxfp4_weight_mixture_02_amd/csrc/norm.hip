// Root-mean-square norm of the rows of a residual stream (gfx950), with the
// residual's addition before it and its result in bf16, in 8 bits with scales
// or both; and its gradients.
//
//   s = x + r (rounded to their type: the new stream)
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
//   dx = rstd (w dy - xhat mean(w dy xhat)) + ds,  dw = sum over rows of dy xhat,
//   xhat = s rstd
//
// One pass over the data: a row lives in the registers of NW waves, C chunks
// of 8 elements a lane, so that 16 lanes side by side hold one 128-element
// block of the 8-bit result.  Squares, means and the weight's gradient are
// summed in fp32; everything is rounded once, when it is stored.
#include "common.hpp"
#include "fp8.hpp"
#include "norm.hpp"

namespace mxmoe {

// Eight consecutive elements as they are stored, zeros from `left` on.
template <bool F32>
struct Raw8 {
  u32x4 q[F32 ? 2 : 1];
};
template <bool F32, bool VEC>
__device__ __forceinline__ Raw8<F32> raw8(const void* x, int64_t at, int64_t left) {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.q[i] = u32x4{0u, 0u, 0u, 0u};
  if (VEC) {
    if (left > 0) {
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(x) + at * (F32 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < (F32 ? 2 : 1); ++i) r.q[i] = p[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) {
        if (F32)
          r.q[i >> 2][i & 3] = static_cast<const uint32_t*>(x)[at + i];
        else
          r.q[0][i >> 1] |= (uint32_t)static_cast<const uint16_t*>(x)[at + i] << (16 * (i & 1));
      }
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ float value(const Raw8<F32>& r, int i) {
  if (F32) return __uint_as_float(r.q[F32 ? i >> 2 : 0][i & 3]);
  const uint32_t w = r.q[0][i >> 1];
  return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
}
// The weight's eight elements: its type is an argument, not a template's (the
// branch is uniform).
template <bool VEC>
__device__ __forceinline__ void weight8(const NormArgs& a, int64_t k0, float (&w)[8]) {
  if (a.w_f32) {
    const Raw8<true> r = raw8<true, VEC>(a.w, k0, a.H - k0);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = value<true>(r, i);
  } else {
    const Raw8<false> r = raw8<false, VEC>(a.w, k0, a.H - k0);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = value<false>(r, i);
  }
}
// Eight values rounded to fp32 or bf16, those before `left`.
template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void* p, int64_t at, int64_t left, const float (&v)[8]) {
  if (VEC) {
    if (left <= 0) return;
    u32x4* d = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p) + at * (F32 ? 4 : 2));
    if (F32) {
      d[0] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
      d[1] = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
    } else {
      d[0] = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) {
      if (F32)
        static_cast<float*>(p)[at + i] = v[i];
      else
        static_cast<uint16_t*>(p)[at + i] = (uint16_t)f32_to_bf16(v[i]);
    }
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
// The sum over a row's NW waves, in their order.  Called by all of them.
template <int NW, class V>
__device__ __forceinline__ V row_sum(V v, V* slots, int wave, int lane) {
  v = wave_sum(v);
  if (NW == 1) return v;
  __syncthreads();   // the slots' last readers are done
  if (lane == 0) slots[wave] = v;
  __syncthreads();
  v = slots[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) v += slots[i];
  return v;
}

// 1 / sqrt(mean of the squares + eps).  A sum of squares that fp32 cannot
// hold (elements from about 1e18 on, or a tiny eps under tiny elements) is
// formed again in fp64; a NaN or an infinity in the row stays one.
template <int NW, int C>
__device__ __forceinline__ float row_rstd(const float (&v)[C][8], int64_t H, float eps, double* slots, int wave,
                                          int lane) {
  // sums of 8, of the chunks, then in fp64 over the lanes: the reciprocal's
  // own error decides how many 8-bit elements round the other way
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = fmaf(v[c][i], v[c][i], t);
    ss += t;
  }
  const double m = row_sum<NW>((double)ss, slots, wave, lane) / (double)H + (double)eps;
  if (m > 1e-30 && m < 3e38) return (float)(1.0 / sqrt(m));
  double sd = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sd += (double)v[c][i] * (double)v[c][i];
  sd = row_sum<NW>(sd, slots, wave, lane);
  return (float)(1.0 / sqrt(sd / (double)H + (double)eps));
}

// A row for NW waves; four waves a workgroup, or NW where that is more.  Bound
// by HBM: 16381 x 2880 bf16 with the residual, both results: 85 us, 5.0 TB/s;
// 2047 x 2880 fp32, bf16 result: 15.6 us, 5.3 TB/s.  One row: 3.7 us.
template <bool F32, bool VEC, int NW, int C>
__global__ __launch_bounds__(64 * (NW < 4 ? 4 : NW)) void norm_kernel(NormArgs a) {
  __shared__ double slots[NW];
  const int lane = threadIdx.x & 63, all = threadIdx.x >> 6, wave = all % NW;
  const int64_t row = (int64_t)blockIdx.x * (NW < 4 ? 4 / NW : 1) + all / NW;
  if (row >= a.T) return;   // whole waves, and with NW >= 4 none
  Raw8<F32> x[C], r[C];
  const int64_t at = row * a.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
    x[c] = raw8<F32, VEC>(a.x, at + k0, a.H - k0);
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
      r[c] = raw8<F32, VEC>(a.residual, at + k0, a.H - k0);
    }
  }
  float v[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = value<F32>(x[c], i);
    if (a.residual) {
      const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] += value<F32>(r[c], i);
        if (!F32) v[c][i] = bf16_to_f32((uint16_t)f32_to_bf16(v[c][i]));   // the stream as it is stored
      }
      store8<F32, VEC>(a.sum, at + k0, a.H - k0, v[c]);
    }
  }
  const float rstd = row_rstd<NW, C>(v, a.H, a.eps, slots, wave, lane);
  if (wave == 0 && lane == 0) a.rstd[row] = rstd;
  const int64_t pitch = fp8_pitch(a.H), spitch = fp8_scale_pitch(a.T);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
    float w[8];
    weight8<VEC>(a, k0, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * rstd * w[i];
    if (a.y) store8<false, VEC>(a.y, at + k0, a.H - k0, v[c]);
    if (a.codes) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (k0 + i >= a.H) v[c][i] = 0.0f;   // past the row: 0 times a NaN is one
        m = max(m, finite_bits(v[c][i]));
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
      const int e = e4m3_exponent(m);
      const float f = e4m3_inverse(e);
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = nan_unless_finite(v[c][i]) * f;
      if (k0 < pitch) {
        *reinterpret_cast<u32x2*>(a.codes + row * pitch + k0) =
            u32x2{e4m3_pack4(q[0], q[1], q[2], q[3]), e4m3_pack4(q[4], q[5], q[6], q[7])};
        if ((lane & 15) == 0) a.scales[(k0 >> 7) * spitch + row] = (uint8_t)(e + 127);
      }
    }
  }
}

// Gradients.  Workgroup b takes the row groups b, b + gridDim.x, ..; each lane
// sums its columns' part of dw over its rows, the workgroup's waves add theirs
// in order through LDS, and the parts [workgroups][H] are joined by another
// launch (one workgroup writes dw itself).  Bound by HBM: 16384 x 2880 bf16
// with the sum's own gradient in 77.8 us (4.8 TB/s), the join 5.5.
template <bool F32, bool VEC, int NW, int C>
__global__ __launch_bounds__(64 * (NW < 4 ? 4 : NW)) void norm_bwd_kernel(NormArgs a) {
  constexpr int ROWS = NW < 4 ? 4 / NW : 1;   // rows at a time
  __shared__ double slots[NW];
  __shared__ float add[ROWS == 1 ? 1 : C * NW * 512];
  const int lane = threadIdx.x & 63, all = threadIdx.x >> 6, wave = all % NW;
  float dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  const int64_t groups = (a.T + ROWS - 1) / ROWS;
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t row = g * ROWS + all / NW;
    if (row >= a.T) break;   // whole waves, and with NW >= 4 none: no barrier is missed
    const int64_t at = row * a.H;
    Raw8<F32> x[C], ds[C];
    Raw8<false> dy[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
      x[c] = raw8<F32, VEC>(a.x, at + k0, a.H - k0);
      dy[c] = raw8<false, VEC>(a.dy, at + k0, a.H - k0);
    }
    if (a.residual) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
        ds[c] = raw8<F32, VEC>(a.residual, at + k0, a.H - k0);
      }
    }
    const float rstd = a.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
      float w[8];
      weight8<VEC>(a, k0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = value<false>(dy[c], i) * (value<F32>(x[c], i) * rstd);
        dw[c][i] += p;
        dot = fmaf(w[i], p, dot);
      }
    }
    dot = row_sum<NW>(dot, reinterpret_cast<float*>(slots), wave, lane) / (float)a.H;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
      float w[8], d[8];
      weight8<VEC>(a, k0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = rstd * (w[i] * value<false>(dy[c], i) - value<F32>(x[c], i) * rstd * dot);
        if (a.residual) d[i] += value<F32>(ds[c], i);
      }
      store8<F32, VEC>(a.sum, at + k0, a.H - k0, d);
    }
  }
  if (ROWS > 1) {   // the waves' sums, one wave after the other
#pragma unroll 1
    for (int u = 0; u < ROWS; ++u) {
      if (all / NW == u) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = &add[((c * NW + wave) * 8 + i) * 64 + lane];
            dw[c][i] = u ? *p + dw[c][i] : dw[c][i];
            *p = dw[c][i];
          }
      }
      __syncthreads();
    }
    if (all / NW != ROWS - 1) return;   // the last one has the sum
  }
  float* out = gridDim.x == 1 ? a.dw : a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k0 = ((int64_t)(c * NW + wave) * 64 + lane) * 8;
    if (VEC && gridDim.x > 1)
      store8<true, true>(out, k0, a.H - k0, dw[c]);
    else
      store8<true, false>(out, k0, a.H - k0, dw[c]);   // dw may have any alignment
  }
}

// dw: the parts' sum, 64 columns a workgroup, 16 slices of the parts side by
// side, joined in their order.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* __restrict__ part, int64_t H, int parts,
                                                         float* __restrict__ dw) {
  __shared__ float slots[16][64];
  const int c = threadIdx.x & 63, u = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + c;
  float v = 0.0f;
  if (k < H) {
#pragma unroll 8
    for (int p = u; p < parts; p += 16) v += part[(int64_t)p * H + k];
  }
  slots[u][c] = v;
  __syncthreads();
  if (u || k >= H) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) v += slots[i][c];
  dw[k] = v;
}

// ------------------------------------------------------------------ launchers

static bool norm_vec(const NormArgs& a) {
  auto ok = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  return a.H % 8 == 0 && ok(a.x) && ok(a.residual) && ok(a.w) && ok(a.sum) && ok(a.y) && ok(a.dy);
}

// Waves of a row and chunks of a lane, forward.  One wave a row moves most
// bytes while rows fill the card; fewer rows, or longer ones, take more waves.
struct NormShape {
  int nw, c;
};
static NormShape norm_shape(int64_t T, int64_t H) {
  const int w = (int)((H + 511) / 512);   // chunks of one wave
  if (w <= 6 && T >= 1024) return {1, w <= 2 ? 2 : w <= 4 ? 4 : 6};
  if (w <= 16) return {4, w <= 4 ? 1 : w <= 8 ? 2 : 4};
  return {16, w <= 32 ? 2 : 4};
}
// Backward: a lane also holds the weight and its part of dw, so rows are split
// wider, to 16 waves on a CU (16384 x 2880: one wave a row, 4 on a CU, 138 us;
// four waves, 105 registers, 8 on a CU 109 us, 16 on a CU 84; twice as many
// workgroups and parts 91).
static NormShape norm_bwd_shape(int64_t H) {
  const int w = (int)((H + 511) / 512);
  if (w <= 2) return {1, w};
  if (w <= 8) return {4, w <= 4 ? 1 : 2};
  if (w <= 16) return {8, 2};
  return {16, w <= 32 ? 2 : 4};
}
int64_t norm_blocks(int64_t T, int64_t H) { return norm_shape(T, H).nw == 1 ? (T + 3) / 4 : T; }
int norm_threads(int64_t T, int64_t H) { return norm_shape(T, H).nw == 16 ? 1024 : 256; }
static unsigned norm_bwd_grid(int64_t T, int64_t H) {
  const int nw = norm_bwd_shape(H).nw;
  const int64_t groups = nw == 1 ? (T + 3) / 4 : T, most = nw <= 4 ? 1024 : 4096 / nw;
  return (unsigned)(groups < most ? groups : most);
}

#define NORM_LAUNCH(kernel, grid, NW, C)                                                  \
  do {                                                                                    \
    const dim3 g_((unsigned)(grid)), b_(64 * (NW < 4 ? 4 : NW));                          \
    const bool vec_ = norm_vec(a);                                                        \
    if (a.f32 && vec_) hipLaunchKernelGGL((kernel<true, true, NW, C>), g_, b_, 0, s, a);  \
    else if (a.f32) hipLaunchKernelGGL((kernel<true, false, NW, C>), g_, b_, 0, s, a);    \
    else if (vec_) hipLaunchKernelGGL((kernel<false, true, NW, C>), g_, b_, 0, s, a);     \
    else hipLaunchKernelGGL((kernel<false, false, NW, C>), g_, b_, 0, s, a);              \
    return hipGetLastError();                                                             \
  } while (0)

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const int64_t grid = norm_blocks(a.T, a.H);
  const NormShape n = norm_shape(a.T, a.H);
  switch (100 * n.nw + n.c) {
    case 102: NORM_LAUNCH(norm_kernel, grid, 1, 2);
    case 104: NORM_LAUNCH(norm_kernel, grid, 1, 4);
    case 106: NORM_LAUNCH(norm_kernel, grid, 1, 6);
    case 401: NORM_LAUNCH(norm_kernel, grid, 4, 1);
    case 402: NORM_LAUNCH(norm_kernel, grid, 4, 2);
    case 404: NORM_LAUNCH(norm_kernel, grid, 4, 4);
    case 1602: NORM_LAUNCH(norm_kernel, grid, 16, 2);
    default: NORM_LAUNCH(norm_kernel, grid, 16, 4);
  }
}

size_t norm_part_bytes(int64_t T, int64_t H) {
  const unsigned g = norm_bwd_grid(T, H);
  return g == 1 ? 0 : (size_t)g * H * sizeof(float);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  if (norm_part_bytes(a.T, a.H) && !a.part) return hipErrorInvalidValue;
  const unsigned grid = norm_bwd_grid(a.T, a.H);
  const NormShape n = norm_bwd_shape(a.H);
  switch (100 * n.nw + n.c) {
    case 101: NORM_LAUNCH(norm_bwd_kernel, grid, 1, 1);
    case 102: NORM_LAUNCH(norm_bwd_kernel, grid, 1, 2);
    case 401: NORM_LAUNCH(norm_bwd_kernel, grid, 4, 1);
    case 402: NORM_LAUNCH(norm_bwd_kernel, grid, 4, 2);
    case 802: NORM_LAUNCH(norm_bwd_kernel, grid, 8, 2);
    case 1602: NORM_LAUNCH(norm_bwd_kernel, grid, 16, 2);
    default: NORM_LAUNCH(norm_bwd_kernel, grid, 16, 4);
  }
}

hipError_t launch_norm_join(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((a.H + 63) / 64)), dim3(1024), 0, s, a.part, a.H,
                     (int)norm_bwd_grid(a.T, a.H), a.dw);
  return hipGetLastError();
}

}  // namespace mxmoe
