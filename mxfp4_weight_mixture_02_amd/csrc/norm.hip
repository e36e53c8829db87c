// Root-mean-square norm of the rows of a residual stream (gfx950), with the
// residual's addition before it and its result in bf16, in 8 bits with scales
// or both; and its gradients.
//
//   s = x + r (rounded to their type: the new stream)
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
//   dx = rstd (w dy - xhat mean(w dy xhat)) + ds,  dw = sum over rows of dy xhat,
//   xhat = s rstd
//
// One pass over the data (but for the gradient of more than 16384 columns): a row
// lives in the registers of LR lanes (16 to 1024), C chunks of 8 elements each, so
// that 16 lanes side by side hold one 128-element block of the 8-bit result.  Squares, means and the weight's gradient are
// summed in fp32; everything is rounded once, when it is stored.
#include "common.hpp"
#include "fp8.hpp"
#include "norm.hpp"

namespace mxmoe {

// Eight consecutive elements as they are stored, zeros from `left` on.  Rows of
// any length begin at any element, and the memory takes 16-byte accesses at any:
// WHOLE (H % 8 == 0) leaves out the rows' ends, which go element by element.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
template <bool F32>
struct Raw8 {
  u32x4 q[F32 ? 2 : 1];
};
template <bool F32, bool WHOLE>
__device__ __forceinline__ Raw8<F32> raw8(const void* x, int64_t at, int64_t left) {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.q[i] = u32x4{0u, 0u, 0u, 0u};
  if (WHOLE ? left > 0 : left >= 8) {
    const u32x4_any* p = reinterpret_cast<const u32x4_any*>(static_cast<const uint8_t*>(x) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) r.q[i] = p[i];
  } else if (!WHOLE) {
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
template <bool WHOLE>
__device__ __forceinline__ void weight8(const NormArgs& a, int64_t k0, float (&w)[8]) {
  if (a.w_f32) {
    const Raw8<true> r = raw8<true, WHOLE>(a.w, k0, a.H - k0);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = value<true>(r, i);
  } else {
    const Raw8<false> r = raw8<false, WHOLE>(a.w, k0, a.H - k0);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = value<false>(r, i);
  }
}
// Eight values rounded to fp32 or bf16, those before `left`.
template <bool F32, bool WHOLE>
__device__ __forceinline__ void store8(void* p, int64_t at, int64_t left, const float (&v)[8]) {
  if (WHOLE ? left > 0 : left >= 8) {
    u32x4_any* d = reinterpret_cast<u32x4_any*>(static_cast<uint8_t*>(p) + at * (F32 ? 4 : 2));
    if (F32) {
      d[0] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
      d[1] = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
    } else {
      d[0] = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  } else if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) {
        if (F32)
          static_cast<float*>(p)[at + i] = v[i];
        else
          static_cast<uint16_t*>(p)[at + i] = (uint16_t)f32_to_bf16(v[i]);
      }
  }
}

// The sum over a row's LR lanes: of a part of a wave, or of whole ones in their
// order, which all call it.
template <int LR, class V>
__device__ __forceinline__ V row_sum(V v, V* slots, int wave, int lane) {
#pragma unroll
  for (int d = 1; d < (LR < 64 ? LR : 64); d <<= 1) v += __shfl_xor(v, d);
  if (LR <= 64) return v;
  __syncthreads();   // the slots' last readers are done
  if (lane == 0) slots[wave] = v;
  __syncthreads();
  v = slots[0];
#pragma unroll
  for (int i = 1; i < LR / 64; ++i) v += slots[i];
  return v;
}

// 1 / sqrt(mean of the squares + eps).  A sum of squares that fp32 cannot
// hold (elements from about 1e18 on, or a tiny eps under tiny elements) is
// formed again in fp64; a NaN or an infinity in the row stays one.
template <int LR, int C>
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
  const double m = row_sum<LR>((double)ss, slots, wave, lane) / (double)H + (double)eps;
  if (m > 1e-30 && m < 3e38) return (float)(1.0 / sqrt(m));
  double sd = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sd += (double)v[c][i] * (double)v[c][i];
  sd = row_sum<LR>(sd, slots, wave, lane);
  return (float)(1.0 / sqrt(sd / (double)H + (double)eps));
}

// The threads of a workgroup whose rows have LR lanes each.
constexpr int norm_block(int lr) { return lr < 256 ? 256 : lr; }

// A row for LR lanes; 256 threads a workgroup, or LR where that is more.  Bound
// by HBM: 16381 x 2880 bf16 with the residual, both results: 85 us, 5.0 TB/s;
// 2047 x 2880 fp32, bf16 result: 15.5 us, 5.3 TB/s; 4096 x 16384 bf16 121 us and
// 4096 x 32768 238, 5.0 TB/s; below some 4000 rows of 2880 by the launch and its
// one round of loads (1024 rows 11 us, 2.4 TB/s).  One row: 3.6 us.
template <bool F32, bool WHOLE, int LR, int C>
__global__ __launch_bounds__(norm_block(LR)) void norm_kernel(NormArgs a) {
  __shared__ double slots[LR < 64 ? 1 : LR / 64];
  const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) % (LR < 64 ? 1 : LR / 64), l = threadIdx.x % LR;
  const int64_t row = (int64_t)blockIdx.x * (norm_block(LR) / LR) + threadIdx.x / LR;
  if (row >= a.T) return;   // all of a row's lanes, and with several waves none
  Raw8<F32> x[C], r[C];
  const int64_t at = row * a.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k0 = (c * LR + l) * 8;
    x[c] = raw8<F32, WHOLE>(a.x, at + k0, a.H - k0);
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = (c * LR + l) * 8;
      r[c] = raw8<F32, WHOLE>(a.residual, at + k0, a.H - k0);
    }
  }
  float v[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = value<F32>(x[c], i);
    if (a.residual) {
      const int64_t k0 = (c * LR + l) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] += value<F32>(r[c], i);
        if (!F32) v[c][i] = bf16_to_f32((uint16_t)f32_to_bf16(v[c][i]));   // the stream as it is stored
      }
      store8<F32, WHOLE>(a.sum, at + k0, a.H - k0, v[c]);
    }
  }
  const float rstd = row_rstd<LR, C>(v, a.H, a.eps, slots, wave, lane);
  if (l == 0) a.rstd[row] = rstd;
  const int64_t pitch = fp8_pitch(a.H), spitch = fp8_scale_pitch(a.T);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k0 = (c * LR + l) * 8;
    float w[8];
    weight8<WHOLE>(a, k0, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * rstd * w[i];
    if (a.y) store8<false, WHOLE>(a.y, at + k0, a.H - k0, v[c]);
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
// with the sum's own gradient in 77.8 us (4.8 TB/s), the join 5.5; both together
// 4096 x 16384 118 us (4.6 TB/s).  Of more than 16384 columns a row is read twice, for
// a workgroup's 1024 threads have 128 registers each, and of these 28 to 53 still
// go to scratch memory: 4096 x 32768 bf16 300 us, 3.6 TB/s (fp32 510, 3.7).
template <bool F32, bool WHOLE, int LR, int C>
__global__ __launch_bounds__(norm_block(LR)) void norm_bwd_kernel(NormArgs a) {
  constexpr int ROWS = norm_block(LR) / LR;   // rows at a time
  constexpr bool LATE = C > 2;   // a row is read twice, chunk by chunk
  __shared__ double slots[LR < 64 ? 1 : LR / 64];
  __shared__ float add[ROWS == 1 ? 1 : C * LR * 8];
  const int lane = threadIdx.x & 63, all = threadIdx.x >> 6, wave = all % (LR < 64 ? 1 : LR / 64);
  const int l = threadIdx.x % LR;
  float dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  const int64_t groups = (a.T + ROWS - 1) / ROWS;
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t row = g * ROWS + threadIdx.x / LR;
    if (row >= a.T) break;   // all of a row's lanes, and with several waves none: no barrier is missed
    const int64_t at = row * a.H;
    Raw8<F32> x[C], ds[C];
    Raw8<false> dy[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = (c * LR + l) * 8;
      if (LATE) continue;
      x[c] = raw8<F32, WHOLE>(a.x, at + k0, a.H - k0);
      dy[c] = raw8<false, WHOLE>(a.dy, at + k0, a.H - k0);
    }
    if (a.residual && !LATE) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t k0 = (c * LR + l) * 8;
        ds[c] = raw8<F32, WHOLE>(a.residual, at + k0, a.H - k0);
      }
    }
    const float rstd = a.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = (c * LR + l) * 8;
      if (LATE) {
        x[c] = raw8<F32, WHOLE>(a.x, at + k0, a.H - k0);
        dy[c] = raw8<false, WHOLE>(a.dy, at + k0, a.H - k0);
      }
      float w[8];
      weight8<WHOLE>(a, k0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = value<false>(dy[c], i) * (value<F32>(x[c], i) * rstd);
        dw[c][i] += p;
        dot = fmaf(w[i], p, dot);
      }
      if (LATE) asm volatile("" : "+v"(dot)::"memory");   // no load is kept or moved ahead
    }
    dot = row_sum<LR>(dot, reinterpret_cast<float*>(slots), wave, lane) / (float)a.H;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k0 = (c * LR + l) * 8;
      float w[8], d[8];
      weight8<WHOLE>(a, k0, w);
      if (LATE) {
        x[c] = raw8<F32, WHOLE>(a.x, at + k0, a.H - k0);
        dy[c] = raw8<false, WHOLE>(a.dy, at + k0, a.H - k0);
        if (a.residual) ds[c] = raw8<F32, WHOLE>(a.residual, at + k0, a.H - k0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = rstd * (w[i] * value<false>(dy[c], i) - value<F32>(x[c], i) * rstd * dot);
        if (a.residual) d[i] += value<F32>(ds[c], i);
      }
      store8<F32, WHOLE>(a.sum, at + k0, a.H - k0, d);
      if (LATE) asm volatile("" : "+v"(dot)::"memory");
    }
  }
  if (ROWS > 1) {   // the rows of a wave, then the waves' sums, one wave after the other
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int d = LR; d < 64; d <<= 1) dw[c][i] += __shfl_xor(dw[c][i], d);
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
      if (all == u && lane < LR) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = &add[(c * 8 + i) * LR + l];
            dw[c][i] = u ? *p + dw[c][i] : dw[c][i];
            *p = dw[c][i];
          }
      }
      __syncthreads();
    }
    if (all != 3 || lane >= LR) return;   // the last wave has the sum
  }
  float* out = gridDim.x == 1 ? a.dw : a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k0 = (c * LR + l) * 8;
    store8<true, WHOLE>(out, k0, a.H - k0, dw[c]);
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

// Lanes of a row and chunks of 8 a lane, forward.  A wave a row, or a part of one,
// moves most bytes while rows fill the card; fewer rows of over 512, or longer
// ones, take more waves.
struct NormShape {
  int lr, c;
};
static NormShape norm_shape(int64_t T, int64_t H) {
  const int w = (int)((H + 511) / 512);   // chunks of one wave
  if (w == 1) return {H <= 128 ? 16 : H <= 256 ? 32 : 64, 1};
  if (w <= 6 && T >= 1024) return {64, w <= 2 ? 2 : w <= 4 ? 4 : 6};
  if (w <= 16) return {256, w <= 4 ? 1 : w <= 8 ? 2 : 4};
  return {1024, w <= 32 ? 2 : 4};
}
// Backward: a lane also holds the weight and its part of dw, so rows are split
// wider, to 16 waves on a CU (16384 x 2880: one wave a row, 4 on a CU, 138 us;
// four waves, 105 registers, 8 on a CU 109 us, 16 on a CU 84; twice as many
// workgroups and parts 91).
static NormShape norm_bwd_shape(int64_t H) {
  const int w = (int)((H + 511) / 512);
  if (w <= 2) return {H <= 128 ? 16 : H <= 256 ? 32 : 64, w};
  if (w <= 8) return {256, w <= 4 ? 1 : 2};
  if (w <= 16) return {512, 2};
  return {1024, w <= 32 ? 2 : 4};
}
int norm_threads(int64_t T, int64_t H) { return norm_block(norm_shape(T, H).lr); }
int64_t norm_blocks(int64_t T, int64_t H) {
  const int64_t rows = norm_threads(T, H) / norm_shape(T, H).lr;
  return (T + rows - 1) / rows;
}
// Workgroups: all that the card holds for many rows; a third as many as groups
// of rows, but one for each CU, while their parts of dw weigh as much as the rows
// (2880 columns, both launches, us: 700 rows, 256 workgroups 11.5, 700 14.0; 1024
// rows, the rule's 341 14.4, 256 13.3, 1024 16.2; 2047 rows, the rule's 682 20.2, 256
// 23.9, 1024 19.1).
static unsigned norm_bwd_grid(int64_t T, int64_t H) {
  const int lr = norm_bwd_shape(H).lr, block = norm_block(lr);
  const int64_t groups = (T + block / lr - 1) / (block / lr), most = 4 * 65536 / block;
  const int64_t third = groups / 3 < 256 ? 256 : groups / 3 < most ? groups / 3 : most;
  return (unsigned)(groups < third ? groups : third);
}

#define NORM_LAUNCH(kernel, grid, LR, C)                                                    \
  do {                                                                                      \
    const dim3 g_((unsigned)(grid)), b_(norm_block(LR));                                    \
    const bool whole_ = a.H % 8 == 0;                                                       \
    if (a.f32 && whole_) hipLaunchKernelGGL((kernel<true, true, LR, C>), g_, b_, 0, s, a);  \
    else if (a.f32) hipLaunchKernelGGL((kernel<true, false, LR, C>), g_, b_, 0, s, a);      \
    else if (whole_) hipLaunchKernelGGL((kernel<false, true, LR, C>), g_, b_, 0, s, a);     \
    else hipLaunchKernelGGL((kernel<false, false, LR, C>), g_, b_, 0, s, a);                \
    return hipGetLastError();                                                               \
  } while (0)

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const int64_t grid = norm_blocks(a.T, a.H);
  const NormShape n = norm_shape(a.T, a.H);
  switch (10 * n.lr + n.c) {
    case 161: NORM_LAUNCH(norm_kernel, grid, 16, 1);
    case 321: NORM_LAUNCH(norm_kernel, grid, 32, 1);
    case 641: NORM_LAUNCH(norm_kernel, grid, 64, 1);
    case 642: NORM_LAUNCH(norm_kernel, grid, 64, 2);
    case 644: NORM_LAUNCH(norm_kernel, grid, 64, 4);
    case 646: NORM_LAUNCH(norm_kernel, grid, 64, 6);
    case 2561: NORM_LAUNCH(norm_kernel, grid, 256, 1);
    case 2562: NORM_LAUNCH(norm_kernel, grid, 256, 2);
    case 2564: NORM_LAUNCH(norm_kernel, grid, 256, 4);
    case 10242: NORM_LAUNCH(norm_kernel, grid, 1024, 2);
    default: NORM_LAUNCH(norm_kernel, grid, 1024, 4);
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
  switch (10 * n.lr + n.c) {
    case 161: NORM_LAUNCH(norm_bwd_kernel, grid, 16, 1);
    case 321: NORM_LAUNCH(norm_bwd_kernel, grid, 32, 1);
    case 641: NORM_LAUNCH(norm_bwd_kernel, grid, 64, 1);
    case 642: NORM_LAUNCH(norm_bwd_kernel, grid, 64, 2);
    case 2561: NORM_LAUNCH(norm_bwd_kernel, grid, 256, 1);
    case 2562: NORM_LAUNCH(norm_bwd_kernel, grid, 256, 2);
    case 5122: NORM_LAUNCH(norm_bwd_kernel, grid, 512, 2);
    case 10242: NORM_LAUNCH(norm_bwd_kernel, grid, 1024, 2);
    default: NORM_LAUNCH(norm_bwd_kernel, grid, 1024, 4);
  }
}

hipError_t launch_norm_join(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((a.H + 63) / 64)), dim3(1024), 0, s, a.part, a.H,
                     (int)norm_bwd_grid(a.T, a.H), a.dw);
  return hipGetLastError();
}

}  // namespace mxmoe
