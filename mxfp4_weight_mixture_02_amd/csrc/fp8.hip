// Dense products in 8-bit floating point with one scale for each block of
// 128 (gfx950): quantizers, the transposition of weights, the product on the
// scaled matrix cores, and its forms for few rows.
//
// Elements are OCP E4M3, scales UE8M0 (powers of two, 2^(s - 127)): the
// scaled MFMA of gfx950 applies them to the operands in the matrix core, so
// the accumulators need no multiplication between K blocks.  A power of two
// moves only the exponent of an element, so against an arbitrary fp32 scale
// nothing of the three mantissa bits is lost (only up to one binade of the
// subnormal end of the range).
//
// Storage: codes [rows, K rounded up to 128] with zeros in the padding, so
// no kernel has a K tail; scales K block by K block, so that the rows of a
// tile have theirs side by side.
#include "common.hpp"
#include "fp8.hpp"

namespace mxmoe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- quantizers

// Eight consecutive elements of a row, zeros from `limit` on.  VEC: the row
// and K allow 16-byte loads of whole groups.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t at, int64_t left, float (&v)[8]) {
  if (VEC) {
    if (left <= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      return;
    }
    if (F32) {
      const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + at);
      const f32x4 a = p[0], b = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[i + 4] = b[i];
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (i < left)
        v[i] = F32 ? static_cast<const float*>(x)[at + i]
                   : bf16_to_f32(static_cast<const uint16_t*>(x)[at + i]);
    }
  }
}

// One K block of 16 rows per workgroup: 16 lanes per row, 8 elements each
// (128 contiguous code bytes a row; the 16 rows' scales side by side).
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const void* __restrict__ x, int64_t rows,
                                                       int64_t K, int64_t pitch, int64_t spitch,
                                                       int kblocks, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
  const int kb = blockIdx.x % kblocks;
  const int64_t row = (int64_t)(blockIdx.x / kblocks) * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  const int64_t k0 = (int64_t)kb * 128 + 8 * l;
  float v[8];
  load8<F32, VEC>(x, row * K + k0, row < rows ? K - k0 : 0, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[i]));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  const int e = e4m3_exponent(m);
  const float f = e4m3_inverse(e);
  if (row >= rows) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = nan_unless_finite(v[i]) * f;
  *reinterpret_cast<u32x2*>(codes + row * pitch + k0) =
      u32x2{e4m3_pack4(v[0], v[1], v[2], v[3]), e4m3_pack4(v[4], v[5], v[6], v[7])};
  if (l == 0) scales[(int64_t)kb * spitch + row] = (uint8_t)(e + 127);
}

// Blocks of 128 rows of one column, written as rows of the transpose: a
// workgroup takes 128 rows x 64 columns through LDS (fp32, one column a
// row of 129 words), then 4 threads a column, 32 rows each.
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void fp8_cols_kernel(const void* __restrict__ x, int64_t rows,
                                                       int64_t K, int64_t pitch, int64_t spitch,
                                                       int ctiles, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
  __shared__ float t[64][129];
  const int tid = threadIdx.x;
  const int64_t rb = blockIdx.x / ctiles, c0 = (int64_t)(blockIdx.x % ctiles) * 64;
  const int64_t r0 = rb * 128;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = 32 * p + (tid >> 3), c = 8 * (tid & 7);
    float v[8];
    load8<F32, VEC>(x, (r0 + r) * K + c0 + c, r0 + r < rows ? K - c0 - c : 0, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[c + i][r] = v[i];
  }
  __syncthreads();
  const int c = tid >> 2, q = tid & 3;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, finite_bits(t[c][32 * q + i]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  const int e = e4m3_exponent(m);
  const float f = e4m3_inverse(e);
  if (c0 + c >= K) return;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float* s = &t[c][32 * q + 4 * i];
    w[i] = e4m3_pack4(nan_unless_finite(s[0]) * f, nan_unless_finite(s[1]) * f,
                     nan_unless_finite(s[2]) * f, nan_unless_finite(s[3]) * f);
  }
  u32x4* d = reinterpret_cast<u32x4*>(codes + (c0 + c) * pitch + r0 + 32 * q);
  d[0] = u32x4{w[0], w[1], w[2], w[3]};
  d[1] = u32x4{w[4], w[5], w[6], w[7]};
  if (q == 0) scales[rb * spitch + c0 + c] = (uint8_t)(e + 127);
}

// One 128 x 128 block per workgroup; 16 lanes a row, 8 rows a thread.
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void fp8_blocks_kernel(const void* __restrict__ x, int64_t rows,
                                                         int64_t K, int64_t pitch, int kblocks,
                                                         int64_t rblocks,
                                                         uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  __shared__ uint32_t top[4];
  const int tid = threadIdx.x;
  const int kb = blockIdx.x % kblocks;
  const int64_t rb = blockIdx.x / kblocks;
  const int64_t k0 = (int64_t)kb * 128 + 8 * (tid & 15), r0 = rb * 128 + (tid >> 4);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t r = r0 + 16 * p;
    load8<F32, VEC>(x, r * K + k0, r < rows ? K - k0 : 0, v[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[p][i]));
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((tid & 63) == 0) top[tid >> 6] = m;
  __syncthreads();
  m = max(max(top[0], top[1]), max(top[2], top[3]));
  const int e = e4m3_exponent(m);
  const float f = e4m3_inverse(e);
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t r = r0 + 16 * p;
    if (r < rows) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = nan_unless_finite(v[p][i]) * f;
      *reinterpret_cast<u32x2*>(codes + r * pitch + k0) =
          u32x2{e4m3_pack4(y[0], y[1], y[2], y[3]), e4m3_pack4(y[4], y[5], y[6], y[7])};
    }
  }
  if (tid == 0) scales[(int64_t)kb * rblocks + rb] = (uint8_t)(e + 127);
}

// One 128 x 128 block of codes per workgroup, bytes through LDS; the
// padding columns of the transpose (rows past the matrix) are zeros.
__global__ __launch_bounds__(256) void fp8_transpose_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int64_t K,
    int64_t pitch, int64_t pitch_t, int kblocks, int64_t rblocks, uint8_t* __restrict__ codes_t,
    uint8_t* __restrict__ scales_t) {
  __shared__ uint8_t t[128][132];
  const int tid = threadIdx.x;
  const int kb = blockIdx.x % kblocks;
  const int64_t rb = blockIdx.x / kblocks;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = 32 * p + (tid >> 3), c = 16 * (tid & 7);
    const int64_t row = rb * 128 + r;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (row < rows) v = *reinterpret_cast<const u32x4*>(codes + row * pitch + (int64_t)kb * 128 + c);
#pragma unroll
    for (int i = 0; i < 16; ++i) t[c + i][r] = (uint8_t)(v[i >> 2] >> (8 * (i & 3)));
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = 32 * p + (tid >> 3), c = 16 * (tid & 7);
    const int64_t row = (int64_t)kb * 128 + r;
    if (row < K) {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(&t[r][c + 4 * i]);
      *reinterpret_cast<u32x4*>(codes_t + row * pitch_t + rb * 128 + c) = v;
    }
  }
  if (tid == 0) scales_t[rb * kblocks + kb] = scales[(int64_t)kb * rblocks + rb];
}

// ------------------------------------------------------------------- products

// out[m][n] = sum_k X[m][k] W[n][k].  W is the MFMA's A operand (D rows n)
// and X the B operand (D columns m), in v_mfma_scale_f32_16x16x128_f8f6f4:
// one instruction spans a whole 128-element scale block, so a lane's scale
// byte is its row's (lane l feeds row l % 16 and, since both operands hold
// 8-bit elements in the same layout, any 32 bytes of the row as long as W
// and X take the same ones).
//
// Row mapping.  A wave's W rows are its F_N fragments interleaved: fragment
// i, MFMA row r is row pi(r) * F_N + i with pi(4 q + v) = 4 v + q; so the
// values that lane q holds in accumulator register v, over the fragments,
// are consecutive n (one wide store), and the four lanes q side by side
// fill 64-byte pieces.  X: fragment j, column c is row c * F_M + j, so a
// lane's F_M scale bytes are one load, picked by op_sel.
__device__ __forceinline__ int fp8_pi(int r) { return 4 * (r & 3) + (r >> 2); }

template <int SEL_A, int SEL_B>
__device__ __forceinline__ f32x4 fp8_mfma(const i32x8& a, const i32x8& b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, SEL_A, sa, SEL_B, sb);
}
__device__ __forceinline__ f32x4 fp8_mfma(const i32x8& a, const i32x8& b, f32x4 c, int sel_a,
                                          int sa, int sel_b, int sb) {
  // the selectors are constants after unrolling
  switch (sel_a * 4 + sel_b) {
    case 0: return fp8_mfma<0, 0>(a, b, c, sa, sb);
    case 1: return fp8_mfma<0, 1>(a, b, c, sa, sb);
    case 2: return fp8_mfma<0, 2>(a, b, c, sa, sb);
    case 3: return fp8_mfma<0, 3>(a, b, c, sa, sb);
    case 4: return fp8_mfma<1, 0>(a, b, c, sa, sb);
    case 5: return fp8_mfma<1, 1>(a, b, c, sa, sb);
    case 6: return fp8_mfma<1, 2>(a, b, c, sa, sb);
    case 7: return fp8_mfma<1, 3>(a, b, c, sa, sb);
    case 8: return fp8_mfma<2, 0>(a, b, c, sa, sb);
    case 9: return fp8_mfma<2, 1>(a, b, c, sa, sb);
    case 10: return fp8_mfma<2, 2>(a, b, c, sa, sb);
    case 11: return fp8_mfma<2, 3>(a, b, c, sa, sb);
    case 12: return fp8_mfma<3, 0>(a, b, c, sa, sb);
    case 13: return fp8_mfma<3, 1>(a, b, c, sa, sb);
    case 14: return fp8_mfma<3, 2>(a, b, c, sa, sb);
    default: return fp8_mfma<3, 3>(a, b, c, sa, sb);
  }
}

// fp32 results.  Inside one instruction the scaled matrix core drops what
// lies below 2^-13 of its largest product (measured: 2^16 + 2^2 gives 2^16),
// 1.5e-5 of a result over random values: far below the rounding of a bf16
// result (1.6e-3), far above that of an fp32 one.  So fp32 results take the
// bf16 matrix core, whose products and sums are fp32: an E4M3 code times its
// scale is a bf16 (from 2^-126 on), converted in registers, 16 values to a
// lane's 16 bytes, in four instructions of 32 elements.
__device__ __forceinline__ void fp8_to_bf16(const i32x8& c, uint32_t scale, bf16x8 (&v)[4]) {
  const float f = scale_operand(scale);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    u32x4 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t x = (uint32_t)c[2 * s + h];
      w[2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, f, false));
      w[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, f, true));
    }
    v[s] = as_bf16x8(w);
  }
}
__device__ __forceinline__ uint32_t byte_of(uint32_t w, int i) { return (w >> (8 * i)) & 0xFFu; }

// F consecutive outputs out[m][n ..], plus the bias; whole vectors where
// the row allows it.
template <int F, bool F32>
__device__ __forceinline__ void fp8_store(const Fp8Gemm& g, int64_t m, int64_t n, float (&v)[F],
                                          bool wide) {
  if (m >= g.M || n >= g.N) return;
  if (g.bias) {
#pragma unroll
    for (int i = 0; i < F; ++i)
      if (n + i < g.N) v[i] += bf16_to_f32(g.bias[n + i]);
  }
  const int64_t at = m * g.N + n;
  if (wide) {   // N % F == 0: the F values exist and are aligned
    if (F32) {
      f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at);
#pragma unroll
      for (int i = 0; i < F / 4; ++i) d[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    } else {
      u32x2* d = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.out) + at);
      if (F == 8)
        *reinterpret_cast<u32x4*>(d) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                             pack_bf16x2(v[F - 4], v[F - 3]), pack_bf16x2(v[F - 2], v[F - 1])};
      else
        d[0] = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < F; ++i)
    if (n + i < g.N) {
      if (F32)
        static_cast<float*>(g.out)[at + i] = v[i];
      else
        static_cast<uint16_t*>(g.out)[at + i] = (uint16_t)f32_to_bf16(v[i]);
    }
}

constexpr int FP8_RSRC_W3 = 0x00020000;   // raw buffer, untyped

template <int WN_, int WM_, int FN_, int FM_>
struct Fp8Tile {
  static constexpr int WN = WN_, WM = WM_, FN = FN_, FM = FM_;
  static constexpr int NW = WN * WM;          // waves
  static constexpr int BN = WN * FN * 16, BM = WM * FM * 16;
  static constexpr int STAGE = (BN + BM) * 128;
  static constexpr int LOADS = (BN + BM) / 8 / NW;   // 1 KB copies per wave and step
  static_assert(LOADS <= 8 && LOADS * NW * 8 == BN + BM, "Fp8Wave::off");
};

// A wave's part of a tile's main loop.
struct Fp8Wave {
  __amdgpu_buffer_rsrc_t rw, rx;
  uint32_t off[8];             // this lane's 16 bytes of each copy, at K block 0
  const uint8_t *sx, *sw;      // this lane's scale bytes, at K block 0
  int64_t sxp, swp;            // and their step from K block to K block
  int wave, woff, xoff, s0;    // fragment addresses in a stage: row, first chunk
};

// Copies of K block kb into a stage: this wave's 1 KB pieces; piece p is
// rows 8 p .. 8 p + 7 of the W tile, then of the X tile.
template <class T>
__device__ __forceinline__ void fp8_copy(const Fp8Wave& g, uint8_t* __restrict__ st, int kb) {
#pragma unroll
  for (int i = 0; i < T::LOADS; ++i) {
    const int p = g.wave * T::LOADS + i;
    if (p < T::BN / 8)   // uniform
      __builtin_amdgcn_raw_ptr_buffer_load_lds(g.rw, (lptr_t)(st + p * 1024), 16, g.off[i], kb * 128, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(g.rx, (lptr_t)(st + p * 1024), 16, g.off[i], kb * 128, 0, 0);
  }
}

struct Fp8Scales {
  uint32_t x[2], w[2];
};

template <class T, bool WROWS>
__device__ __forceinline__ void fp8_scales(const Fp8Wave& g, int kb, Fp8Scales& s) {
#pragma unroll
  for (int i = 0; i < T::FM / 4; ++i) s.x[i] = *reinterpret_cast<const uint32_t*>(g.sx + kb * g.sxp + 4 * i);
  if (WROWS) {
#pragma unroll
    for (int i = 0; i < T::FN / 4; ++i) s.w[i] = *reinterpret_cast<const uint32_t*>(g.sw + kb * g.swp + 4 * i);
  } else {
    s.w[0] = g.sw[kb * g.swp];
  }
}

__device__ __forceinline__ i32x8 fp8_frag(const uint8_t* p, int s0) {
  const u32x4 lo = *reinterpret_cast<const u32x4*>(p + s0);
  const u32x4 hi = *reinterpret_cast<const u32x4*>(p + (s0 ^ 16));
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// One K block: wait for this wave's copies of it, meet the other waves
// (which also ends their reads of the other stage), start the next block's
// copies there, multiply.  cur and nxt do not overlap: the compiler need
// not wait for the copies before it reads cur.
template <class T, bool WROWS, bool F32>
__device__ __forceinline__ void fp8_step(const Fp8Wave& g, const uint8_t* __restrict__ cur,
                                         uint8_t* __restrict__ nxt, int kb, int kblocks,
                                         Fp8Scales& sc, f32x4 (&acc)[T::FN][T::FM]) {
  constexpr int FN = T::FN, FM = T::FM;
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
  barrier_only();
  const Fp8Scales c = sc;
  if (kb + 1 < kblocks) {
    fp8_copy<T>(g, nxt, kb + 1);
    fp8_scales<T, WROWS>(g, kb + 1, sc);
  }
  if (F32) {
    bf16x8 b[FM][4];
#pragma unroll
    for (int j = 0; j < FM; ++j)
      fp8_to_bf16(fp8_frag(cur + g.xoff + j * 128, g.s0), byte_of(c.x[j >> 2], j & 3), b[j]);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      bf16x8 a[4];
      fp8_to_bf16(fp8_frag(cur + g.woff + i * 128, g.s0), WROWS ? byte_of(c.w[i >> 2], i & 3) : c.w[0], a);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < FM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s], b[j][s], acc[i][j], 0, 0, 0);
    }
    return;
  }
  i32x8 b[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) b[j] = fp8_frag(cur + g.xoff + j * 128, g.s0);
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const i32x8 a = fp8_frag(cur + g.woff + i * 128, g.s0);
#pragma unroll
    for (int j = 0; j < FM; ++j)
      acc[i][j] = fp8_mfma(a, b[j], acc[i][j], WROWS ? i & 3 : 0, (int)c.w[WROWS ? i >> 2 : 0], j & 3,
                           (int)c.x[j >> 2]);
  }
}

// One BN x BM tile per workgroup, WN x WM waves of (16 FN) x (16 FM); K in
// steps of one scale block (128), two LDS stages.  LDS rows are 128 bytes in
// 16-byte chunks; chunk c of a row whose fragment row is r sits at slot c ^
// (r % 8), so 8 consecutive lanes' reads cover all banks.
template <int WN, int WM, int FN, int FM, bool WROWS, bool F32>
__global__ __launch_bounds__(64 * WN * WM) void fp8_gemm_kernel(Fp8Gemm g, int ntiles, int mtiles) {
  using T = Fp8Tile<WN, WM, FN, FM>;
  __shared__ __align__(1024) uint8_t lds[2 * T::STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  Fp8Wave v;
  v.wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // tile of this block: XCD x takes a contiguous range of the order in which
  // bands of 8 m-tiles run through all n-tiles, m fastest
  int nt, mt;
  {
    const int L = ntiles * mtiles, b = blockIdx.x;
    const int x = b & 7, base = L >> 3, extra = L & 7;
    const int item = x * base + min(x, extra) + (b >> 3);
    const int band = item / (8 * ntiles), rows = min(8, mtiles - 8 * band);
    const int local = item - band * 8 * ntiles;
    mt = band * 8 + local % rows;
    nt = local / rows;
  }
  const int64_t n0 = (int64_t)nt * T::BN, m0 = (int64_t)mt * T::BM;
  const int64_t pitch = fp8_pitch(g.K);
  const int kblocks = (int)(pitch / 128);
  // copies: lane l brings slot l % 8 of row l / 8 of a piece.  Rows past the
  // matrix repeat its last row (their results are dropped).
  const int nrows = (int)min((int64_t)T::BN, g.N - n0), mrows = (int)min((int64_t)T::BM, g.M - m0);
  v.rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.w + n0 * pitch), (short)0,
                                           (int)(nrows * pitch), FP8_RSRC_W3);
  v.rx = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.x + m0 * pitch), (short)0,
                                           (int)(mrows * pitch), FP8_RSRC_W3);
#pragma unroll
  for (int i = 0; i < T::LOADS; ++i) {
    const int p = v.wave * T::LOADS + i;
    const bool isw = p < T::BN / 8;
    const int row = 8 * (isw ? p : p - T::BN / 8) + (lane >> 3);
    const int fr = isw ? fp8_pi((row % (16 * FN)) / FN) : (row % (16 * FM)) / FM;
    v.off[i] = (uint32_t)min(row, (isw ? nrows : mrows) - 1) * (uint32_t)pitch +
               (((lane & 7) ^ (fr & 7)) << 4);
  }
  const int wn = v.wave / WM, wm = v.wave % WM;
  const int r = lane & 15, q = lane >> 4;
  // scales: X's FM bytes of this lane's rows; W's one byte of the wave's
  // 128-row block, or its FN rows' bytes
  const int64_t nw0 = n0 + wn * 16 * FN;
  v.sxp = fp8_scale_pitch(g.M);
  v.sx = g.sx + min(m0 + wm * 16 * FM + r * FM, v.sxp - FM);
  v.swp = WROWS ? fp8_scale_pitch(g.N) : (g.N + 127) / 128;
  v.sw = g.sw + (WROWS ? min(nw0 + fp8_pi(r) * FN, v.swp - FN) : min(nw0 / 128, v.swp - 1));
  v.woff = (wn * 16 * FN + fp8_pi(r) * FN) * 128;
  v.xoff = T::BN * 128 + (wm * 16 * FM + r * FM) * 128;
  v.s0 = ((2 * q) ^ (r & 7)) << 4;
  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  Fp8Scales sc;
  fp8_copy<T>(v, lds, 0);
  fp8_scales<T, WROWS>(v, 0, sc);
  for (int kb = 0; kb < kblocks; kb += 2) {
    fp8_step<T, WROWS, F32>(v, lds, lds + T::STAGE, kb, kblocks, sc, acc);
    if (kb + 1 < kblocks) fp8_step<T, WROWS, F32>(v, lds + T::STAGE, lds, kb + 1, kblocks, sc, acc);
  }
  const bool wide = g.N % FN == 0;
#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float o[FN];
#pragma unroll
      for (int i = 0; i < FN; ++i) o[i] = acc[i][j][t];
      fp8_store<FN, F32>(g, m0 + wm * 16 * FM + r * FM + j, nw0 + (4 * t + q) * FN, o, wide);
    }
}

// Few rows: a workgroup takes 16 rows of W and its NW waves split the K
// blocks; every wave streams its part of W straight into fragments (a lane
// 32 bytes of its row, a wave 16 whole 128-byte lines) and the partial sums
// meet in LDS in wave order.  FUSED: X comes as bf16 and is rounded to E4M3
// in the lane that feeds it to the matrix core: the lane's 32 elements, the
// block's largest magnitude from the four lanes that share the row.
constexpr int SK_NW = 8, SK_CH = 4;   // waves; K blocks in flight per wave

template <int FM, bool WROWS, bool F32, bool FUSED, bool VEC>
__global__ __launch_bounds__(64 * SK_NW) void fp8_skinny_kernel(Fp8Gemm g, const uint16_t* __restrict__ xb) {
  __shared__ f32x4 part[SK_NW][FM][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t pitch = fp8_pitch(g.K);
  const int kblocks = (int)(pitch / 128);
  const int b0 = wave * kblocks / SK_NW, b1 = (wave + 1) * kblocks / SK_NW;
  const int64_t n = min(n0 + r, g.N - 1);
  const uint8_t* w = g.w + n * pitch + 32 * q;
  const int64_t sxp = fp8_scale_pitch(g.M);
  const int64_t swp = WROWS ? fp8_scale_pitch(g.N) : (g.N + 127) / 128;
  const uint8_t* sw = g.sw + (WROWS ? n : n / 128);
  f32x4 acc[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = b0; c0 < b1; c0 += SK_CH) {
    u32x4 lo[SK_CH], hi[SK_CH];
    uint32_t s[SK_CH];
#pragma unroll
    for (int u = 0; u < SK_CH; ++u) {
      const int64_t kb = min(c0 + u, b1 - 1);
      lo[u] = gload16(w + kb * 128);
      hi[u] = gload16(w + kb * 128 + 16);
      s[u] = sw[kb * swp];
    }
#pragma unroll
    for (int u = 0; u < SK_CH; ++u) {
      if (c0 + u >= b1) break;
      const int64_t kb = c0 + u;
      const i32x8 a = {(int)lo[u][0], (int)lo[u][1], (int)lo[u][2], (int)lo[u][3],
                       (int)hi[u][0], (int)hi[u][1], (int)hi[u][2], (int)hi[u][3]};
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const int64_t m = min((int64_t)(16 * j + r), g.M - 1);
        i32x8 b;
        uint32_t sb;
        if (FUSED) {
          const int64_t k0 = kb * 128 + 32 * q;
          float v[4][8];
          uint32_t top = 0;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            load8<false, VEC>(xb, m * g.K + k0 + 8 * p, g.K - k0 - 8 * p, v[p]);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, finite_bits(v[p][i]));
          }
          top = max(top, (uint32_t)__shfl_xor((int)top, 16));
          top = max(top, (uint32_t)__shfl_xor((int)top, 32));
          const int e = e4m3_exponent(top);
          const float f = e4m3_inverse(e);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] = nan_unless_finite(v[p][i]) * f;
            b[2 * p] = (int)e4m3_pack4(v[p][0], v[p][1], v[p][2], v[p][3]);
            b[2 * p + 1] = (int)e4m3_pack4(v[p][4], v[p][5], v[p][6], v[p][7]);
          }
          sb = (uint32_t)(e + 127);
        } else {
          const u32x4 xl = gload16(g.x + m * pitch + kb * 128 + 32 * q);
          const u32x4 xh = gload16(g.x + m * pitch + kb * 128 + 32 * q + 16);
          b = i32x8{(int)xl[0], (int)xl[1], (int)xl[2], (int)xl[3], (int)xh[0], (int)xh[1], (int)xh[2], (int)xh[3]};
          sb = g.sx[kb * sxp + m];
        }
        if (F32) {
          bf16x8 av[4], bv[4];
          fp8_to_bf16(a, s[u], av);
          fp8_to_bf16(b, sb, bv);
#pragma unroll
          for (int t = 0; t < 4; ++t)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[t], bv[t], acc[j], 0, 0, 0);
        } else {
          acc[j] = fp8_mfma<0, 0>(a, b, acc[j], (int)s[u], (int)sb);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < FM; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  // lane l holds D rows 4 (l / 16) .. + 3 (n) of column l % 16 (m)
  const bool wide = g.N % 4 == 0;
  for (int j = wave; j < FM; j += SK_NW) {
    f32x4 sum = part[0][j][lane];
#pragma unroll
    for (int u = 1; u < SK_NW; ++u) sum += part[u][j][lane];
    float o[4] = {sum[0], sum[1], sum[2], sum[3]};
    fp8_store<4, F32>(g, 16 * j + r, n0 + 4 * q, o, wide);
  }
}

// ------------------------------------------------------------------ launchers

#define FP8_QUANT(kernel, grid, ...)                                                             \
  do {                                                                                           \
    const bool vec = K % 8 == 0 && (reinterpret_cast<uintptr_t>(x) % 16) == 0;                    \
    if (x_f32) {                                                                                  \
      if (vec)                                                                                    \
        hipLaunchKernelGGL((kernel<true, true>), dim3((unsigned)(grid)), dim3(256), 0, s, __VA_ARGS__);  \
      else                                                                                        \
        hipLaunchKernelGGL((kernel<true, false>), dim3((unsigned)(grid)), dim3(256), 0, s, __VA_ARGS__); \
    } else {                                                                                      \
      if (vec)                                                                                    \
        hipLaunchKernelGGL((kernel<false, true>), dim3((unsigned)(grid)), dim3(256), 0, s, __VA_ARGS__); \
      else                                                                                        \
        hipLaunchKernelGGL((kernel<false, false>), dim3((unsigned)(grid)), dim3(256), 0, s, __VA_ARGS__); \
    }                                                                                             \
    return hipGetLastError();                                                                     \
  } while (0)

hipError_t launch_fp8_quantize_rows(const void* x, int x_f32, int64_t rows, int64_t K,
                                    uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t kb = fp8_pitch(K) / 128;
  FP8_QUANT(fp8_rows_kernel, kb * ((rows + 15) / 16), x, rows, K, fp8_pitch(K),
            fp8_scale_pitch(rows), (int)kb, codes, scales);
}

hipError_t launch_fp8_quantize_cols(const void* x, int x_f32, int64_t rows, int64_t K,
                                    uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t ct = (K + 63) / 64;
  FP8_QUANT(fp8_cols_kernel, ct * ((rows + 127) / 128), x, rows, K, fp8_pitch(rows),
            fp8_scale_pitch(K), (int)ct, codes, scales);
}

hipError_t launch_fp8_quantize_blocks(const void* x, int x_f32, int64_t rows, int64_t K,
                                      uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t kb = fp8_pitch(K) / 128, rb = (rows + 127) / 128;
  FP8_QUANT(fp8_blocks_kernel, kb * rb, x, rows, K, fp8_pitch(K), (int)kb, rb, codes, scales);
}

hipError_t launch_fp8_transpose(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t K, uint8_t* codes_t, uint8_t* scales_t, hipStream_t s) {
  const int64_t kb = fp8_pitch(K) / 128, rb = (rows + 127) / 128;
  hipLaunchKernelGGL(fp8_transpose_kernel, dim3((unsigned)(kb * rb)), dim3(256), 0, s, codes, scales,
                     rows, K, fp8_pitch(K), fp8_pitch(rows), (int)kb, rb, codes_t, scales_t);
  return hipGetLastError();
}

template <int WN, int WM, int FN, int FM>
static hipError_t gemm_tile(const Fp8Gemm& g, hipStream_t s) {
  using T = Fp8Tile<WN, WM, FN, FM>;
  const int64_t nt = (g.N + T::BN - 1) / T::BN, mt = (g.M + T::BM - 1) / T::BM;
  const dim3 grid((unsigned)(nt * mt)), block(64 * T::NW);
  if (g.w_rows) {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_gemm_kernel<WN, WM, FN, FM, true, true>), grid, block, 0, s, g, (int)nt, (int)mt);
    else
      hipLaunchKernelGGL((fp8_gemm_kernel<WN, WM, FN, FM, true, false>), grid, block, 0, s, g, (int)nt, (int)mt);
  } else {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_gemm_kernel<WN, WM, FN, FM, false, true>), grid, block, 0, s, g, (int)nt, (int)mt);
    else
      hipLaunchKernelGGL((fp8_gemm_kernel<WN, WM, FN, FM, false, false>), grid, block, 0, s, g, (int)nt, (int)mt);
  }
  return hipGetLastError();
}

template <int FM>
static hipError_t skinny(const Fp8Gemm& g, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * SK_NW);
  const uint16_t* none = nullptr;
  if (g.w_rows) {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_skinny_kernel<FM, true, true, false, true>), grid, block, 0, s, g, none);
    else
      hipLaunchKernelGGL((fp8_skinny_kernel<FM, true, false, false, true>), grid, block, 0, s, g, none);
  } else {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_skinny_kernel<FM, false, true, false, true>), grid, block, 0, s, g, none);
    else
      hipLaunchKernelGGL((fp8_skinny_kernel<FM, false, false, false, true>), grid, block, 0, s, g, none);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t s) {
  if (g.M <= 16) return skinny<1>(g, s);
  if (g.M <= 32) return skinny<2>(g, s);
  if (g.M <= 64) return skinny<4>(g, s);
  // 256 x 256 tiles once they fill the 256 CUs, else 128 x 128
  const int64_t big = ((g.N + 255) / 256) * ((g.M + 255) / 256);
  if (big >= 256) return gemm_tile<2, 4, 8, 4>(g, s);
  return gemm_tile<2, 2, 4, 4>(g, s);
}

bool fp8_fused_fits(int64_t M, int64_t K) { return M <= 16; }

hipError_t launch_fp8_fused(const Fp8Gemm& g, const uint16_t* x, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * SK_NW);
  const bool vec = g.K % 8 == 0 && (reinterpret_cast<uintptr_t>(x) % 16) == 0;
  if (g.out_f32) {
    if (vec)
      hipLaunchKernelGGL((fp8_skinny_kernel<1, false, true, true, true>), grid, block, 0, s, g, x);
    else
      hipLaunchKernelGGL((fp8_skinny_kernel<1, false, true, true, false>), grid, block, 0, s, g, x);
  } else {
    if (vec)
      hipLaunchKernelGGL((fp8_skinny_kernel<1, false, false, true, true>), grid, block, 0, s, g, x);
    else
      hipLaunchKernelGGL((fp8_skinny_kernel<1, false, false, true, false>), grid, block, 0, s, g, x);
  }
  return hipGetLastError();
}

}  // namespace mxmoe
