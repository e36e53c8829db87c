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
// (128 contiguous code bytes a row; the 16 rows' scales side by side).  Bound
// by HBM: 16384 x 2880 bf16 in 31.1 us, 4.6 TB/s.
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
// row of 129 words), then 4 threads a column, 32 rows each.  Bound by HBM:
// 16384 x 2880 bf16 in 27.9 us, 5.1 TB/s.
template <bool F32, bool VEC>
__device__ __forceinline__ void fp8_cols(const void* __restrict__ x, int64_t rows, int64_t K, int64_t pitch,
                                         int64_t spitch, int ctiles, uint8_t* __restrict__ codes,
                                         uint8_t* __restrict__ scales, unsigned block, float (*t)[129]) {
  const int tid = threadIdx.x;
  const int64_t rb = block / ctiles, c0 = (int64_t)(block % ctiles) * 64;
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
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void fp8_cols_kernel(const void* __restrict__ x, int64_t rows,
                                                       int64_t K, int64_t pitch, int64_t spitch,
                                                       int ctiles, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
  __shared__ float t[64][129];
  fp8_cols<F32, VEC>(x, rows, K, pitch, spitch, ctiles, codes, scales, blockIdx.x, t);
}
// Two bf16 matrices of the same rows in one launch: the first `blocks`
// workgroups have a.  A launch of its own is 3 us more of a whole dW (5760 x
// 2880 x 4093: 161 us, 158).
struct Fp8Cols {
  const void* x;
  int64_t K, spitch;
  uint8_t *codes, *scales;
  int ctiles, vec;
};
__global__ __launch_bounds__(256) void fp8_cols_pair_kernel(Fp8Cols a, Fp8Cols b, int64_t rows, int64_t pitch,
                                                            unsigned blocks) {
  __shared__ float t[64][129];
  const bool first = blockIdx.x < blocks;
  const Fp8Cols m = first ? a : b;
  const unsigned block = blockIdx.x - (first ? 0 : blocks);
  if (m.vec)
    fp8_cols<false, true>(m.x, rows, m.K, pitch, m.spitch, m.ctiles, m.codes, m.scales, block, t);
  else
    fp8_cols<false, false>(m.x, rows, m.K, pitch, m.spitch, m.ctiles, m.codes, m.scales, block, t);
}

// One 128 x 128 block per workgroup; 16 lanes a row, 8 rows a thread.  Bound
// by HBM: 46080 x 2880 bf16 in 91 us, 4.4 TB/s.
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
// padding columns of the transpose (rows past the matrix) are zeros.  Bound by
// HBM: 46080 x 2880 in 44.3 us, 6.0 TB/s.
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
    if constexpr (F == 2) {
      if (F32)
        *reinterpret_cast<f32x2*>(static_cast<float*>(g.out) + at) = f32x2{v[0], v[1]};
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(g.out) + at) = pack_bf16x2(v[0], v[1]);
    } else if constexpr (F32) {
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

// A workgroup's tile: WN x WM waves of (16 FN) x (16 FM), and NST LDS stages.
// A stage holds one K block: BN rows of W and BM rows of X (128 bytes each),
// X's BM scale bytes (room for 256) and W's scales (256 bytes).
template <int WN_, int WM_, int FN_, int FM_, int NST_>
struct Fp8Tile {
  static constexpr int WN = WN_, WM = WM_, FN = FN_, FM = FM_, NST = NST_;
  static constexpr int NW = WN * WM;          // waves
  static constexpr int BN = WN * FN * 16, BM = WM * FM * 16;
  static constexpr int SX = (BN + BM) * 128, SW = SX + 256, STAGE = SW + 256;
  static constexpr int LOADS = (BN + BM) / 8 / NW;   // 1 KB copies per wave and step
  static_assert(LOADS <= 8 && LOADS * NW * 8 == BN + BM && NW % 2 == 0, "copies");
  static_assert(BN <= 256 && BM <= 256 && NST >= 2 && NST * STAGE <= 160 * 1024, "LDS");
  static_assert((NST - 1) * (LOADS + 1) < 64, "vector-memory counter");
  static constexpr bool SPREAD = 2 * NST * STAGE > 160 * 1024;   // one workgroup on a CU
  // scale bytes of X and W are read four at a time, or with F % 4 one by one
  static constexpr int XW = FM % 4 ? FM : FM / 4, WW = FN % 4 ? FN : FN / 4;
};

// Copy from global memory to LDS: 16, 4 or 1 bytes a lane from base + off +
// soff to LDS address lds + (16, 4, 4) * lane.  As assembly, because the
// compiler makes every later LDS read wait for every such copy in flight
// that it cannot prove to go elsewhere, and with a ring of stages it can
// prove nothing.  The kernel waits itself (fp8_wait) before it reads a
// stage.  A copy has no output register; its address is read at issue.  m0
// is a reserved register, which the compiler writes right before each use of
// its own: the clobber keeps such a pair on one side of a copy (none of these
// kernels has one), and its warning says only that m0 is not saved.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void lds_copy(u32x4 rsrc, uint32_t lds, uint32_t off, uint32_t soff) {
  if (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0", "memory");
  else if (BYTES == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0", "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0", "memory");
}
#pragma clang diagnostic pop
// Raw buffer of `bytes` bytes at p (a wave-uniform pointer).
__device__ __forceinline__ u32x4 buffer_of(const uint8_t* p, int64_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), (uint32_t)FP8_RSRC_W3};
}

// A wave's part of a tile's main loop.
struct Fp8Wave {
  u32x4 rw, rx, rs;            // W's and X's rows of the tile, and this wave's scales
  uint32_t off[8];             // this lane's 16 bytes of each copy, at K block 0
  uint32_t soff, sstep;        // its scale copy, and the step to the next K block
  uint32_t lds;                // LDS address of the stages
  int wave, woff, xoff, s0;    // fragment addresses in a stage: row, first chunk
  int sxoff, swoff;            // scale addresses in a stage
};

// Copies of K block kb into the stage at LDS offset st: this wave's 1 KB
// pieces (piece p is rows 8 p .. 8 p + 7 of the W tile, then of the X tile)
// and the scales of X (even waves) or W (odd waves; all of them write the
// same bytes, so that every wave has as many copies in flight).
template <class T, bool WROWS>
__device__ __forceinline__ void fp8_copy_piece(const Fp8Wave& g, uint32_t st, int kb, int i) {
  if (i < T::LOADS) {
    const int p = g.wave * T::LOADS + i;   // uniform
    lds_copy<16>(p < T::BN / 8 ? g.rw : g.rx, g.lds + st + p * 1024, g.off[i], kb * 128);
  } else if ((g.wave & 1) == 0) {
    lds_copy<4>(g.rs, g.lds + st + T::SX, g.soff, kb * g.sstep);
  } else if (WROWS) {
    lds_copy<4>(g.rs, g.lds + st + T::SW, g.soff, kb * g.sstep);
  } else {
    lds_copy<1>(g.rs, g.lds + st + T::SW, g.soff, kb * g.sstep);
  }
}
template <class T, bool WROWS>
__device__ __forceinline__ void fp8_copy(const Fp8Wave& g, uint32_t st, int kb) {
#pragma unroll
  for (int i = 0; i <= T::LOADS; ++i) fp8_copy_piece<T, WROWS>(g, st, kb, i);
}

// Wait until at most `blocks` K blocks' copies of this wave are under way,
// and for all its LDS reads.
template <class T>
__device__ __forceinline__ void fp8_wait(int blocks) {
  // a constant for every count that a ring of up to 4 stages has
  if (blocks <= 0)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
  else if (blocks == 1 || T::NST <= 2)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(T::LOADS + 1, 0));
  else if (blocks == 2 || T::NST <= 3)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * (T::LOADS + 1), 0));
  else
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(3 * (T::LOADS + 1), 0));
}

__device__ __forceinline__ i32x8 fp8_frag(const uint8_t* p, int s0) {
  const u32x4 lo = *reinterpret_cast<const u32x4*>(p + s0);
  const u32x4 hi = *reinterpret_cast<const u32x4*>(p + (s0 ^ 16));
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// A K block's scales of this lane's rows: words of four bytes, or bytes.
template <class T>
struct Fp8Scales {
  uint32_t x[T::XW], w[T::WW];
};
template <class T, bool WROWS>
__device__ __forceinline__ Fp8Scales<T> fp8_scales(const Fp8Wave& g, const uint8_t* st) {
  Fp8Scales<T> s;
#pragma unroll
  for (int i = 0; i < T::XW; ++i)
    s.x[i] = T::FM % 4 ? st[g.sxoff + i] : *reinterpret_cast<const uint32_t*>(st + g.sxoff + 4 * i);
#pragma unroll
  for (int i = 0; i < (WROWS ? T::WW : 1); ++i)
    s.w[i] = WROWS && T::FN % 4 ? st[g.swoff + i] : *reinterpret_cast<const uint32_t*>(st + g.swoff + 4 * i);
  return s;
}

// The K loop: wait for the block's copies, meet the others (which ends their
// reads of the previous block's stage), start the copies of block kb + NST -
// 1 there, multiply.  bf16 results on the scaled matrix core, fp32 results
// as bf16 products (twice the matrix time).
template <class T, bool WROWS, bool F32>
__device__ __forceinline__ void fp8_loop(const Fp8Wave& g, int kblocks, const uint8_t* lds,
                                         f32x4 (&acc)[T::FN][T::FM]) {
  constexpr int FN = T::FN, FM = T::FM, LAST = T::NST * T::STAGE;
#pragma unroll
  for (int k = 0; k < T::NST - 1; ++k)
    if (k < kblocks) fp8_copy<T, WROWS>(g, k * T::STAGE, k);
  int st = 0;
  for (int kb = 0; kb < kblocks; ++kb) {
    fp8_wait<T>(min(T::NST - 1, kblocks - kb) - 1);
    barrier_only();
    const uint32_t prev = st == 0 ? LAST - T::STAGE : st - T::STAGE;
    const bool more = kb + T::NST - 1 < kblocks;
    // A copy instruction holds its wave until the CU's memory pipe takes it
    // (17 cycles each).  With one workgroup on a CU they are spread over the
    // rows of products (256 x 256 tiles -3%); with two, which fill each
    // other's gaps, they go first (128 x 128 tiles: spread +7%).
    constexpr int PER = T::SPREAD ? (T::LOADS + FN) / FN : T::LOADS + 1;
    auto copies = [&](int i) {
      if (more) {
#pragma unroll
        for (int c = i * PER; c < (i + 1) * PER && c <= T::LOADS; ++c)
          fp8_copy_piece<T, WROWS>(g, prev, kb + T::NST - 1, c);
      }
    };
    const uint8_t* cur = lds + st;
    if (!T::SPREAD) copies(0);
    const Fp8Scales<T> c = fp8_scales<T, WROWS>(g, cur);
    if (F32) {
      bf16x8 b[FM][4];
#pragma unroll
      for (int j = 0; j < FM; ++j)
        fp8_to_bf16(fp8_frag(cur + g.xoff + j * 2048, g.s0), byte_of(c.x[FM % 4 ? j : j >> 2], FM % 4 ? 0 : j & 3), b[j]);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        bf16x8 a[4];
        fp8_to_bf16(fp8_frag(cur + g.woff + i * 2048, g.s0),
                    byte_of(c.w[!WROWS ? 0 : FN % 4 ? i : i >> 2], WROWS && FN % 4 == 0 ? i & 3 : 0), a);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < FM; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s], b[j][s], acc[i][j], 0, 0, 0);
        if (T::SPREAD) copies(i);
      }
    } else {
      i32x8 b[FM];
#pragma unroll
      for (int j = 0; j < FM; ++j) b[j] = fp8_frag(cur + g.xoff + j * 2048, g.s0);
      i32x8 a[2];
      a[0] = fp8_frag(cur + g.woff, g.s0);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        // one workgroup: the next row's fragment is read a row ahead
        if (T::SPREAD && i + 1 < FN) a[(i + 1) & 1] = fp8_frag(cur + g.woff + (i + 1) * 2048, g.s0);
        if (!T::SPREAD && i > 0) a[i & 1] = fp8_frag(cur + g.woff + i * 2048, g.s0);
        if (T::SPREAD) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < FM; ++j)
          acc[i][j] = fp8_mfma(a[i & 1], b[j], acc[i][j], WROWS && FN % 4 == 0 ? i & 3 : 0,
                               (int)c.w[!WROWS ? 0 : FN % 4 ? i : i >> 2],
                               FM % 4 ? 0 : j & 3, (int)c.x[FM % 4 ? j : j >> 2]);
        if (T::SPREAD) {
          __builtin_amdgcn_sched_barrier(0);
          copies(i);
        }
      }
    }
    st = st + T::STAGE == LAST ? 0 : st + T::STAGE;
  }
}

// Tile `item` of the order in which bands of 8 m-tiles run through all
// n-tiles, m fastest.
__device__ __forceinline__ void fp8_tile_at(int item, int ntiles, int mtiles, int& nt, int& mt) {
  const int band = item / (8 * ntiles), rows = min(8, mtiles - 8 * band);
  const int local = item - band * 8 * ntiles;
  mt = band * 8 + local % rows;
  nt = local / rows;
}

// One BN x BM tile per workgroup; K in steps of one scale block (128).  In
// LDS an operand's 16-row fragments follow each other, a row is 128 bytes in
// 16-byte chunks, and chunk c of fragment row r sits at slot c ^ (r / 2 % 8):
// the rows that a read touches in one cycle spread over all banks.
//
// 8192^3 in 256 x 256 tiles, bf16 results: 410 us (2680 TFLOP/s) on a cool card,
// 465 to 503 (2190) at the clock it holds after other such work; fp32 results
// 770 to 810 us; 4096^3 56 us, 2450.  The rest was measured at 503.  What
// bounds it: a K block's matrix instructions and its LDS traffic (192 KB of
// fragments, 64 KB of copies) take 2048 cycles each, so the two have to overlap
// fully; the matrix cores are busy 57% of the time at the 1.8 GHz of that run.
// Without the products the same loop takes 307 us, without the copies 413,
// without the LDS reads 456.  Tried and dropped: four waves of 128 x 128 (537
// us), fragments of the next K block read ahead (registers spill), workgroups
// that stay for several tiles and start the next one's copies under the last
// K block (512 against 505).
template <class T, bool WROWS, bool F32>
__global__ __launch_bounds__(64 * T::NW) void fp8_gemm_kernel(Fp8Gemm g, int ntiles, int mtiles,
                                                              int first, int count, int splits) {
  constexpr int FN = T::FN, FM = T::FM, WM = T::WM;
  __shared__ __align__(1024) uint8_t lds[T::NST * T::STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  Fp8Wave v;
  v.wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Tiles `first` .. `first + count - 1`: XCD x takes a contiguous range of
  // them (with splits, every tile's parts one after the other).
  int nt, mt, split, tile;
  {
    const int L = count * splits, b = blockIdx.x;
    const int x = b & 7, base = L >> 3, extra = L & 7;
    const int item = x * base + min(x, extra) + (b >> 3);
    split = item % splits;
    tile = item / splits;
    fp8_tile_at(first + tile, ntiles, mtiles, nt, mt);
  }
  const int64_t n0 = (int64_t)nt * T::BN, m0 = (int64_t)mt * T::BM;
  const int64_t pitch = fp8_pitch(g.K);
  const int all = (int)(pitch / 128);
  const int kb0 = (int)((int64_t)all * split / splits), kblocks = (int)((int64_t)all * (split + 1) / splits) - kb0;
  // copies: lane l brings slot l % 8 of row l / 8 of a piece.  Rows past the
  // matrix repeat its last row (their results are dropped).
  const int nrows = (int)min((int64_t)T::BN, g.N - n0), mrows = (int)min((int64_t)T::BM, g.M - m0);
  v.rw = buffer_of(g.w + n0 * pitch, nrows * pitch);
  v.rx = buffer_of(g.x + m0 * pitch, mrows * pitch);
  v.lds = (uint32_t)(uintptr_t)(lptr_t)lds;
#pragma unroll
  for (int i = 0; i < T::LOADS; ++i) {
    const int p = v.wave * T::LOADS + i;
    const bool isw = p < T::BN / 8;
    const int at = 8 * (isw ? p : p - T::BN / 8) + (lane >> 3);   // LDS row of the operand
    const int fr = at & 15, f = at >> 4;                          // its fragment row and fragment
    const int row = isw ? f / FN * 16 * FN + fp8_pi(fr) * FN + f % FN : f / FM * 16 * FM + fr * FM + f % FM;
    v.off[i] = (uint32_t)min(row, (isw ? nrows : mrows) - 1) * (uint32_t)pitch + (uint32_t)kb0 * 128 +
               (((lane & 7) ^ ((fr >> 1) & 7)) << 4);
  }
  // scale copies: four bytes a lane of a K block's row of scales, or with
  // 128-row blocks of W one byte a lane, from the tile's first on (within
  // the row of scales; lanes past the tile bring bytes that are not read)
  {
    const int64_t swp = WROWS ? fp8_scale_pitch(g.N) : (g.N + 127) / 128, sxp = fp8_scale_pitch(g.M);
    const bool isw = v.wave & 1;
    const int64_t sp = isw ? swp : sxp, at = isw ? (WROWS ? n0 : n0 / 128) : m0;
    const int left = (int)min(sp - at, (int64_t)256);   // >= 16, or >= 1 of single bytes
    v.soff = (isw && !WROWS) ? min(lane, left - 1) : min(4 * lane, left - 4);
    v.sstep = (uint32_t)sp;
    v.rs = buffer_of((isw ? g.sw : g.sx) + kb0 * sp + at, (kblocks - 1) * sp + left);
  }
  const int wn = v.wave / WM, wm = v.wave % WM;
  const int r = lane & 15, q = lane >> 4;
  v.woff = (wn * 16 * FN + r) * 128;
  v.xoff = (T::BN + wm * 16 * FM + r) * 128;
  v.s0 = ((2 * q) ^ ((r >> 1) & 7)) << 4;
  v.sxoff = T::SX + wm * 16 * FM + r * FM;
  v.swoff = T::SW + (WROWS ? wn * 16 * FN + fp8_pi(r) * FN : wn * 16 * FN / 128 * 4);
  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  fp8_loop<T, WROWS, F32>(v, kblocks, lds, acc);
  const int64_t nw0 = n0 + wn * 16 * FN;
  const bool wide = g.N % FN == 0;
  if (splits > 1) {   // the tile's part, the rows that exist, as [BM][BN] fp32
    float* part = g.part + ((int64_t)split * count + tile) * (T::BN * T::BM);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      if (wm * 16 * FM + r * FM + j >= mrows) break;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float* d = part + (wm * 16 * FM + r * FM + j) * T::BN + wn * 16 * FN + (4 * t + q) * FN;
#pragma unroll
        for (int i = 0; i < FN; i += FN < 4 ? FN : 4) {
          if constexpr (FN < 4)
            *reinterpret_cast<f32x2*>(d) = f32x2{acc[0][j][t], acc[1][j][t]};
          else
            *reinterpret_cast<f32x4*>(d + i) = f32x4{acc[i][j][t], acc[i + 1][j][t], acc[i + 2][j][t], acc[i + 3][j][t]};
        }
      }
    }
    return;
  }
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

// The sum of each tile's `splits` fp32 parts in their order, plus the bias:
// 1024 values of a tile per workgroup, 4 a thread.  Latency and the parts'
// bytes: 128 x 512 in 8 parts in 4.6 us.
template <bool F32>
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8Gemm g, int ntiles, int mtiles, int first,
                                                       int count, int splits, int bn, int bm) {
  const int per = bn * bm / 1024, tile = blockIdx.x / per;
  const int i = (blockIdx.x % per * 256 + threadIdx.x) * 4;   // in the tile
  int nt, mt;
  fp8_tile_at(first + tile, ntiles, mtiles, nt, mt);
  const int64_t m = (int64_t)mt * bm + i / bn, n = (int64_t)nt * bn + i % bn;
  if (m >= g.M || n >= g.N) return;
  const float* p = g.part + (int64_t)tile * bn * bm + i;
  const int64_t step = (int64_t)count * bn * bm;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(p + s * step);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += x[e];
  }
  fp8_store<4, F32>(g, m, n, v, g.N % 4 == 0);
}

// Few rows: a workgroup takes 16 rows of W and its waves split the K blocks;
// every wave streams its part of W straight into fragments and the partial
// sums meet in LDS in wave order.  Lane (r, q) takes bytes 16 q .. + 15 and
// 64 + 16 q .. + 15 of its row's block, of W and of X alike, so a load
// instruction brings 64 contiguous bytes of each of 16 rows.
constexpr int SK_NW = 8, SK_CH = 3;   // waves; K blocks in flight per wave

// A row's fragments and scales of K blocks c0 .. c0 + SK_CH - 1 (past b1 - 1: that
// block again, not multiplied).
struct SkinnyW {
  u32x4 lo[SK_CH], hi[SK_CH];
  uint32_t s[SK_CH];
};
__device__ __forceinline__ void skinny_load(const uint8_t* w, const uint8_t* sw, int64_t swp, int c0,
                                            int b1, SkinnyW& f) {
#pragma unroll
  for (int u = 0; u < SK_CH; ++u) {
    const int64_t kb = min(c0 + u, b1 - 1);
    f.lo[u] = gload16(w + kb * 128);
    f.hi[u] = gload16(w + kb * 128 + 64);
    f.s[u] = sw[kb * swp];
  }
}
template <bool F32>
__device__ __forceinline__ f32x4 skinny_product(const u32x4& wl, const u32x4& wh, uint32_t sw,
                                                const u32x4& xl, const u32x4& xh, uint32_t sx, f32x4 acc) {
  const i32x8 a = {(int)wl[0], (int)wl[1], (int)wl[2], (int)wl[3], (int)wh[0], (int)wh[1], (int)wh[2], (int)wh[3]};
  const i32x8 b = {(int)xl[0], (int)xl[1], (int)xl[2], (int)xl[3], (int)xh[0], (int)xh[1], (int)xh[2], (int)xh[3]};
  if (!F32) return fp8_mfma<0, 0>(a, b, acc, (int)sw, (int)sx);
  bf16x8 av[4], bv[4];
  fp8_to_bf16(a, sw, av);
  fp8_to_bf16(b, sx, bv);
#pragma unroll
  for (int t = 0; t < 4; ++t) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[t], bv[t], acc, 0, 0, 0);
  return acc;
}
// The waves' sums in their order, plus the bias, by the first wave.  Lane l
// holds D rows 4 (l / 16) .. + 3 (n) of column l % 16 (m).
template <bool F32>
__device__ __forceinline__ void skinny_store(const Fp8Gemm& g, f32x4 (*part)[64], int64_t n0, int wave, int lane) {
  if (wave) return;
  f32x4 sum = part[0][lane];
#pragma unroll
  for (int u = 1; u < SK_NW; ++u) sum += part[u][lane];
  float o[4] = {sum[0], sum[1], sum[2], sum[3]};
  fp8_store<4, F32>(g, lane & 15, n0 + 4 * (lane >> 4), o, g.N % 4 == 0);
}

// 8-bit X, up to 16 rows: X's fragments come straight from memory too, all
// loads of SK_CH K blocks before the first product.  Bound by the latency of
// W's loads: 16 rows by 5760 x 2880 from HBM in 8.4 us, one row in 6.6 (16.6
// MB, 2.0 and 2.5 TB/s).
template <bool WROWS, bool F32>
__global__ __launch_bounds__(64 * SK_NW) void fp8_skinny_kernel(Fp8Gemm g) {
  __shared__ f32x4 part[SK_NW][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t pitch = fp8_pitch(g.K);
  const int kblocks = (int)(pitch / 128);
  const int b0 = wave * kblocks / SK_NW, b1 = (wave + 1) * kblocks / SK_NW;
  const int64_t n = min(n0 + r, g.N - 1), m = min((int64_t)r, g.M - 1);
  const uint8_t* w = g.w + n * pitch + 16 * q;
  const uint8_t* x = g.x + m * pitch + 16 * q;
  const int64_t sxp = fp8_scale_pitch(g.M);
  const int64_t swp = WROWS ? fp8_scale_pitch(g.N) : (g.N + 127) / 128;
  const uint8_t* sw = g.sw + (WROWS ? n : n / 128);
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = b0; c0 < b1; c0 += SK_CH) {
    SkinnyW fx, fw;
    skinny_load(x, g.sx + m, sxp, c0, b1, fx);
    skinny_load(w, sw, swp, c0, b1, fw);
#pragma unroll
    for (int u = 0; u < SK_CH; ++u) {
      if (c0 + u >= b1) continue;
      acc = skinny_product<F32>(fw.lo[u], fw.hi[u], fw.s[u], fx.lo[u], fx.hi[u], fx.s[u], acc);
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  skinny_store<F32>(g, part, n0, wave, lane);
}

// bf16 X of up to 16 rows, rounded to E4M3 here: every workgroup rounds all
// of X into LDS (16 lanes a block, 8 elements a lane), while its first W
// loads are under way.  Rounding in the lanes that feed the matrix core
// instead repeated it for the 16 columns, and was most of the time at one
// row.  LDS row kb * M + m holds row m's block kb, 16-byte chunk c at slot c
// ^ (m % 8).  One row by 5760 x 2880 from HBM in 7.1 us, 2.3 TB/s, of which
// the launch is about 3.
constexpr int FUSED_BYTES = 32768, FUSED_ROUNDS = FUSED_BYTES / 8 / (64 * SK_NW);

template <bool F32, bool VEC>
__global__ __launch_bounds__(64 * SK_NW) void fp8_fused_kernel(Fp8Gemm g, const uint16_t* __restrict__ xb) {
  __shared__ __align__(16) uint8_t xs[FUSED_BYTES];
  __shared__ uint8_t sxs[FUSED_BYTES / 128];
  __shared__ f32x4 part[SK_NW][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t pitch = fp8_pitch(g.K);
  const int M = (int)g.M, kblocks = (int)(pitch / 128);
  const int b0 = wave * kblocks / SK_NW, b1 = (wave + 1) * kblocks / SK_NW;
  const int64_t n = min(n0 + r, g.N - 1);
  const uint8_t* w = g.w + n * pitch + 16 * q;
  const int64_t swp = (g.N + 127) / 128;
  const uint8_t* sw = g.sw + n / 128;
  // the 8 elements of X of each of this thread's turns, then W's first chunk
  const int groups = M * kblocks * 16, turns = (groups + 64 * SK_NW - 1) / (64 * SK_NW);   // turns <= FUSED_ROUNDS
  u32x4 xv[FUSED_ROUNDS];
  if (VEC) {
#pragma unroll
    for (int u = 0; u < FUSED_ROUNDS; ++u) {
      if (u >= turns) break;
      const int id = min(tid + u * 64 * SK_NW, groups - 1), row = id >> 4;
      const int64_t k0 = (int64_t)(row / M) * 128 + 8 * (id & 15);
      xv[u] = gload16(xb + (int64_t)(row % M) * g.K + min(k0, g.K - 8));   // past K: zeroed below
    }
  }
  SkinnyW f;
  if (b0 < b1) skinny_load(w, sw, swp, b0, b1, f);
#pragma unroll
  for (int u = 0; u < FUSED_ROUNDS; ++u) {
    if (u >= turns) break;
    const int id = tid + u * 64 * SK_NW, row = id >> 4, l = id & 15, m = row % M;
    if (id >= groups) break;   // whole blocks: the 16 lanes of one leave together
    const int64_t k0 = (int64_t)(row / M) * 128 + 8 * l;
    float v[8];
    if (VEC) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t h = xv[u][i >> 1];
        v[i] = k0 < g.K ? __uint_as_float((i & 1) ? h & 0xFFFF0000u : h << 16) : 0.0f;
      }
    } else {
      load8<false, false>(xb, m * g.K + k0, g.K - k0, v);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, finite_bits(v[i]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const int e = e4m3_exponent(top);
    const float k = e4m3_inverse(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = nan_unless_finite(v[i]) * k;
    *reinterpret_cast<u32x2*>(xs + row * 128 + (((l >> 1) ^ (m & 7)) << 4) + 8 * (l & 1)) =
        u32x2{e4m3_pack4(v[0], v[1], v[2], v[3]), e4m3_pack4(v[4], v[5], v[6], v[7])};
    if (l == 0) sxs[row] = (uint8_t)(e + 127);
  }
  wave_lds_sync();
  barrier_only();   // leaves W's loads under way
  const int m = min(r, M - 1);
  const uint8_t* x = xs + m * 128;
  const int s0 = (q ^ (m & 7)) << 4, s1 = ((q + 4) ^ (m & 7)) << 4;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = b0; c0 < b1; c0 += SK_CH) {
    if (c0 > b0) skinny_load(w, sw, swp, c0, b1, f);
#pragma unroll
    for (int u = 0; u < SK_CH; ++u) {
      const int kb = c0 + u;
      if (kb >= b1) continue;
      const u32x4 xl = *reinterpret_cast<const u32x4*>(x + kb * M * 128 + s0);
      const u32x4 xh = *reinterpret_cast<const u32x4*>(x + kb * M * 128 + s1);
      acc = skinny_product<F32>(f.lo[u], f.hi[u], f.s[u], xl, xh, sxs[kb * M + m], acc);
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  skinny_store<F32>(g, part, n0, wave, lane);
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

hipError_t launch_fp8_quantize_cols_pair(const uint16_t* x, int64_t K, uint8_t* codes, uint8_t* scales,
                                         const uint16_t* x2, int64_t K2, uint8_t* codes2,
                                         uint8_t* scales2, int64_t rows, hipStream_t s) {
  auto of = [](const uint16_t* p, int64_t k, uint8_t* c, uint8_t* sc) {
    return Fp8Cols{p, k, fp8_scale_pitch(k), c, sc, (int)((k + 63) / 64),
                   k % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0};
  };
  const Fp8Cols a = of(x, K, codes, scales), b = of(x2, K2, codes2, scales2);
  const int64_t rb = (rows + 127) / 128, blocks = rb * a.ctiles, all = blocks + rb * b.ctiles;
  hipLaunchKernelGGL(fp8_cols_pair_kernel, dim3((unsigned)all), dim3(256), 0, s, a, b, rows,
                     fp8_pitch(rows), (unsigned)blocks);
  return hipGetLastError();
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

// Tiles first .. first + count - 1, in `splits` parts of K.
template <class T>
static hipError_t gemm_tiles(const Fp8Gemm& g, int first, int count, int splits, hipStream_t s) {
  const int nt = (int)((g.N + T::BN - 1) / T::BN), mt = (int)((g.M + T::BM - 1) / T::BM);
  const dim3 grid((unsigned)((int64_t)count * splits)), block(64 * T::NW);
  if (g.w_rows) {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_gemm_kernel<T, true, true>), grid, block, 0, s, g, nt, mt, first, count, splits);
    else
      hipLaunchKernelGGL((fp8_gemm_kernel<T, true, false>), grid, block, 0, s, g, nt, mt, first, count, splits);
  } else {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_gemm_kernel<T, false, true>), grid, block, 0, s, g, nt, mt, first, count, splits);
    else
      hipLaunchKernelGGL((fp8_gemm_kernel<T, false, false>), grid, block, 0, s, g, nt, mt, first, count, splits);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const dim3 join((unsigned)((int64_t)count * (T::BN * T::BM / 1024)));
  if (g.out_f32)
    hipLaunchKernelGGL(fp8_join_kernel<true>, join, dim3(256), 0, s, g, nt, mt, first, count, splits, T::BN, T::BM);
  else
    hipLaunchKernelGGL(fp8_join_kernel<false>, join, dim3(256), 0, s, g, nt, mt, first, count, splits, T::BN, T::BM);
  return hipGetLastError();
}

static hipError_t skinny(const Fp8Gemm& g, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * SK_NW);
  if (g.w_rows) {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_skinny_kernel<true, true>), grid, block, 0, s, g);
    else
      hipLaunchKernelGGL((fp8_skinny_kernel<true, false>), grid, block, 0, s, g);
  } else {
    if (g.out_f32)
      hipLaunchKernelGGL((fp8_skinny_kernel<false, true>), grid, block, 0, s, g);
    else
      hipLaunchKernelGGL((fp8_skinny_kernel<false, false>), grid, block, 0, s, g);
  }
  return hipGetLastError();
}

// How a product runs: a tile (-1: few rows), the tiles that are computed
// whole, and the parts of K in which the others are.
struct Fp8Plan {
  int tile, whole, rest, splits;
};

// The tiles, W rows x X rows, with what a launch of each takes, for bf16 and
// for fp32 results: `lat` us for a K block while a CU has one workgroup, `thr`
// us for each workgroup that a CU has when it has more, and `c` us for every
// `res` of them (launch, first copies, stores).  Fitted to launches of 64 to
// 2048 rows by 5760 x 2880, 2880 x 5760, 4096 x 4096 and 8192 x 1024 whose W
// comes from HBM; over 170 sizes of 1 to 2048 rows the choice is 1% slower on
// average than the best of all tiles and parts, at most 20%.
// Wide tiles keep the matrix cores busy, narrow ones reach all CUs and bring
// W faster (us; 5760 x 2880):
//   rows       64    128    256    512   1024   2048
//   256 x 256  38.2  38.9   41.2   41.0   41.1   41.7
//   256 x 192  36.7  38.0   37.9   38.1   38.2   39.1
//   128 x 192  21.6  22.7   24.3   24.9   46.3   48.4
//   128 x 128  23.5  28.2   27.7   27.5   32.1   54.5   two stages, two workgroups on a CU
//   128 x 128  18.4  20.1   19.9   20.1   38.3   57.1   three stages, one
//   64 x 128   14.4  15.3   15.5   24.5   34.4   60.1
//   64 x 64    12.2  12.6   17.8   26.6   44.2   84.1
//   32 x 64    10.1  14.1   18.7   31.0   54.8   99.5
//   32 x 32    10.5  12.8   22.6   35.6   64.7    121   (32 rows: 8.9)
struct Fp8Shape {
  int bn, bm, res;
  float lat[2], thr[2], c[2];
};
static constexpr Fp8Shape FP8_SHAPE[] = {
    {256, 256, 1, {1.40f, 2.52f}, {1.40f, 2.52f}, {7.5f, 10.3f}},
    {256, 192, 1, {1.33f, 2.12f}, {1.33f, 2.12f}, {7.2f, 9.3f}},
    {128, 192, 1, {0.73f, 1.28f}, {0.73f, 1.28f}, {7.0f, 7.4f}},
    {128, 128, 2, {0.90f, 1.00f}, {0.59f, 0.87f}, {4.9f, 5.8f}},
    {128, 128, 1, {0.60f, 1.08f}, {0.60f, 1.08f}, {5.7f, 5.8f}},
    {64, 128, 2, {0.46f, 0.65f}, {0.38f, 0.52f}, {4.4f, 4.6f}},
    {64, 64, 2, {0.37f, 0.55f}, {0.27f, 0.36f}, {3.9f, 4.0f}},
    {32, 64, 3, {0.28f, 0.38f}, {0.22f, 0.25f}, {3.7f, 3.8f}},
    {32, 32, 4, {0.24f, 0.37f}, {0.13f, 0.21f}, {3.5f, 3.5f}},
};

// The tile of the least time.  The tiles of a last round that leaves CUs idle
// may be split over K, in parts of 3 blocks or more; another launch joins the
// fp32 parts, which costs the launches and the parts' bytes (written and read
// at 4 TB/s).
static Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, bool f32) {
  // one fragment of rows: streaming W in 16-row groups over K, while there are
  // enough of these (16 rows, 5760 x 2880: 8.4 us against 8.9 in 32 x 32
  // tiles; 4096 x 4096: 7.4, 9.6; 512 x 8192: 10.7, 7.8)
  if (M <= 16 && N >= 1024) return {-1, 0, 0, 1};
  const int64_t kb = fp8_pitch(K) / 128;
  Fp8Plan best{};
  float least = -1.0f;
  for (int i = 0; i < (int)(sizeof(FP8_SHAPE) / sizeof(FP8_SHAPE[0])); ++i) {
    const Fp8Shape& t = FP8_SHAPE[i];
    const int64_t tiles = ((N + t.bn - 1) / t.bn) * ((M + t.bm - 1) / t.bm);
    if (tiles > 1 << 23) continue;   // more than a launch takes; the wide ones of such a product are fewer
    auto launch = [&](int64_t groups, int64_t blocks) {
      const int64_t w = (groups + 255) / 256, rounds = (w + t.res - 1) / t.res;
      const float block = w > 1 && t.thr[f32] * (float)w > t.lat[f32] ? t.thr[f32] * (float)w : t.lat[f32];
      return groups == 0 ? 0.0f : block * (float)blocks + t.c[f32] * (float)rounds;
    };
    const float us = launch(tiles, kb);
    if (least < 0.0f || us < least) {
      least = us;
      best = {i, (int)tiles, 0, 1};
    }
    const int64_t rest = tiles % (256 * t.res);
    if (rest == 0 || rest > 128) continue;
    const int64_t s = kb / 3 < 256 / rest ? kb / 3 : 256 / rest;
    if (s < 2) continue;
    const int64_t tile = (int64_t)t.bn * (M < t.bm ? M : t.bm);
    const float join = (tiles > rest ? 6.0f : 3.0f) + (float)(s * rest * tile) * 8.0f / 4.0e6f;
    const float split = launch(tiles - rest, kb) + launch(rest * s, (kb + s - 1) / s) + join;
    if (split < least) {
      least = split;
      best = {i, (int)(tiles - rest), (int)rest, (int)s};
    }
  }
  return best;
}

size_t fp8_part_bytes(int64_t M, int64_t N, int64_t K, int out_f32) {
  const Fp8Plan p = fp8_plan(M, N, K, out_f32 != 0);
  return p.rest ? (size_t)p.splits * p.rest * FP8_SHAPE[p.tile].bn * FP8_SHAPE[p.tile].bm * sizeof(float) : 0;
}

template <class T>
static hipError_t gemm(const Fp8Gemm& g, const Fp8Plan& p, hipStream_t s) {
  if (p.rest && !g.part) return hipErrorInvalidValue;
  if (p.whole) {
    const hipError_t e = gemm_tiles<T>(g, 0, p.whole, 1, s);
    if (e != hipSuccess) return e;
  }
  return p.rest ? gemm_tiles<T>(g, p.whole, p.rest, p.splits, s) : hipSuccess;
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t s) {
  const Fp8Plan p = fp8_plan(g.M, g.N, g.K, g.out_f32 != 0);
  switch (p.tile) {
    case 0: return gemm<Fp8Tile<2, 4, 8, 4, 2>>(g, p, s);
    case 1: return gemm<Fp8Tile<2, 4, 8, 3, 2>>(g, p, s);
    case 2: return gemm<Fp8Tile<2, 4, 4, 3, 3>>(g, p, s);
    case 3: return gemm<Fp8Tile<2, 2, 4, 4, 2>>(g, p, s);
    case 4: return gemm<Fp8Tile<2, 2, 4, 4, 3>>(g, p, s);
    case 5: return gemm<Fp8Tile<1, 4, 4, 2, 3>>(g, p, s);
    case 6: return gemm<Fp8Tile<1, 4, 4, 1, 4>>(g, p, s);
    case 7: return gemm<Fp8Tile<1, 4, 2, 1, 4>>(g, p, s);
    case 8: return gemm<Fp8Tile<1, 2, 2, 1, 4>>(g, p, s);
    default: return skinny(g, s);
  }
}

// The one-launch form: X's codes fit its LDS, and rounding them in every
// workgroup costs less than a launch of its own (5760 x 2880 from HBM, us: 5
// rows 9.1 against about 10, 8 rows 10.9, 9.8; 2880 x 5760, 5 rows 11.0, 9.5).
// With few columns, whose product also joins K parts, it may cost more (512 x
// 2880, 8 rows 7.4, 9.0).
bool fp8_fused_fits(int64_t M, int64_t N, int64_t K) {
  return M <= 16 && M * fp8_pitch(K) <= (N < 1024 ? FUSED_BYTES : FUSED_BYTES / 2);
}

hipError_t launch_fp8_fused(const Fp8Gemm& g, const uint16_t* x, hipStream_t s) {
  if (!fp8_fused_fits(g.M, g.N, g.K)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * SK_NW);
  const bool vec = g.K % 8 == 0 && (reinterpret_cast<uintptr_t>(x) % 16) == 0;
  if (g.out_f32) {
    if (vec)
      hipLaunchKernelGGL((fp8_fused_kernel<true, true>), grid, block, 0, s, g, x);
    else
      hipLaunchKernelGGL((fp8_fused_kernel<true, false>), grid, block, 0, s, g, x);
  } else {
    if (vec)
      hipLaunchKernelGGL((fp8_fused_kernel<false, true>), grid, block, 0, s, g, x);
    else
      hipLaunchKernelGGL((fp8_fused_kernel<false, false>), grid, block, 0, s, g, x);
  }
  return hipGetLastError();
}

}  // namespace mxmoe
