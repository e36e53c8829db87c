// Dense products in microscaled 4-bit floating point (gfx950): E2M1 elements,
// a UE8M0 scale for each 32 of K, as the expert block's weights have them.
//
// out = X W^T with X rounded to MXFP4 and W as stored, on the scaled matrix
// core: v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands' codes and
// scales, its products are exact and its sums fp32 (with elements of 4 bits
// nothing is dropped: sums of blocks 2^24 apart came out as in fp32).  The
// input's gradient dX = dY W sums along W's rows, where a block of 32 has as
// many scales: no scaled product.  dY stays in bf16 and W is decoded, exactly,
// for the bf16 matrix core: as its codes are read for few rows of dY, else once
// into a transposed copy.
//
// Storage: W's codes stay where they are ([N, K / 2]); X's rows are padded
// with zeros to 256, so whatever a row of W is followed by is multiplied by 0.
// Scales are ordered for the matrix core's lanes: lane (r, q) of a fragment
// feeds row r's elements 64 q .. 64 q + 63 of a block of 256, in two
// instructions, so [K block][q][row][2] puts the two scales of all rows of a
// lane side by side.
#include "common.hpp"
#include "fp4.hpp"
#include "ring.hpp"

namespace mxmoe {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- quantizer

// Scale exponent of a block whose largest magnitude has these bits: the
// smallest e with amax <= 6 * 2^e, at least -127.
__device__ __forceinline__ int e2m1_exponent(uint32_t amax_bits) {
  const int E = (int)(amax_bits >> 23);
  return E == 0 ? -127 : max(E - 129 + ((amax_bits & 0x7FFFFFu) > 0x400000u), -127);
}

// A lane's eight elements of a block of 32 (four lanes side by side) -> their
// codes; the block's scale byte.  A block with an infinity or a NaN has the
// scale NaN (255) and codes 0.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));   // lanes ^ 1
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));   // lanes ^ 2
}
__device__ __forceinline__ uint32_t fp4_codes(const float (&v)[8], uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = quad_max(m);
  if (m >= 0x7F800000u) {
    scale = 255;
    return 0;
  }
  scale = (uint32_t)(e2m1_exponent(m) + 127);
  const float f = scale_operand(scale);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], f, 3);
}
// the same of eight bf16 as they are stored
__device__ __forceinline__ uint32_t fp4_codes(const u32x4& x, uint32_t& scale) {
  u16x2 t = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, x[i] & 0x7FFF7FFFu));
  const uint32_t m = quad_max(max((uint32_t)t[0], (uint32_t)t[1])) << 16;
  if (m >= 0x7F800000u) {
    scale = 255;
    return 0;
  }
  scale = (uint32_t)(e2m1_exponent(m) + 127);
  const float f = scale_operand(scale);
  // (a bit cast of a vector's element itself takes the first one's bits)
  const uint32_t x0 = x[0], x1 = x[1], x2 = x[2], x3 = x[3];
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x0), f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x1), f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x2), f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x3), f, 3);
}

// The memory takes 16-byte accesses at any element, so rows of any length are
// read and written so, but for their ends.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
typedef uint32_t __attribute__((aligned(2))) u32_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef f32x2 __attribute__((aligned(4))) f32x2_any;

// Eight consecutive elements of a row as bf16 pairs, zeros from `left` on.
// WHOLE: rows have no ends.
template <bool WHOLE>
__device__ __forceinline__ u32x4 bf16x8_at(const uint16_t* x, int64_t at, int64_t left) {
  u32x4 r = {0u, 0u, 0u, 0u};
  if (WHOLE ? left > 0 : left >= 8) {
    r = *reinterpret_cast<const u32x4_any*>(x + at);
  } else if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) r[i >> 1] |= (uint32_t)x[at + i] << (16 * (i & 1));
  }
  return r;
}

// One K block of 256 of 16 rows per workgroup: 32 lanes a row, 8 elements
// each, two rounds of 8 rows; the scales leave by LDS in their order.  bf16
// pairs are rounded as they are stored: the maximum as 16-bit integers, the
// conversion by the hardware's, whose ties go to even.  Bound by HBM: 16384 x
// 2880 bf16 in 22 to 29 us (with X in the last-level cache, or not), 4.2 TB/s;
// 2047 x 2880 in 4.8.
template <bool F32, bool WHOLE>
__global__ __launch_bounds__(256) void fp4_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t K,
                                                       int64_t pitch, int64_t srows, int kblocks,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t sc[128];   // [4][16 rows][2]
  const int kb = blockIdx.x % kblocks, tid = threadIdx.x, l = tid & 31;
  const int64_t r0 = (int64_t)(blockIdx.x / kblocks) * 16, k0 = (int64_t)kb * 256 + 8 * l;
  uint32_t c[2], s[2];
  if (F32) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int64_t row = r0 + 8 * p + (tid >> 5), left = row < rows ? K - k0 : 0;
      float v[8];
      if (WHOLE || left >= 8) {
        f32x4 a = {0, 0, 0, 0}, b = a;
        if (left > 0) {
          const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(x) + row * K + k0);
          a = q[0];
          b = q[1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = a[i];
          v[i + 4] = b[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? static_cast<const float*>(x)[row * K + k0 + i] : 0.0f;
      }
      c[p] = fp4_codes(v, s[p]);
    }
  } else {
    u32x4 v[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int64_t row = r0 + 8 * p + (tid >> 5);
      v[p] = bf16x8_at<WHOLE>(static_cast<const uint16_t*>(x), row * K + k0, row < rows ? K - k0 : 0);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) c[p] = fp4_codes(v[p], s[p]);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int at = 8 * p + (tid >> 5);
    const int64_t row = r0 + at;
    if (row < rows) *reinterpret_cast<uint32_t*>(codes + row * pitch + k0 / 2) = c[p];
    if ((l & 3) == 0) sc[(l >> 3) * 32 + at * 2 + ((l >> 2) & 1)] = (uint8_t)s[p];   // block l / 4: pair l / 8
  }
  __syncthreads();
  if (tid < 8)   // 16 rows' two bytes: 32 a pair
    *reinterpret_cast<u32x4*>(scales + ((int64_t)kb * 4 + (tid >> 1)) * srows * 2 + r0 * 2 + 16 * (tid & 1)) =
        *reinterpret_cast<const u32x4*>(sc + 16 * tid);
}

// Scales [rows, K / 32] into that order; zeros (2^-127) past K and past the rows.
__global__ __launch_bounds__(256) void fp4_scales_kernel(const uint8_t* __restrict__ scales, int64_t rows, int64_t k32,
                                                         int64_t srows, int64_t total, uint8_t* __restrict__ ordered) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // a pair of bytes: (K block * 4 + q) * srows + row
  if (i >= total) return;
  const int64_t row = i % srows, b = i / srows * 2;
  uint32_t v = 0;
  if (row < rows) {
    if (b < k32) v = scales[row * k32 + b];
    if (b + 1 < k32) v |= (uint32_t)scales[row * k32 + b + 1] << 8;
  }
  reinterpret_cast<uint16_t*>(ordered)[i] = (uint16_t)v;
}

// ------------------------------------------------------------------- products

template <int SEL_A, int SEL_B>
__device__ __forceinline__ f32x4 fp4_mfma(const i32x8& a, const i32x8& b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, SEL_A, sa, SEL_B, sb);
}
__device__ __forceinline__ f32x4 fp4_mfma(const i32x8& a, const i32x8& b, f32x4 c, int sel_a, int sa, int sel_b,
                                          int sb) {
  // the selectors are constants after unrolling
  switch (sel_a * 4 + sel_b) {
    case 0: return fp4_mfma<0, 0>(a, b, c, sa, sb);
    case 1: return fp4_mfma<0, 1>(a, b, c, sa, sb);
    case 2: return fp4_mfma<0, 2>(a, b, c, sa, sb);
    case 3: return fp4_mfma<0, 3>(a, b, c, sa, sb);
    case 4: return fp4_mfma<1, 0>(a, b, c, sa, sb);
    case 5: return fp4_mfma<1, 1>(a, b, c, sa, sb);
    case 6: return fp4_mfma<1, 2>(a, b, c, sa, sb);
    case 7: return fp4_mfma<1, 3>(a, b, c, sa, sb);
    case 8: return fp4_mfma<2, 0>(a, b, c, sa, sb);
    case 9: return fp4_mfma<2, 1>(a, b, c, sa, sb);
    case 10: return fp4_mfma<2, 2>(a, b, c, sa, sb);
    case 11: return fp4_mfma<2, 3>(a, b, c, sa, sb);
    case 12: return fp4_mfma<3, 0>(a, b, c, sa, sb);
    case 13: return fp4_mfma<3, 1>(a, b, c, sa, sb);
    case 14: return fp4_mfma<3, 2>(a, b, c, sa, sb);
    default: return fp4_mfma<3, 3>(a, b, c, sa, sb);
  }
}
// 16 bytes of codes as an operand (4-bit formats read its first four registers)
__device__ __forceinline__ i32x8 fp4_operand(const u32x4& v) {
  const i32x4 x = __builtin_bit_cast(i32x4, v);
  return __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
}

// A workgroup's tile: WN x WM waves of (16 FN) x (16 FM), and NST LDS stages.
// A stage holds one K block, 128 bytes of each of BN rows of W and BM rows of
// X (256 elements in 4 bits, 64 in bf16), and in 4 bits their scales: 8 bytes
// a row, [4][rows][2].  Copies bring 1 KB.
template <int WN_, int WM_, int FN_, int FM_, int NST_, bool FP4_>
struct Fp4Tile {
  static constexpr int WN = WN_, WM = WM_, FN = FN_, FM = FM_, NST = NST_;
  static constexpr bool FP4 = FP4_;
  static constexpr int NW = WN * WM;
  static constexpr int BN = WN * FN * 16, BM = WM * FM * 16;
  static constexpr int CX = FP4 ? (BM + 127) / 128 : 0, CW = FP4 ? (BN + 127) / 128 : 0;   // scale copies
  static constexpr int SX = (BN + BM) * 128, SW = SX + CX * 1024, STAGE = SW + CW * 1024;
  static constexpr int LOADS = (BN + BM) / 8 / NW;   // copies of rows per wave and step
  static constexpr int COPIES = LOADS + (FP4 ? 1 : 0);
  static_assert(LOADS <= 8 && LOADS * NW * 8 == BN + BM && CX + CW <= NW, "copies");
  static_assert(BN <= 256 && BM <= 256 && NST >= 2 && NST <= 4 && NST * STAGE <= 160 * 1024, "LDS");
  static_assert(NST * COPIES < 64, "vector-memory counter");
  static constexpr bool SEVERAL = BN * BM >= 128 * 128;   // a workgroup may take several tiles
  static constexpr int AHEAD = FN > 2 ? 3 : 2;       // steps that fragments are read ahead
  // words with the scale pairs of a lane's rows: two rows a word, or with odd F one
  static constexpr int XW = FM % 2 ? FM : FM / 2, WW = FN / 2;
  static_assert(FN == 2 || FN == 4 || FN == 8, "pairs of scales, steps");
};

// The 16-byte slot of a fragment row's chunk c in LDS.  A 16-byte read serves
// 16 lanes in two cycles, eight rows of one lane quarter (0-3 and 12-15, or
// 4-11) and the other eight of the next quarter, and there are 16 slots in the
// 64 banks: these slots differ for all 16.  (With
// row / 2 alone every read took twice its cycles.)
__device__ __forceinline__ int fp4_slot(int row, int c) {
  return c ^ (((row ^ row >> 1) >> 2 & 1) << 2 | (row >> 1 & 1) << 1 | row >> 3);
}

// A wave's part of a tile's main loop.
struct Fp4Wave {
  u32x4 rw, rx, rs;            // W's and X's rows of the tile, and this wave's scales
  uint32_t off[8];             // this lane's 16 bytes of each copy, at K block 0
  uint32_t soff, sstep;        // its scale copy, and the step to the next K block
  uint32_t sdst;               // where in a stage its scales go
  uint32_t lds;                // LDS address of the stages
  int wave, woff, xoff, s0;    // fragment addresses in a stage: row, first chunk
  int sxoff, swoff;            // scale addresses in a stage
};

// Copies of K block kb into the stage at LDS offset st: this wave's 1 KB
// pieces (rows of the W tile, then of the X tile) and one of the scales'
// (several waves may write the same bytes, so that every wave has as many
// copies in flight).  Where W's rows end inside the last block, the copies go on
// into the next row, which meets zeros of X; behind the tile's last row the
// buffer ends, and its bounds check gives zeros.
template <class T>
__device__ __forceinline__ void fp4_copy_piece(const Fp4Wave& g, uint32_t st, int kb, int i) {
  if (i < T::LOADS) {
    const int p = g.wave * T::LOADS + i;   // uniform
    lds_copy<16>(p < T::BN / 8 ? g.rw : g.rx, g.lds + st + p * 1024, g.off[i], kb * 128);
  } else {
    lds_copy<16>(g.rs, g.lds + st + g.sdst, g.soff, kb * g.sstep);
  }
}

// The scale pairs of a K block of this lane's rows.
template <class T>
struct Fp4Scales {
  uint32_t x[T::XW], w[T::WW];
};
template <class T>
__device__ __forceinline__ Fp4Scales<T> fp4_scales(const Fp4Wave& g, const uint8_t* st) {
  Fp4Scales<T> s;
#pragma unroll
  for (int i = 0; i < T::XW; ++i)
    s.x[i] = T::FM % 2 ? *reinterpret_cast<const uint16_t*>(st + g.sxoff + 2 * i)
                       : *reinterpret_cast<const uint32_t*>(st + g.sxoff + 4 * i);
#pragma unroll
  for (int i = 0; i < T::WW; ++i) s.w[i] = *reinterpret_cast<const uint32_t*>(st + g.swoff + 4 * i);
  return s;
}

// A K block's products, in steps of one fragment row of W by the wave's FM
// fragments of X (FM instructions): 2 FN steps, of which step s reads the
// fragment of step s + 3.  So a block's first reads come three steps before the
// last one ends, and the matrix cores have those steps' work while they wait:
// there, with all reads of the block behind it, a wave waits for its copies of
// the next block, meets the others, and starts the copies of the block NST
// further on into the stage that is free now.  One basic block: with branches
// in it the compiler gathers the products at its end.
template <class T>
struct Fp4Frags {
  u32x4 a[4], b[2][T::FM];   // fragments of W by step % 4, of X by half of the block
  Fp4Scales<T> c;
};
template <class T>
__device__ __forceinline__ void fp4_read_a(const Fp4Wave& g, const uint8_t* st, int step, Fp4Frags<T>& f) {
  f.a[step & 3] = *reinterpret_cast<const u32x4*>(st + g.woff + step % T::FN * 2048 + (step < T::FN ? g.s0 : g.s0 ^ 16));
}
template <class T>
__device__ __forceinline__ void fp4_read_b(const Fp4Wave& g, const uint8_t* st, int half, Fp4Frags<T>& f) {
#pragma unroll
  for (int j = 0; j < T::FM; ++j)
    f.b[half][j] = *reinterpret_cast<const u32x4*>(st + g.xoff + j * 2048 + (half ? g.s0 ^ 16 : g.s0));
}
// COPY: with copies of block kb of the tile that g has set out, else all that
// are under way are waited for.  `there`: the next block's have been waited for
// already.  Moves st on.
template <class T, bool COPY>
__device__ __forceinline__ void fp4_block(const Fp4Wave& g, int kb, int there, const uint8_t* lds, int& st,
                                          Fp4Frags<T>& f, f32x4 (&acc)[T::FN][T::FM]) {
  constexpr int FN = T::FN, FM = T::FM, S = 2 * FN, AHEAD = T::AHEAD, PER = (T::COPIES + AHEAD - 1) / AHEAD;
  const int after = st + T::STAGE == T::NST * T::STAGE ? 0 : st + T::STAGE;
  Fp4Scales<T> next{};
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (s == (FN > AHEAD ? FN - AHEAD : 0)) fp4_read_b<T>(g, lds + st, 1, f);
    if (s + AHEAD < S) {
      fp4_read_a<T>(g, lds + st, s + AHEAD, f);
    } else {
      if (s + AHEAD == S) {
        // (a branch of its own inside the assembly leaves the block whole)
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(%1)\n1:"
                     ::"s"(there), "n"(COPY ? (T::NST - 2) * T::COPIES : 0) : "scc", "memory");
        barrier_only();
        if (T::FP4) next = fp4_scales<T>(g, lds + after);
        fp4_read_b<T>(g, lds + after, 0, f);
      }
      fp4_read_a<T>(g, lds + after, s + AHEAD - S, f);
      if (COPY) {
#pragma unroll
        for (int i = (s + AHEAD - S) * PER; i < (s + AHEAD - S + 1) * PER && i < T::COPIES; ++i)
          fp4_copy_piece<T>(g, st, kb, i);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    const int i = s % FN, t = s / FN;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      if constexpr (T::FP4)
        acc[i][j] = fp4_mfma(fp4_operand(f.a[s & 3]), fp4_operand(f.b[t][j]), acc[i][j], 2 * (i & 1) + t,
                             (int)f.c.w[i >> 1], FM % 2 ? t : 2 * (j & 1) + t, (int)f.c.x[FM % 2 ? j : j >> 1]);
      else
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(f.a[s & 3]), as_bf16x8(f.b[t][j]), acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  f.c = next;
  st = after;
}

// F values of the bias from n on, zeros past N and without one.
template <int F>
__device__ __forceinline__ void fp4_bias(const uint16_t* bias, int64_t n, int64_t N, float (&v)[F]) {
  if (!bias) N = 0;
  if (n + F <= N) {
#pragma unroll
    for (int i = 0; i < F; i += 2) {
      const uint32_t w = *reinterpret_cast<const u32_any*>(bias + n + i);
      v[i] = __uint_as_float(w << 16);
      v[i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < F; ++i) v[i] = n + i < N ? bf16_to_f32(bias[n + i]) : 0.0f;
  }
}
// F consecutive results out[m][n ..].
template <int F, bool F32>
__device__ __forceinline__ void fp4_store(void* out, int64_t M, int64_t N, int64_t m, int64_t n, const float (&v)[F]) {
  if (m >= M) return;
  const int64_t at = m * N + n;
  if (n + F <= N) {
    if constexpr (F32) {
      float* d = static_cast<float*>(out) + at;
      if constexpr (F == 2) {
        *reinterpret_cast<f32x2_any*>(d) = f32x2{v[0], v[1]};
      } else {
#pragma unroll
        for (int i = 0; i < F; i += 4)
          *reinterpret_cast<f32x4_any*>(d + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
      }
    } else {
      uint16_t* d = static_cast<uint16_t*>(out) + at;
      if constexpr (F == 2)
        *reinterpret_cast<u32_any*>(d) = pack_bf16x2(v[0], v[1]);
      else if constexpr (F == 4)
        *reinterpret_cast<u32x2_any*>(d) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      else
        *reinterpret_cast<u32x4_any*>(d) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < F; ++i)
    if (n + i < N) {
      if (F32)
        static_cast<float*>(out)[at + i] = v[i];
      else
        static_cast<uint16_t*>(out)[at + i] = (uint16_t)f32_to_bf16(v[i]);
    }
}

// A tile's place: its rows, and its part of K.
struct Fp4Place {
  int64_t n0, m0;
  int nrows, mrows, split, tile, kb0, kblocks;
};

// BN x BM tiles, one or several after the other for a workgroup: the last
// blocks of a tile bring the first ones of the next, so that only its stores
// stand between two tiles' products.  In LDS an operand's 16-row fragments
// follow each other, their rows in 16-byte chunks (fp4_slot).  W is the MFMA's A
// operand (D rows n), its rows interleaved over a wave's fragments so that the
// values of a lane are consecutive n.
//
// Bound by power: the matrix instructions alone, on random codes, reach 6.7
// PFLOP/s on the card (8.8 on zeros), and with the copies and the LDS reads
// that feed them 4.6 (8192^3, 239 us).  16384 x 5760 x 2880: 167 us, 3.3
// PFLOP/s, with K padded by 7%, six rounds of tiles that are 5.75, and 189 MB of
// results; a tile after another on its own (188 us) took 142 without its
// stores, 120 without its copies, 101 without the matrix instructions, 66
// without any of the three: their times add up, a slower clock behind them.
// 2047 x 5760 x 2880: 28 us, 2.4 PFLOP/s, one round.  The larger a wave's part of
// a tile the fewer LDS reads for a product, so 256 x 256 wins where there are
// rounds of it.  Tried without gain: stages of 64 bytes a row, four waves with
// 128 x 128 each, 96-column waves, rows of X at an odd pitch, stores of whole
// KB or past the caches, workgroups that start one after the other.  In bf16:
// 2048 x 2880 x 5760, 62 us, 1.1 PFLOP/s (the library's 8192^3: 1.35).
template <class T, bool F32, bool PARTS>
__global__ __launch_bounds__(64 * T::NW) void fp4_gemm_kernel(Fp4Gemm g, int64_t xp, int ntiles, int mtiles, int first,
                                                              int count, int splits) {
  constexpr int FN = T::FN, FM = T::FM, WM = T::WM, NST = T::NST;
  constexpr bool SEVERAL = T::SEVERAL && !PARTS;
  __shared__ __align__(1024) uint8_t lds[NST * T::STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int r = lane & 15, q = lane >> 4;
  Fp4Wave v;
  v.wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  v.lds = (uint32_t)(uintptr_t)(lptr_t)lds;
  const int wn = v.wave / WM, wm = v.wave % WM;
  v.woff = (wn * 16 * FN + r) * 128;
  v.xoff = (T::BN + wm * 16 * FM + r) * 128;
  v.s0 = fp4_slot(r, 2 * q) << 4;
  v.sxoff = T::SX + q * 2 * T::BM + 2 * (wm * 16 * FM + r * FM);
  v.swoff = T::SW + q * 2 * T::BN + 2 * (wn * 16 * FN + w_row(r) * FN);
  const int all = (int)(xp / 128);   // X's rows are whole K blocks
  // Sets out the copies of item `item` (with splits, every tile's parts one
  // after the other).
  auto place = [&](int item) {
    Fp4Place w;
    w.split = PARTS ? item % splits : 0;
    w.tile = PARTS ? item / splits : item;
    int nt, mt;
    tile_at(first + w.tile, ntiles, mtiles, nt, mt);
    w.n0 = (int64_t)nt * T::BN;
    w.m0 = (int64_t)mt * T::BM;
    w.kb0 = PARTS ? (int)((int64_t)all * w.split / splits) : 0;
    w.kblocks = PARTS ? (int)((int64_t)all * (w.split + 1) / splits) - w.kb0 : all;
    // copies: lane l brings slot l % 8 of row l / 8 of a piece.  Rows past the
    // matrix repeat its last row (their results are dropped).
    w.nrows = (int)min((int64_t)T::BN, g.N - w.n0);
    w.mrows = (int)min((int64_t)T::BM, g.M - w.m0);
    v.rw = buffer_of(g.w + w.n0 * g.wp, w.nrows * g.wp);
    v.rx = buffer_of(g.x + w.m0 * xp, w.mrows * xp);
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const int p = v.wave * T::LOADS + i;
      const bool isw = p < T::BN / 8;
      const int at = 8 * (isw ? p : p - T::BN / 8) + (lane >> 3);   // LDS row of the operand
      const int fr = at & 15, f = at >> 4;                          // its fragment row and fragment
      const int row = isw ? f / FN * 16 * FN + w_row(fr) * FN + f % FN : f / FM * 16 * FM + fr * FM + f % FM;
      v.off[i] = (uint32_t)min(row, (isw ? w.nrows : w.mrows) - 1) * (uint32_t)(isw ? g.wp : xp) +
                 (uint32_t)w.kb0 * 128 + (fp4_slot(fr, lane & 7) << 4);
    }
    if (T::FP4) {
      // scale copies: 16 bytes a lane, 8 rows' pairs; rows past the scales
      // repeat their last 16 bytes
      const int c = v.wave % (T::CX + T::CW);   // uniform
      const bool isw = c >= T::CX;
      const int rows = isw ? T::BN : T::BM;
      const int64_t srows = fp4_scale_rows(isw ? g.N : g.M), at = isw ? w.n0 : w.m0;
      const int chunk = min(64 * (isw ? c - T::CX : c) + lane, rows / 2 - 1);
      const int p = chunk / (rows / 8), o = 16 * (chunk % (rows / 8));
      const int left = (int)min((srows - at) * 2, (int64_t)2 * rows);   // bytes of a pair's rows, >= 32
      v.soff = (uint32_t)(p * 2 * srows) + (uint32_t)min(o, left - 16);
      v.sstep = (uint32_t)(8 * srows);
      v.sdst = T::SX + c * 1024;
      v.rs = buffer_of((isw ? g.sw : g.sx) + w.kb0 * 8 * srows + at * 2,
                       (w.kblocks - 1) * 8 * srows + 6 * srows + left);
    }
    return w;
  };
  // XCD x takes a contiguous range of the items, its workgroups one after the
  // other of it
  int item, end, step;
  {
    const int L = count * splits, b = blockIdx.x, x = b & 7;
    const int base = L >> 3, extra = L & 7;
    item = x * base + min(x, extra) + (b >> 3);
    end = (x + 1) * base + min(x + 1, extra);
    step = ((int)gridDim.x - x + 7) >> 3;
  }
  Fp4Place w = place(item), ahead = w;   // what is multiplied, what is copied
  int left = w.kblocks, next = NST;        // blocks of w to come; the next block to copy
#pragma unroll
  for (int k = 0; k < NST; ++k)
    if (SEVERAL || k < left) {
#pragma unroll
      for (int i = 0; i < T::COPIES; ++i) fp4_copy_piece<T>(v, k * T::STAGE, min(k, left - 1), i);
    }
  ring_wait<T>((SEVERAL ? NST : min(NST, left)) - 1);
  barrier_only();
  Fp4Frags<T> f;
  if (T::FP4) f.c = fp4_scales<T>(v, lds);
  fp4_read_b<T>(v, lds, 0, f);
#pragma unroll
  for (int i = 0; i < T::AHEAD; ++i) fp4_read_a<T>(v, lds, i, f);
  int st = 0, there = 0;
  f32x4 acc[FN][FM];
  auto zero = [&]() {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  zero();
  if constexpr (!SEVERAL) {
    // the last blocks read a stage ahead that holds nothing new
    for (; left > NST; --left) fp4_block<T, true>(v, next++, 0, lds, st, f, acc);
    for (; left > 1; --left) fp4_block<T, false>(v, 0, 0, lds, st, f, acc);
  }
  for (;;) {
    if (SEVERAL && next >= ahead.kblocks) {   // the copies go on with the next tile
      item += step;
      next = 0;
      if (item < end) {
        ahead = place(item);
      } else {   // or with nothing: all of an empty buffer is past its end, and no memory is read
        ahead.kblocks = 1 << 30;
        v.rw[2] = v.rx[2] = v.rs[2] = 0;
      }
    }
    fp4_block<T, SEVERAL>(v, next++, there, lds, st, f, acc);
    there = 0;
    if (--left) continue;
    const Fp4Place done = w;
    const bool more = SEVERAL && item < end;   // whole tiles: the host gives several only K of more blocks than stages
    const int64_t nw0 = done.n0 + wn * 16 * FN;
    if constexpr (PARTS) {   // the tile's part, the rows that exist, as [BM][BN] fp32
      float* part = g.part + ((int64_t)done.split * count + done.tile) * (T::BN * T::BM);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        if (wm * 16 * FM + r * FM + j >= done.mrows) break;
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
      break;
    }
    // The copies of the next tile's second block come before the stores: a
    // wait for them later would be one for the stores.
    if (more) __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t n = nw0 + (4 * t + q) * FN;
      float bias[FN];   // once for the lane's FM columns
      fp4_bias<FN>(g.bias, n, g.N, bias);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        float o[FN];
#pragma unroll
        for (int i = 0; i < FN; ++i) o[i] = acc[i][j][t] + bias[i];
        fp4_store<FN, F32>(g.out, g.M, g.N, done.m0 + wm * 16 * FM + r * FM + j, n, o);
      }
    }
    if (!more) break;
    zero();
    w = ahead;
    left = w.kblocks;
    there = 1;
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));   // no copy outlives the workgroup
}

// Few rows: a workgroup takes 16 rows of W and its waves split K in units of
// 128; every wave streams its part of W straight into fragments (lane (r, q):
// block 4 u + q of row r), and the partial sums meet in LDS in wave order.
// Bound by the latency of a launch with a trip to HBM in it: 16 x 5760 x 2880
// in 6.8 us (one row 5.6, of them an empty launch 2).
constexpr int FK_NW = 8, FK_CH = 3;   // waves; units in flight per wave

struct SkinnyW4 {
  u32x4 c[FK_CH];
  uint32_t s[FK_CH];
};
// W's units c0 .. of this lane's row (past u1 - 1 that unit again, not
// multiplied; chunks past the row's end its last chunk, which meets zeros).
__device__ __forceinline__ void skinny4_load(const uint8_t* w, int64_t wp, const uint8_t* sw, int64_t srows, int q,
                                             int c0, int u1, SkinnyW4& f) {
#pragma unroll
  for (int i = 0; i < FK_CH; ++i) {
    const int64_t u = min(c0 + i, u1 - 1);
    f.c[i] = gload16(w + min(u * 64 + 16 * q, wp - 16));
    f.s[i] = sw[(u >> 1) * 8 * srows + (2 * (u & 1) + (q >> 1)) * 2 * srows + (q & 1)];
  }
}
// The waves' sums in their order, plus the bias, by the first wave.  Lane l
// holds D rows 4 (l / 16) .. + 3 (n) of column l % 16 (m).
template <bool F32>
__device__ __forceinline__ void skinny4_store(const Fp4Gemm& g, f32x4 (*part)[64], int64_t n0, int wave, int lane) {
  if (wave) return;
  f32x4 sum = part[0][lane];
#pragma unroll
  for (int u = 1; u < FK_NW; ++u) sum += part[u][lane];
  const int64_t n = n0 + 4 * (lane >> 4);
  float bias[4];
  fp4_bias<4>(g.bias, n, g.N, bias);
  const float o[4] = {sum[0] + bias[0], sum[1] + bias[1], sum[2] + bias[2], sum[3] + bias[3]};
  fp4_store<4, F32>(g.out, g.M, g.N, lane & 15, n, o);
}

// 4-bit X, up to 16 rows.
template <bool F32>
__global__ __launch_bounds__(64 * FK_NW) void fp4_skinny_kernel(Fp4Gemm g) {
  __shared__ f32x4 part[FK_NW][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t xp = fp4_pitch(g.K);
  const int units = (int)((g.K + 127) / 128);
  const int u0 = wave * units / FK_NW, u1 = (wave + 1) * units / FK_NW;
  const int64_t n = min(n0 + r, g.N - 1), m = min((int64_t)r, g.M - 1);
  const int64_t srw = fp4_scale_rows(g.N), srx = fp4_scale_rows(g.M);
  const uint8_t *w = g.w + n * g.wp, *x = g.x + m * xp;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = u0; c0 < u1; c0 += FK_CH) {
    SkinnyW4 fx, fw;
    skinny4_load(x, xp, g.sx + 2 * m, srx, q, c0, u1, fx);
    skinny4_load(w, g.wp, g.sw + 2 * n, srw, q, c0, u1, fw);
#pragma unroll
    for (int i = 0; i < FK_CH; ++i)
      if (c0 + i < u1)
        acc = fp4_mfma<0, 0>(fp4_operand(fw.c[i]), fp4_operand(fx.c[i]), acc, (int)fw.s[i], (int)fx.s[i]);
  }
  part[wave][lane] = acc;
  __syncthreads();
  skinny4_store<F32>(g, part, n0, wave, lane);
}

// bf16 X of up to 16 rows, rounded here: every workgroup rounds all of X into
// LDS (4 lanes a block) while its first W loads are under way.  LDS unit u of
// row m is 64 bytes at (u M + m) * 64, its four scales at (u M + m) * 4.  One
// row, 5760 x 2880: 4.7 us (1.9 TB/s of W), an empty launch 2.
constexpr int FUSED4_BYTES = 20480, FUSED4_ROUNDS = FUSED4_BYTES / 4 / (64 * FK_NW);

template <bool F32, bool WHOLE>
__global__ __launch_bounds__(64 * FK_NW) void fp4_fused_kernel(Fp4Gemm g, const uint16_t* __restrict__ xb) {
  __shared__ __align__(16) uint8_t xs[FUSED4_BYTES];
  __shared__ uint8_t sxs[FUSED4_BYTES / 16];
  __shared__ f32x4 part[FK_NW][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int M = (int)g.M, units = (int)((g.K + 127) / 128);
  const int u0 = wave * units / FK_NW, u1 = (wave + 1) * units / FK_NW;
  const int64_t n = min(n0 + r, g.N - 1);
  const int64_t srw = fp4_scale_rows(g.N);
  const uint8_t* w = g.w + n * g.wp;
  // the 8 elements of X of each of this thread's turns, then W's first units
  const int groups = M * units * 16, turns = (groups + 64 * FK_NW - 1) / (64 * FK_NW);   // turns <= FUSED4_ROUNDS
  u32x4 xv[FUSED4_ROUNDS];
#pragma unroll
  for (int i = 0; i < FUSED4_ROUNDS; ++i) {
    if (i < turns) {
      const int id = min(tid + i * 64 * FK_NW, groups - 1), m = id / (units * 16), k0 = 8 * (id % (units * 16));
      xv[i] = bf16x8_at<WHOLE>(xb, m * g.K + k0, g.K - k0);
    }
  }
  SkinnyW4 f;
  if (u0 < u1) skinny4_load(w, g.wp, g.sw + 2 * n, srw, q, u0, u1, f);
#pragma unroll
  for (int i = 0; i < FUSED4_ROUNDS; ++i) {
    const int id = tid + i * 64 * FK_NW, m = id / (units * 16), l = id % (units * 16);
    if (id < groups) {   // whole blocks: the four lanes of one go together
      uint32_t s;
      const uint32_t c = fp4_codes(xv[i], s);
      const int at = (l >> 4) * M + m;   // its unit
      *reinterpret_cast<uint32_t*>(xs + at * 64 + 4 * (l & 15)) = c;
      if ((l & 3) == 0) sxs[at * 4 + ((l >> 2) & 3)] = (uint8_t)s;
    }
  }
  wave_lds_sync();
  barrier_only();   // leaves W's loads under way
  const int m = min(r, M - 1);
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = u0; c0 < u1; c0 += FK_CH) {
    if (c0 > u0) skinny4_load(w, g.wp, g.sw + 2 * n, srw, q, c0, u1, f);
#pragma unroll
    for (int i = 0; i < FK_CH; ++i) {
      if (c0 + i >= u1) continue;
      const int at = (c0 + i) * M + m;
      const u32x4 x = *reinterpret_cast<const u32x4*>(xs + at * 64 + 16 * q);
      acc = fp4_mfma<0, 0>(fp4_operand(f.c[i]), fp4_operand(x), acc, (int)f.s[i], (int)sxs[at * 4 + q]);
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  skinny4_store<F32>(g, part, n0, wave, lane);
}

// ------------------------------------------------------------- input's gradient

// W [N, K] decoded and transposed: 64 rows x 128 elements a workgroup, a thread
// two rows x 8 elements, pairs of rows through LDS as words.  Bound by HBM: 5760
// x 2880 in 12 us (3.5 TB/s; with 256 elements a workgroup, whole lines both
// ways, 15).
__global__ __launch_bounds__(256) void fp4_dequant_t_kernel(const uint8_t* __restrict__ w, int64_t wp,
                                                            const uint8_t* __restrict__ sw, int64_t N, int64_t K,
                                                            int ktiles, int64_t np, uint16_t* __restrict__ wt) {
  __shared__ uint32_t t[128][33];
  const int tid = threadIdx.x;
  const int64_t n0 = (int64_t)(blockIdx.x / ktiles) * 64, k0 = (int64_t)(blockIdx.x % ktiles) * 128;
  const int64_t srows = fp4_scale_rows(N);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int pair = tid & 31, grp = 8 * p + (tid >> 5);   // grp: 8 elements
    const int64_t k = k0 + 8 * grp, b = k >> 5;
    u32x4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = n0 + 2 * pair + h;
      v[h] = u32x4{0u, 0u, 0u, 0u};
      if (n < N && k < K) {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(w + n * wp + k / 2);
        const uint32_t s = sw[((b >> 3) * 4 + ((b >> 1) & 3)) * srows * 2 + 2 * n + (b & 1)];
        v[h] = dequant8_bf16(c, scale_operand(s));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[8 * grp + 2 * i][pair] = (v[0][i] & 0xFFFFu) | (v[1][i] << 16);
      t[8 * grp + 2 * i + 1][pair] = (v[0][i] >> 16) | (v[1][i] & 0xFFFF0000u);
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int k = 32 * p + (tid >> 3), c = 4 * (tid & 7);
    if (k0 + k < K)
      *reinterpret_cast<u32x4*>(wt + (k0 + k) * np + n0 + 2 * c) = u32x4{t[k][c], t[k][c + 1], t[k][c + 2], t[k][c + 3]};
  }
}

// Few rows of dY: W's codes straight into fragments, with no copy in between.
// The sum over n may take its terms in any order and columns of the result may
// be in any: lane (r, q) reads a word of codes, columns 8 r .. + 7, of each of
// the eight rows of W at 8 q, and the values of column 8 r + t of those rows are its
// part of fragment t; dY's rows are the other operand.  A workgroup has 128 columns,
// 16 rows of dY and a part of n, which its waves share in units of 32; their sums
// meet in LDS and those of the parts in another launch, in their order.  Bound
// by the loads' round trips: a wave asks for its next unit behind a unit's
// products and decodes it at once, and a CU has one workgroup, two waves a SIMD.
// By counters (W 5760 x 2880, 256 rows, 26.6 us) a wave waits for 53% of its time and
// issues vector instructions in 23%, the matrix cores are busy 17%, and HBM gives 1.0
// TB/s (16 rows: 61%, 19%, 4%, 0.7 TB/s).  Both launches, us (by way of the
// copy): 1 row 9.0 (24), 16 rows 10 (28), 64 rows 15 (28), 256 rows 33 (48), 512
// rows 48 (59).  Units read two and more ahead brought no gain.
template <int MT>
struct DxUnit {
  uint32_t w[8];
  u32x4 s, y[MT];
};
constexpr int DX_WAVES = 8;
template <int MT, bool WHOLE>
__global__ __launch_bounds__(64 * DX_WAVES) void fp4_dx_few_kernel(Fp4Gemm g, const uint16_t* __restrict__ dy,
                                                                   int ktiles, int splits) {
  __shared__ f32x4 red[DX_WAVES / 2][8 * MT][64];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // XCD x takes a contiguous range of the items: neighbours of 128 columns share
  // lines of W
  int item;
  {
    const int L = (int)gridDim.x, x = blockIdx.x & 7;
    item = x * (L >> 3) + min(x, L & 7) + (blockIdx.x >> 3);
  }
  const int split = item / ktiles;
  const int64_t k = (int64_t)(item % ktiles) * 128 + 8 * r, m0 = (int64_t)blockIdx.y * 16 * MT;
  const int64_t N = g.N, srows = fp4_scale_rows(N), units = (N + 31) / 32;
  const int u1 = (int)(units * (split + 1) / splits);
  const int b = (int)(k >> 5);
  // columns past K are computed as the first ones and not stored
  const uint8_t* w = g.w + (k < g.K ? k / 2 : 0);
  const uint8_t* sw = g.sw + (k < g.K ? ((int64_t)(b >> 3) * 4 + ((b >> 1) & 3)) * srows * 2 : 0);
  const int par = 8 * (b & 1);   // the block's byte of a pair
  auto load = [&](int u, DxUnit<MT>& f) {
    const int64_t n = 32 * (int64_t)u + 8 * q;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f.w[j] = 0;   // rows past N have no codes
      if (n + j < N) f.w[j] = *reinterpret_cast<const uint32_t*>(w + (n + j) * g.wp);
    }
    f.s = u32x4{0u, 0u, 0u, 0u};
    if (n < N) f.s = *reinterpret_cast<const u32x4*>(sw + 2 * n);
    if (!WHOLE) {   // past the rows any bytes may stand, NaN too
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j >= N) f.s[j >> 1] &= j & 1 ? 0xFFFFu : 0u;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) f.y[i] = bf16x8_at<WHOLE>(dy, min(m0 + 16 * i + r, g.M - 1) * N + n, N - n);
  };
  f32x4 acc[MT][8];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  DxUnit<MT> f;
  int u = (int)(units * split / splits) + wave;
  if (u < u1) load(u, f);
  while (u < u1) {
    u32x4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = dequant8_bf16(f.w[j], scale_operand(f.s[j >> 1] >> (16 * (j & 1) + par) & 255));
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      u32x4 c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = v[2 * j][t >> 1], hi = v[2 * j + 1][t >> 1];
        c[j] = t & 1 ? lo >> 16 | (hi & 0xFFFF0000u) : (lo & 0xFFFFu) | hi << 16;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(f.y[i]), as_bf16x8(c), acc[i][t], 0, 0, 0);
    }
    u += DX_WAVES;
    if (u < u1) load(u, f);
  }
#pragma unroll
  for (int h = DX_WAVES / 2; h >= 1; h /= 2) {
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t) red[wave - h][8 * i + t][lane] = acc[i][t];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t) acc[i][t] += red[wave][8 * i + t][lane];
    }
    __syncthreads();
  }
  if (wave) return;
  void* out = splits > 1 ? static_cast<void*>(g.part + (int64_t)split * g.M * g.K) : g.out;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // D row 4 q + e: a row of dY
      float o[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) o[t] = acc[i][t][e];
      const int64_t m = m0 + 16 * i + 4 * q + e;
      if (splits > 1 || g.out_f32)
        fp4_store<8, true>(out, g.M, g.K, m, k, o);
      else
        fp4_store<8, false>(out, g.M, g.K, m, k, o);
    }
}

// The parts' sum: four elements a thread.
__global__ __launch_bounds__(256) void dx_join_kernel(const float* __restrict__ part, int64_t count, int splits,
                                                      void* __restrict__ out, int out_f32) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (i + 4 <= count) {
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const f32x4 p = *reinterpret_cast<const f32x4_any*>(part + s * count + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += p[e];
    }
  } else {
    for (int s = 0; s < splits; ++s)
      for (int e = 0; e < 3; ++e)
        if (i + e < count) v[e] += part[s * count + i + e];
  }
  if (out_f32)
    fp4_store<4, true>(out, 1, count, 0, i, v);
  else
    fp4_store<4, false>(out, 1, count, 0, i, v);
}

// Rows of dY at a pitch of whole K blocks and 16-byte alignment, which the
// product's copies need; left out where dY has them.
__global__ __launch_bounds__(256) void bf16_pad_kernel(const uint16_t* __restrict__ x, int64_t K, int64_t kp,
                                                       int64_t total, uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // 8 elements of the result
  if (i >= total) return;
  const int64_t row = i / (kp / 8), k = i % (kp / 8) * 8;
  reinterpret_cast<u32x4*>(out)[i] = bf16x8_at<false>(x, row * K + k, K - k);
}

// ------------------------------------------------------------------ launchers

hipError_t launch_fp4_quantize(const void* x, int x_f32, int64_t rows, int64_t K, uint8_t* codes, uint8_t* scales,
                               hipStream_t s) {
  const int64_t kb = fp4_kblocks(K);
  const dim3 grid((unsigned)(kb * ((rows + 15) / 16)));
  const bool whole = K % 8 == 0;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, x, rows, K, fp4_pitch(K), fp4_scale_rows(rows), (int)kb, codes,
                       scales);
    return hipGetLastError();
  };
  if (x_f32) return whole ? launch(fp4_rows_kernel<true, true>) : launch(fp4_rows_kernel<true, false>);
  return whole ? launch(fp4_rows_kernel<false, true>) : launch(fp4_rows_kernel<false, false>);
}

hipError_t launch_fp4_scales(const uint8_t* scales, int64_t rows, int64_t K, uint8_t* ordered, hipStream_t s) {
  const int64_t total = fp4_scale_bytes(rows, K) / 2;
  hipLaunchKernelGGL(fp4_scales_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, scales, rows, K / 32,
                     fp4_scale_rows(rows), total, ordered);
  return hipGetLastError();
}

hipError_t launch_fp4_dequant_t(const uint8_t* w, int64_t wp, const uint8_t* sw, int64_t N, int64_t K, uint16_t* wt,
                                hipStream_t s) {
  const int64_t kt = (K + 127) / 128, nt = (N + 63) / 64;
  hipLaunchKernelGGL(fp4_dequant_t_kernel, dim3((unsigned)(kt * nt)), dim3(256), 0, s, w, wp, sw, N, K, (int)kt,
                     fp8_up(N, 64), wt);
  return hipGetLastError();
}

hipError_t launch_bf16_pad(const uint16_t* x, int64_t rows, int64_t K, uint16_t* out, hipStream_t s) {
  const int64_t kp = fp8_up(K, 64), total = rows * kp / 8;
  hipLaunchKernelGGL(bf16_pad_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, x, K, kp, total, out);
  return hipGetLastError();
}

// The tiles' times (GemmShape), for bf16 and for fp32 results, fitted to launches
// of 32 to 16384 rows by 5760 x 2880, 2880 x 5760, 8192 x 1024, 1024 x 8192, 4096
// x 4096, 512 x 512 and 700 x 512 whose W comes from HBM.  The choice is 1% slower
// on average than the best tile, at most 12%.  In 4 bits (us; 5760 x 2880):
//   rows       64    256    512   1024   2047   4096  16384
//   256 x 256  23.6  25.8  26.2   27.0   28.0   52.0    189
//   256 x 192  21.6  23.0  23.4   24.2   26.7   49.0    183
//   128 x 192  15.6  17.4  17.9   30.8   32.7   60.5    226
//   128 x 128  13.6  14.7  15.2   20.0   31.6   53.6    242   two stages, two workgroups on a CU
//   128 x 128  11.6  12.8  13.2   22.8   33.2   61.1    266   three stages, one
//   64 x 128    8.4   9.2  13.4   20.0   34.8   64.4    268
//   64 x 64     7.0   9.8  14.4   24.6   44.1   79.6    331
//   32 x 64     6.3  10.2  16.8   30.5   56.2    107    450
//   32 x 32     6.4  13.3  20.9   37.0   68.0    130    522
static constexpr GemmShape FP4_SHAPE[] = {
    {256, 256, 1, {1.23f, 1.05f}, {1.47f, 1.38f}, {10.8f, 17.5f}},
    {256, 192, 1, {1.26f, 1.10f}, {1.26f, 1.12f}, {7.5f, 13.0f}},
    {128, 192, 1, {0.85f, 0.82f}, {0.75f, 0.79f}, {6.2f, 7.0f}},
    {128, 128, 2, {0.62f, 0.58f}, {0.51f, 0.63f}, {6.6f, 7.3f}},
    {128, 128, 1, {0.54f, 0.50f}, {0.46f, 0.55f}, {5.4f, 6.4f}},
    {64, 128, 2, {0.33f, 0.33f}, {0.29f, 0.36f}, {4.7f, 4.9f}},
    {64, 64, 2, {0.28f, 0.27f}, {0.20f, 0.23f}, {3.2f, 3.3f}},
    {32, 64, 3, {0.25f, 0.26f}, {0.14f, 0.16f}, {2.9f, 2.8f}},
    {32, 32, 3, {0.28f, 0.25f}, {0.08f, 0.09f}, {2.1f, 2.1f}},
};
// The same in bf16, the input's gradient's product.
static constexpr GemmShape BF16_SHAPE[] = {
    {256, 256, 1, {1.14f, 1.14f}, {1.21f, 1.21f}, {13.1f, 16.0f}},
    {256, 192, 1, {0.92f, 0.92f}, {0.94f, 0.94f}, {12.3f, 15.0f}},
    {128, 192, 1, {0.55f, 0.55f}, {0.55f, 0.55f}, {10.3f, 11.0f}},
    {128, 128, 2, {0.52f, 0.52f}, {0.36f, 0.36f}, {12.0f, 13.0f}},
    {128, 128, 1, {0.41f, 0.41f}, {0.37f, 0.37f}, {9.3f, 10.0f}},
    {64, 128, 2, {0.24f, 0.24f}, {0.23f, 0.23f}, {9.3f, 9.5f}},
    {64, 64, 2, {0.18f, 0.18f}, {0.14f, 0.14f}, {6.7f, 6.8f}},
    {32, 64, 3, {0.15f, 0.15f}, {0.11f, 0.11f}, {4.8f, 4.9f}},
    {32, 32, 4, {0.16f, 0.16f}, {0.07f, 0.07f}, {2.9f, 2.9f}},
};
constexpr int GEMM_SHAPES = (int)(sizeof(FP4_SHAPE) / sizeof(FP4_SHAPE[0]));

static GemmPlan fp4_plan(int64_t M, int64_t N, int64_t K, bool f32) {
  if (M <= 16 && N >= 1024) return {-1, 0, 0, 1, 0, 0};
  return gemm_plan(FP4_SHAPE, GEMM_SHAPES, M, N, fp4_kblocks(K), f32);
}
static GemmPlan bf16_plan(int64_t M, int64_t N, int64_t K, bool f32) {
  return gemm_plan(BF16_SHAPE, GEMM_SHAPES, M, N, K / 64, f32);
}
size_t fp4_part_bytes(int64_t M, int64_t N, int64_t K, int out_f32) {
  return gemm_part_bytes(fp4_plan(M, N, K, out_f32 != 0));
}
size_t bf16_part_bytes(int64_t M, int64_t N, int64_t K, int out_f32) {
  return gemm_part_bytes(bf16_plan(M, N, K, out_f32 != 0));
}

// Tiles first .. first + count - 1, in `splits` parts of K.
template <class T>
static hipError_t gemm_tiles(const Fp4Gemm& g, int64_t xp, int first, int count, int splits, hipStream_t s) {
  const int nt = (int)((g.N + T::BN - 1) / T::BN), mt = (int)((g.M + T::BM - 1) / T::BM);
  // As many workgroups as the CUs hold take several tiles each, where a tile has
  // blocks of its own beside those that its neighbours' copies touch.
  const int64_t items = (int64_t)count * splits, held = 256 * (160 * 1024 / (T::NST * T::STAGE));
  const bool several = T::SEVERAL && splits == 1 && items > held && xp / 128 > T::NST;
  const dim3 grid((unsigned)(several ? held : items)), block(64 * T::NW);
  if (splits > 1)
    hipLaunchKernelGGL((fp4_gemm_kernel<T, true, true>), grid, block, 0, s, g, xp, nt, mt, first, count, splits);
  else if (g.out_f32)
    hipLaunchKernelGGL((fp4_gemm_kernel<T, true, false>), grid, block, 0, s, g, xp, nt, mt, first, count, splits);
  else
    hipLaunchKernelGGL((fp4_gemm_kernel<T, false, false>), grid, block, 0, s, g, xp, nt, mt, first, count, splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  Fp8Gemm j{};
  j.M = g.M;
  j.N = g.N;
  j.K = g.K;
  j.bias = g.bias;
  j.out = g.out;
  j.out_f32 = g.out_f32;
  j.part = g.part;
  return launch_gemm_join(j, T::BN, T::BM, first, count, splits, s);
}
template <class T>
static hipError_t gemm(const Fp4Gemm& g, int64_t xp, const GemmPlan& p, hipStream_t s) {
  if (p.rest && !g.part) return hipErrorInvalidValue;
  if (p.whole) {
    const hipError_t e = gemm_tiles<T>(g, xp, 0, p.whole, 1, s);
    if (e != hipSuccess) return e;
  }
  return p.rest ? gemm_tiles<T>(g, xp, p.whole, p.rest, p.splits, s) : hipSuccess;
}
template <bool FP4>
static hipError_t gemm_of(const Fp4Gemm& g, int64_t xp, const GemmPlan& p, hipStream_t s) {
  switch (p.tile) {
    case 0: return gemm<Fp4Tile<2, 4, 8, 4, 2, FP4>>(g, xp, p, s);
    case 1: return gemm<Fp4Tile<2, 4, 8, 3, 2, FP4>>(g, xp, p, s);
    case 2: return gemm<Fp4Tile<2, 4, 4, 3, FP4 ? 3 : 4, FP4>>(g, xp, p, s);
    case 3: return gemm<Fp4Tile<2, 2, 4, 4, 2, FP4>>(g, xp, p, s);
    case 4: return gemm<Fp4Tile<2, 2, 4, 4, 3, FP4>>(g, xp, p, s);
    case 5: return gemm<Fp4Tile<1, 4, 4, 2, 3, FP4>>(g, xp, p, s);
    case 6: return gemm<Fp4Tile<1, 4, 4, 1, 4, FP4>>(g, xp, p, s);
    case 7: return gemm<Fp4Tile<1, 4, 2, 1, FP4 ? 3 : 4, FP4>>(g, xp, p, s);
    default: return gemm<Fp4Tile<1, 2, 2, 1, 4, FP4>>(g, xp, p, s);
  }
}

hipError_t launch_fp4_gemm(const Fp4Gemm& g, hipStream_t s) {
  const GemmPlan p = fp4_plan(g.M, g.N, g.K, g.out_f32 != 0);
  if (p.tile >= 0) return gemm_of<true>(g, fp4_pitch(g.K), p, s);
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * FK_NW);
  if (g.out_f32)
    hipLaunchKernelGGL(fp4_skinny_kernel<true>, grid, block, 0, s, g);
  else
    hipLaunchKernelGGL(fp4_skinny_kernel<false>, grid, block, 0, s, g);
  return hipGetLastError();
}

hipError_t launch_bf16_gemm(const Fp4Gemm& g, hipStream_t s) {
  if (g.K % 64) return hipErrorInvalidValue;
  Fp4Gemm b = g;
  b.wp = 2 * g.K;
  return gemm_of<false>(b, 2 * g.K, bf16_plan(g.M, g.N, g.K, g.out_f32 != 0), s);
}

// The gradient of few rows (above): rows of dY of a workgroup, parts of n and
// time, which is `c` us, `round` for each round of 256 workgroups, and in it `unit` for
// each of a wave's units of n one after the other (`even` or `odd` more where dY's
// rows are at such elements, not at eighths); the join of the parts has its own launch.
// Fitted, like the copy's way below, to both ways' times at 806 sizes of 16 to 1024
// rows, W from HBM of 64 to 12000 rows and columns, every kind of alignment.
struct DxPlan {
  int mt, splits;
  float us;
};
static DxPlan dx_plan(int64_t M, int64_t N, int64_t K) {
  static constexpr struct {
    int mt;
    float unit, even, odd, round, c;
  } SHAPE[] = {{1, 0.81f, 0.09f, 0.19f, 0.42f, 3.3f},
               {2, 1.125f, 0.20f, 0.54f, 2.5f, 2.35f},
               {4, 1.43f, 0.32f, 1.41f, 5.9f, 1.45f}};
  const int64_t units = (N + 31) / 32, most = (units + DX_WAVES - 1) / DX_WAVES;
  DxPlan best{0, 0, 0.0f};
  for (const auto& t : SHAPE) {
    const int64_t items = ((K + 127) / 128) * ((M + 16 * t.mt - 1) / (16 * t.mt));
    const int64_t fill = 256 / items < 1 ? 1 : 256 / items, splits = fill < most ? fill : most;
    const float unit = t.unit + (N % 2 ? t.odd : N % 8 ? t.even : 0.0f);
    float us = t.c + (float)((items * splits + 255) / 256) * (unit * (float)((most + splits - 1) / splits) + t.round);
    if (splits > 1) us += 2.3f + 0.105f * (float)splits + (float)(splits * M * K) * 1.8e-6f;
    if (best.mt == 0 || us < best.us) best = {t.mt, (int)splits, us};
  }
  return best;
}
// By way of the copy: its product, the copy, and dY's padding where it is needed.
static float dx_copy_us(int64_t M, int64_t N, int64_t K, bool f32) {
  const int64_t np = fp8_up(N, 64);
  float us = 0.97f * bf16_plan(M, K, np, f32).us + 3.1f + (float)(np * K) * 0.86e-6f;
  if (N != np) us += 1.95f + (float)(M * np) * 1.9e-6f;
  return us;
}
// At 544 sizes beside the fitted ones the choice of way and workgroup is 0.9%
// slower on average than the best of the four, over 5% slower at 39 of them and 38%
// at the worst (986 x 256 x 5664, 23 us for 17).  5760 x 2880, from the codes and by way
// of the copy: 512 rows 48 and 59 us, 768 rows 77 and 66.  Beyond 1024 rows the copy is
// always made: at 2048 rows of 5760 x 2880 84 us for 120, but up to twice as slow
// while W is small (1405 rows, 3104 x 96: 23.5 for 11.7).
bool fp4_dx_few(int64_t M, int64_t N, int64_t K, int out_f32) {
  return M <= 1024 && dx_plan(M, N, K).us < dx_copy_us(M, N, K, out_f32 != 0);
}
size_t fp4_dx_few_bytes(int64_t M, int64_t N, int64_t K) {
  const int s = dx_plan(M, N, K).splits;
  return s > 1 ? (size_t)s * M * K * sizeof(float) : 0;
}
hipError_t launch_fp4_dx_few(const Fp4Gemm& g, const uint16_t* dy, hipStream_t s) {
  const DxPlan p = dx_plan(g.M, g.N, g.K);
  const int splits = p.splits, ktiles = (int)((g.K + 127) / 128);
  if (splits > 1 && !g.part) return hipErrorInvalidValue;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(ktiles * splits, (unsigned)((g.M + 16 * p.mt - 1) / (16 * p.mt))),
                       dim3(64 * DX_WAVES), 0, s, g, dy, ktiles, splits);
  };
  const bool whole = g.N % 8 == 0;
  if (p.mt == 1)
    whole ? launch(fp4_dx_few_kernel<1, true>) : launch(fp4_dx_few_kernel<1, false>);
  else if (p.mt == 2)
    whole ? launch(fp4_dx_few_kernel<2, true>) : launch(fp4_dx_few_kernel<2, false>);
  else
    whole ? launch(fp4_dx_few_kernel<4, true>) : launch(fp4_dx_few_kernel<4, false>);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t count = g.M * g.K;
  hipLaunchKernelGGL(dx_join_kernel, dim3((unsigned)((count + 1023) / 1024)), dim3(256), 0, s, g.part, count, splits,
                     g.out, g.out_f32);
  return hipGetLastError();
}

// The one-launch form: X's codes fit its LDS, and rounding them in every
// workgroup costs less than a launch of its own (from HBM, us: 5760 x 2880, 4
// rows 6.1 against 7.3, 8 rows 7.9, 7.4; 2880 x 5760, 4 rows 7.0, 7.5; with few
// columns, 512 x 2880, 16 rows 7.8, 7.3).
bool fp4_fused_fits(int64_t M, int64_t N, int64_t K) {
  return M <= 16 && M * ((K + 127) / 128 * 64) <= (N < 1024 ? FUSED4_BYTES : FUSED4_BYTES / 2);
}

hipError_t launch_fp4_fused(const Fp4Gemm& g, const uint16_t* x, hipStream_t s) {
  if (!fp4_fused_fits(g.M, g.N, g.K)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * FK_NW);
  const bool whole = g.K % 8 == 0;
  if (g.out_f32) {
    if (whole)
      hipLaunchKernelGGL((fp4_fused_kernel<true, true>), grid, block, 0, s, g, x);
    else
      hipLaunchKernelGGL((fp4_fused_kernel<true, false>), grid, block, 0, s, g, x);
  } else {
    if (whole)
      hipLaunchKernelGGL((fp4_fused_kernel<false, true>), grid, block, 0, s, g, x);
    else
      hipLaunchKernelGGL((fp4_fused_kernel<false, false>), grid, block, 0, s, g, x);
  }
  return hipGetLastError();
}

}  // namespace mxmoe
