// The router's balance losses with their gradient (gfx950).
//
// Tokens of S ragged sequences, masked ones left out; N_s tokens of sequence s
// count, N in all, S+ sequences have any.  With p the scores divided by their
// sum (softmax, or sigmoid / sum),
//   counts_se  choices of expert e in sequence s
//   P_se       mean of p_e,   f_se = counts_se / (k N_s)
//   balance    mean over the S+ sequences of E sum_e f_se P_se  (1: even)
//   size       mean over the N tokens of logsumexp(logits)^2
//   dlogits_e  = q_e (c_e - sum_j c_j p_j) + b 2 lse softmax_e / N,
//     c_e = a E f_se / (N_s S+),  q = p (softmax) or p (1 - sigmoid)
//
// A token is a row of 16 lanes, four tokens a wave: lane l has the experts 64 j
// + 4 l .. + 3, so a row's sums are four DPP rotations and its loads whole
// 256-byte pieces.  Scores are formed in fp32 relative to the largest of the
// token (of the sigmoids too: logits below -88 keep their ratios), sums over
// a workgroup's tokens in fp32, over workgroups in fp64, in a fixed order.
#include "balance.hpp"
#include "common.hpp"

namespace mxmoe {

template <int ROR>
__device__ __forceinline__ float row_ror(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + ROR, 0xF, 0xF, true));
}
__device__ __forceinline__ float row16_sum(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, row_ror<8>(v));
  v = fmaxf(v, row_ror<4>(v));
  v = fmaxf(v, row_ror<2>(v));
  return fmaxf(v, row_ror<1>(v));
}

// Four elements of a token from expert e on; `fill` past E.
template <bool WIDE>
__device__ __forceinline__ f32x4 four(const float* row, int e, int E, float fill) {
  f32x4 v = {fill, fill, fill, fill};
  if (WIDE) {
    if (e < E) v = *reinterpret_cast<const f32x4*>(row + e);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < E) v[i] = row[e + i];
  }
  return v;
}

// A token's normalised scores p and softmax (the same without SIG), its
// logsumexp and, with SIG, 1 - sigmoid of each logit.  A token of -inf alone
// has p, softmax and logsumexp 0.
template <int J, bool SIG>
struct Scores {
  float p[J][4], soft[J][4], rest[J][4];
  float lse;
};
template <int J, bool SIG, bool WIDE>
__device__ __forceinline__ void scores(const float* row, int E, int l, Scores<J, SIG>& s) {
  constexpr float INF = __builtin_inff();
  f32x4 x[J];
  float m = -INF;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    x[j] = four<WIDE>(row, 64 * j + 4 * l, E, -INF);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, x[j][i]);
  }
  m = row16_max(m);
  if (m == -INF) m = 0.0f;
  float sum = 0.0f, total = 0.0f;
  const float top = fminf(m, 0.0f);   // of min(logit, 0)
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = x[j][i];
      s.soft[j][i] = expf(v - m);
      sum += s.soft[j][i];
      if (SIG) {
        const float a = expf(-fabsf(v)), r = 1.0f / (1.0f + a);
        s.p[j][i] = expf(fminf(v, 0.0f) - top) * r;   // a NaN is in r
        s.rest[j][i] = v >= 0.0f ? a * r : r;
        total += s.p[j][i];
      }
    }
  sum = row16_sum(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  s.lse = sum == 0.0f ? 0.0f : m + logf(sum);
  float div = inv;
  if (SIG) {
    total = row16_sum(total);
    div = total == 0.0f ? 0.0f : 1.0f / total;
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s.soft[j][i] *= inv;
      s.p[j][i] = SIG ? s.p[j][i] * div : s.soft[j][i];
    }
}

// A sequence's first token and the one past its last, whatever the offsets hold.
__device__ __forceinline__ int64_t clamped(const BalanceArgs& a, int s) {
  return min(max((int64_t)a.offsets[s], (int64_t)0), a.T);
}
__device__ __forceinline__ int64_t seq_begin(const BalanceArgs& a, int s) { return a.offsets ? clamped(a, s) : 0; }
__device__ __forceinline__ int64_t seq_end(const BalanceArgs& a, int s) { return a.offsets ? clamped(a, s + 1) : a.T; }
// The first sequence that ends behind token t (S: none does).
__device__ __forceinline__ int seq_after(const BalanceArgs& a, int64_t t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_end(a, mid) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

constexpr int BAL_WAVES = 8;               // waves of a workgroup: 32 tokens at a time
constexpr int BAL_ONE = 256;               // tokens of one sequence that one workgroup takes alone

// The forward's scratch: a slot for each part of a sequence that a workgroup
// has.  Workgroup b's part of sequence s is slot b + s: along the tokens
// either grows, so no two parts share one, and a sequence's are side by side.
struct BalanceWs {
  float* p;         // [slots, E] sums of p
  int32_t* c;       // [slots, E] choices
  float* z;         // [slots] sums of lse^2
  int32_t* n;       // [slots] tokens
  double* seq;      // [S, 2] balance of a sequence, sum of lse^2
};

// Partial sums of tokens block * per .. + per - 1, sequence by sequence.  ONE:
// all tokens are one sequence and this workgroup's, which also finishes.
template <int J, bool SIG, bool WIDE, bool ONE>
__global__ __launch_bounds__(64 * BAL_WAVES) void balance_part_kernel(BalanceArgs a, BalanceWs ws, int per) {
  __shared__ float part[BAL_WAVES][256];
  __shared__ int hist[256];
  __shared__ float zpart[BAL_WAVES];
  __shared__ int npart[BAL_WAVES];
  __shared__ double fin[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & 15, row = tid >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * per, t1 = min(t0 + per, a.T);
  for (int s = ONE || !a.offsets ? 0 : seq_after(a, t0); s < a.S; ++s) {
    const int64_t from = seq_begin(a, s), lo = max(from, t0), hi = min(seq_end(a, s), t1);   // uniform
    if (!ONE && from >= t1) break;
    if (!ONE && lo >= hi) continue;   // ONE: a sequence without tokens has its zeros written
    for (int e = tid; e < 256; e += 64 * BAL_WAVES) hist[e] = 0;
    __syncthreads();   // also: the last part's readers are done
    float acc[J][4] = {};
    float z = 0.0f;
    int n = 0;
    for (int64_t t = lo + row; t < hi; t += 4 * BAL_WAVES) {   // a row's 16 lanes go together
      if (a.mask && !a.mask[t]) continue;
      Scores<J, SIG> q;
      scores<J, SIG, WIDE>(a.logits + t * a.E, a.E, l, q);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] += q.p[j][i];
      if (l < a.k) {
        const int e = a.topk_idx[t * a.k + l];
        if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
      }
      z = fmaf(q.lse, q.lse, z);
      ++n;
    }
    // the wave's four rows, then the waves, in order
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[j][i] += __shfl_xor(acc[j][i], 16);
        acc[j][i] += __shfl_xor(acc[j][i], 32);
        if (lane < 16) part[wave][64 * j + 4 * l + i] = acc[j][i];
      }
    z += __shfl_xor(z, 16);
    z += __shfl_xor(z, 32);
    n += __shfl_xor(n, 16);
    n += __shfl_xor(n, 32);
    if (lane == 0) {
      zpart[wave] = z;
      npart[wave] = n;
    }
    __syncthreads();
    float pe = 0.0f, ze = 0.0f;
    int ne = 0;
#pragma unroll
    for (int u = 0; u < BAL_WAVES; ++u) {
      if (tid < 64 * J) pe += part[u][tid];
      ze += zpart[u];
      ne += npart[u];
    }
    if (!ONE) {
      const int64_t slot = (int64_t)blockIdx.x + s;
      if (tid < a.E) {
        ws.p[slot * a.E + tid] = pe;
        ws.c[slot * a.E + tid] = hist[tid];
      }
      if (tid == 0) {
        ws.z[slot] = ze;
        ws.n[slot] = ne;
      }
      continue;
    }
    double w = 0.0;
    if (tid < a.E) {
      const double mean = ne ? (double)pe / ne : 0.0;
      a.counts[tid] = hist[tid];
      a.prob[tid] = (float)mean;
      w = hist[tid] * mean;
    }
    if (wave < 4) {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) w += __shfl_xor(w, d);
      if (lane == 0) fin[wave] = w;
    }
    __syncthreads();
    if (tid == 0) {
      const double div = ne ? (double)ne : 1.0;
      a.tokens[0] = ne;
      a.losses[0] = (float)((fin[0] + fin[1] + fin[2] + fin[3]) * a.E / (a.k * div));
      a.losses[1] = (float)(ze / div);
    }
  }
}

template <class V>
__device__ __forceinline__ V all_sum(V v, V* slots, int waves) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  v = slots[0];
  for (int i = 1; i < waves; ++i) v += slots[i];
  return v;
}

// A sequence per workgroup: its parts' sums.  1024 threads are EP experts by
// slices of the parts.
template <int EP>
__global__ __launch_bounds__(1024) void balance_seq_kernel(BalanceArgs a, BalanceWs ws, int per) {
  constexpr int SL = 1024 / EP;
  __shared__ double sums[1024];
  __shared__ int cs[1024];
  __shared__ double slots[16];
  __shared__ int islots[16];
  const int tid = threadIdx.x, e = tid % EP, sl = tid / EP, s = blockIdx.x;
  const int64_t lo = seq_begin(a, s), hi = seq_end(a, s);
  const int64_t b0 = lo / per, b1 = hi > lo ? (hi - 1) / per + 1 : b0;   // its workgroups
  double p = 0.0;
  int c = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int64_t b = b0 + sl; b < b1; b += SL) {
      p += (double)ws.p[(b + s) * a.E + e];
      c += ws.c[(b + s) * a.E + e];
    }
  }
  double z = 0.0;
  int n = 0;
  for (int64_t b = b0 + tid; b < b1; b += 1024) {
    z += (double)ws.z[b + s];
    n += ws.n[b + s];
  }
  sums[tid] = p;
  cs[tid] = c;
  z = all_sum(z, slots, 16);
  n = all_sum(n, islots, 16);
  const double div = n ? (double)n : 1.0;
  double w = 0.0;
  if (sl == 0 && e < a.E) {
    for (int u = 1; u < SL; ++u) {
      p += sums[u * EP + e];
      c += cs[u * EP + e];
    }
    const double mean = p / div;
    a.counts[(int64_t)s * a.E + e] = c;
    a.prob[(int64_t)s * a.E + e] = (float)mean;
    w = c * mean;
  }
  w = all_sum(w, slots, 16) * a.E / (a.k * div);
  if (tid) return;
  a.tokens[s] = n;
  if (a.S == 1) {
    a.losses[0] = (float)w;
    a.losses[1] = (float)(z / div);
  } else {
    ws.seq[2 * s] = w;
    ws.seq[2 * s + 1] = z;
  }
}

// Both losses from the sequences' own.
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs a, BalanceWs ws) {
  __shared__ double slots[16];
  double w = 0.0, z = 0.0, n = 0.0, some = 0.0;
  for (int s = threadIdx.x; s < a.S; s += 1024) {
    const int t = a.tokens[s];
    w += ws.seq[2 * s];   // 0 without tokens
    z += ws.seq[2 * s + 1];
    n += t;
    some += t > 0;
  }
  w = all_sum(w, slots, 16);
  z = all_sum(z, slots, 16);
  n = all_sum(n, slots, 16);
  some = all_sum(some, slots, 16);
  if (threadIdx.x) return;
  a.losses[0] = (float)(some > 0.0 ? w / some : 0.0);
  a.losses[1] = (float)(n > 0.0 ? z / n : 0.0);
}

// dlogits: 16 tokens at a time in a workgroup, `per` in all.  A row of lanes
// looks its first token's sequence up and walks on from there.
template <int J, bool SIG, bool WIDE>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceArgs a, const float* __restrict__ dlosses,
                                                          const float* __restrict__ add,
                                                          float* __restrict__ dlogits, int per) {
  __shared__ double slots[4];
  const int tid = threadIdx.x, l = tid & 15, row = tid >> 4;
  double all = 0.0, some = 0.0;
  for (int s = tid; s < a.S; s += 256) {
    const int n = a.tokens[s];
    all += n;
    some += n > 0;
  }
  all = all_sum(all, slots, 4);
  some = all_sum(some, slots, 4);
  const float da = dlosses[0] * (float)a.E / (float)a.k, db = all > 0.0 ? 2.0f * dlosses[1] / (float)all : 0.0f;
  const int64_t t0 = (int64_t)blockIdx.x * per + row, t1 = min((int64_t)(blockIdx.x + 1) * per, a.T);
  int s = a.offsets && t0 < t1 ? seq_after(a, t0) : 0;
  for (int64_t t = t0; t < t1; t += 16) {
    while (s < a.S && seq_end(a, s) <= t) ++s;
    const bool live = s < a.S && seq_begin(a, s) <= t && !(a.mask && !a.mask[t]);
    float d[J][4] = {};
    if (live) {
      Scores<J, SIG> q;
      scores<J, SIG, WIDE>(a.logits + t * a.E, a.E, l, q);
      const float n = (float)a.tokens[s], f = n > 0.0f ? da / (n * n * (float)some) : 0.0f;
      const int32_t* counts = a.counts + (int64_t)s * a.E;
      float c[J][4], dot = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 64 * j + 4 * l + i;
          c[j][i] = e < a.E ? f * (float)counts[e] : 0.0f;
          dot = fmaf(c[j][i], q.p[j][i], dot);
        }
      dot = row16_sum(dot);
      const float h = db * q.lse;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g = q.p[j][i] * (c[j][i] - dot);
          d[j][i] = fmaf(h, q.soft[j][i], SIG ? g * q.rest[j][i] : g);
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = 64 * j + 4 * l;
      if (e >= a.E) continue;
      f32x4 v = {d[j][0], d[j][1], d[j][2], d[j][3]};
      if (add) v += four<WIDE>(add + t * a.E, e, a.E, 0.0f);
      float* o = dlogits + t * a.E + e;
      if (WIDE) {
        *reinterpret_cast<f32x4*>(o) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < a.E) o[i] = v[i];
      }
    }
  }
}

// ------------------------------------------------------------------ launchers

// Tokens of a workgroup: 128, or 32 where sequences are shorter than that
// (each is a round of its own); more while workgroups are many, whose parts
// are then read again.
static int balance_per(int64_t T, int S) {
  int per = (int64_t)S * 128 > T && S > 1 ? 32 : 128;
  while (per < 1024 && (T + per - 1) / per > 256) per *= 2;
  return per;
}
static bool balance_one(int64_t T, int S) { return S == 1 && T <= BAL_ONE; }

static size_t balance_layout(int64_t T, int E, int S, void* base, BalanceWs* ws) {
  const int per = balance_per(T, S);
  const size_t slots = (size_t)((T + per - 1) / per) + S;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = p + at;
    at += up(bytes);
    return r;
  };
  BalanceWs w;
  w.seq = reinterpret_cast<double*>(take((size_t)S * 16));
  w.p = reinterpret_cast<float*>(take(slots * E * 4));
  w.c = reinterpret_cast<int32_t*>(take(slots * E * 4));
  w.z = reinterpret_cast<float*>(take(slots * 4));
  w.n = reinterpret_cast<int32_t*>(take(slots * 4));
  if (ws) *ws = w;
  return at;
}
size_t balance_ws_bytes(int64_t T, int E, int S) {
  return balance_one(T, S) ? 0 : balance_layout(T, E, S, nullptr, nullptr);
}
int balance_launches(int64_t T, int S) { return balance_one(T, S) ? 1 : S == 1 ? 2 : 3; }

template <int J, bool ONE>
static void part(const BalanceArgs& a, const BalanceWs& ws, int per, hipStream_t s) {
  const dim3 grid(ONE ? 1 : (unsigned)((a.T + per - 1) / per)), block(64 * BAL_WAVES);
  if (a.sigmoid) {
    if (a.wide)
      hipLaunchKernelGGL((balance_part_kernel<J, true, true, ONE>), grid, block, 0, s, a, ws, per);
    else
      hipLaunchKernelGGL((balance_part_kernel<J, true, false, ONE>), grid, block, 0, s, a, ws, per);
  } else {
    if (a.wide)
      hipLaunchKernelGGL((balance_part_kernel<J, false, true, ONE>), grid, block, 0, s, a, ws, per);
    else
      hipLaunchKernelGGL((balance_part_kernel<J, false, false, ONE>), grid, block, 0, s, a, ws, per);
  }
}

hipError_t launch_balance(const BalanceArgs& a, int which, void* base, hipStream_t s) {
  BalanceWs ws{};
  if (balance_one(a.T, a.S)) {
    if (a.E <= 64)
      part<1, true>(a, ws, BAL_ONE, s);
    else if (a.E <= 128)
      part<2, true>(a, ws, BAL_ONE, s);
    else
      part<4, true>(a, ws, BAL_ONE, s);
    return hipGetLastError();
  }
  if (!base) return hipErrorInvalidValue;
  balance_layout(a.T, a.E, a.S, base, &ws);
  const int per = balance_per(a.T, a.S);
  if (which == 0) {
    if (a.E <= 64)
      part<1, false>(a, ws, per, s);
    else if (a.E <= 128)
      part<2, false>(a, ws, per, s);
    else
      part<4, false>(a, ws, per, s);
  } else if (which == 1) {
    if (a.E <= 64)
      hipLaunchKernelGGL(balance_seq_kernel<64>, dim3(a.S), dim3(1024), 0, s, a, ws, per);
    else if (a.E <= 128)
      hipLaunchKernelGGL(balance_seq_kernel<128>, dim3(a.S), dim3(1024), 0, s, a, ws, per);
    else
      hipLaunchKernelGGL(balance_seq_kernel<256>, dim3(a.S), dim3(1024), 0, s, a, ws, per);
  } else {
    hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(1024), 0, s, a, ws);
  }
  return hipGetLastError();
}

template <int J>
static void bwd(const BalanceArgs& a, const float* dlosses, const float* add, float* dlogits, int per, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + per - 1) / per)), block(256);
  if (a.sigmoid) {
    if (a.wide)
      hipLaunchKernelGGL((balance_bwd_kernel<J, true, true>), grid, block, 0, s, a, dlosses, add, dlogits, per);
    else
      hipLaunchKernelGGL((balance_bwd_kernel<J, true, false>), grid, block, 0, s, a, dlosses, add, dlogits, per);
  } else {
    if (a.wide)
      hipLaunchKernelGGL((balance_bwd_kernel<J, false, true>), grid, block, 0, s, a, dlosses, add, dlogits, per);
    else
      hipLaunchKernelGGL((balance_bwd_kernel<J, false, false>), grid, block, 0, s, a, dlosses, add, dlogits, per);
  }
}

hipError_t launch_balance_bwd(const BalanceArgs& a, const float* dlosses, const float* add, float* dlogits,
                              hipStream_t s) {
  // 16 tokens a workgroup until the card is full several times over
  int per = 16;
  while ((a.T + per - 1) / per > 4096) per *= 2;
  if (a.E <= 64)
    bwd<1>(a, dlosses, add, dlogits, per, s);
  else if (a.E <= 128)
    bwd<2>(a, dlosses, add, dlogits, per, s);
  else
    bwd<4>(a, dlosses, add, dlogits, per, s);
  return hipGetLastError();
}

}  // namespace mxmoe
