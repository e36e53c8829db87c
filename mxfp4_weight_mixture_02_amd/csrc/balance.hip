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
// 256-byte pieces (16 bytes a lane, at any element).  Scores are formed in fp32 relative to the largest of the
// token (of the sigmoids too: logits below -88 keep their ratios), with the
// hardware's base-2 exponential and reciprocal (1 ulp each; the argument's
// rounding is 2^-24 of it, which the largest scores do not see): the library's
// exponential and division took three quarters of the time.  Squares of the
// logsumexp, which fp32 may not hold though their mean is one, are formed and
// summed in fp64.  Probabilities are summed in fp32 over a wave's tokens (up to 32 a
// lane, then four lanes), in fp64 over waves, rounded to fp32 as a part and
// summed in fp64 over the parts: 35 roundings of 2^-24 at most (in fp64 from a lane
// on, 16384 x 256 took 4% longer).  The order of all sums is fixed.
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

// Four elements of a token from expert e on; `fill` past E.  WHOLE: E % 4 == 0.
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
template <bool WHOLE>
__device__ __forceinline__ f32x4 four(const float* row, int e, int E, float fill) {
  f32x4 v = {fill, fill, fill, fill};
  if (WHOLE ? e < E : e + 4 <= E) {
    v = *reinterpret_cast<const f32x4_any*>(row + e);
  } else if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (e + i < E) v[i] = row[e + i];
  }
  return v;
}

// A lane's logits of a token; -inf past E.
template <int J>
struct Logits {
  f32x4 x[J];
};
template <int J, bool WHOLE>
__device__ __forceinline__ void logits16(const float* row, int E, int l, Logits<J>& v) {
#pragma unroll
  for (int j = 0; j < J; ++j) v.x[j] = four<WHOLE>(row, 64 * j + 4 * l, E, -__builtin_inff());
}
__device__ __forceinline__ float exp_hw(float v) { return __builtin_amdgcn_exp2f(v * 1.4426950408889634f); }

// A token's normalised scores p and softmax (the same without SIG), its
// logsumexp and, with SIG, 1 - sigmoid of each logit.  A token of -inf alone
// has p, softmax and logsumexp 0.
template <int J, bool SIG>
struct Scores {
  float p[J][4], soft[J][4], rest[J][4];
  float lse;
};
template <int J, bool SIG>
__device__ __forceinline__ void scores(const Logits<J>& in, Scores<J, SIG>& s) {
  constexpr float INF = __builtin_inff();
  float m = -INF;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, in.x[j][i]);
  m = row16_max(m);
  if (m == -INF) m = 0.0f;
  float sum = 0.0f, total = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = in.x[j][i];
      s.soft[j][i] = exp_hw(v - m);
      sum += s.soft[j][i];
      if (SIG) {
        // sigmoid over the largest one's exp(min(m, 0)): exp(min(v, 0)) or
        // exp(v - m), over 1 + exp(-|v|)
        const float a = exp_hw(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.0f + a);
        const float g = v < 0.0f ? a : 1.0f;   // a NaN is in r
        s.p[j][i] = (m < 0.0f ? s.soft[j][i] : g) * r;
        s.rest[j][i] = v < 0.0f ? r : a * r;
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
// The first s in lo .. S - 1 with past(s), which holds from some s on (S: for
// none), by the whole wave: 64 places at a time, where a search by halves waits
// for a load each.
template <class F>
__device__ __forceinline__ int first_of(int lo, int S, F past) {
  const int lane = threadIdx.x & 63;
  int hi = S;   // lo .. hi: the answer's range
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64, at = lo + lane * step;
    const uint64_t behind = __ballot(at >= hi || past(at));
    const int f = behind ? __builtin_ctzll(behind) : 64;
    hi = min(hi, lo + f * step);
    if (f) lo += (f - 1) * step + 1;
  }
  return lo;
}

constexpr int BAL_WAVES = 8;               // waves of a workgroup: 32 tokens at a time

// The forward's scratch: a slot for each part of a sequence, its tokens in one
// block of `per` tokens.  Block b's part of sequence s is slot b + s: along the
// tokens either grows, so no two parts share one, and a sequence's are side by
// side.  Slot u has a workgroup of its own, which finds s: the last sequence
// whose first slot is not behind u.
struct BalanceWs {
  float* p;         // [slots, E] sums of p, rounded
  int32_t* c;       // [slots, E] choices
  double* z;        // [slots] sums of lse^2
  int32_t* n;       // [slots] tokens
  double* seq;      // [S, 2] balance of a sequence, sum of lse^2
  int32_t* done;    // sequences that are finished: 0 from the parts' launch
};

// 16384 tokens x 256 experts in 13 sequences, sigmoid, masked: 11 us, 1.5 TB/s: a
// chain of the search, 64 KB a workgroup asked for at once, and the arithmetic.
// (A workgroup for each block, which went through its sequences one after the
// other, took 12.4, and for 33 tokens in 13 sequences the call 41 us against
// 12.5.  Sixteen waves, 64 tokens at a time: 1 us more.)
//
// Partial sums of a slot's tokens.  ONE: all tokens are one sequence and this
// workgroup's, which also finishes.
template <int J, bool SIG, bool WHOLE, bool ONE>
__global__ __launch_bounds__(64 * BAL_WAVES) void balance_part_kernel(BalanceArgs a, BalanceWs ws, int per) {
  __shared__ float part[BAL_WAVES][256];
  __shared__ int hist[256];
  __shared__ double zpart[BAL_WAVES];
  __shared__ int npart[BAL_WAVES];
  __shared__ double fin[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & 15, row = tid >> 4;
  const int slot = blockIdx.x;
  if (!ONE && slot == 0 && tid == 0) *ws.done = 0;
  int s = 0;
  if (!ONE && a.offsets) {
    s = first_of(0, a.S, [&](int i) { return seq_begin(a, i) / per + i > slot; }) - 1;
    if (s < 0) return;   // ahead of the first sequence
  }
  const int64_t t0 = (int64_t)(slot - s) * per;
  const int64_t lo = max(seq_begin(a, s), t0), hi = min(seq_end(a, s), t0 + per);
  if (!ONE && lo >= hi) return;   // ONE: a sequence without tokens has its zeros written
  // A token's loads are issued a round ahead.
  Logits<J> x;
  int live = 1, pick = -1;
  auto fetch = [&](int64_t t, Logits<J>& y, int& on, int& e) {
    logits16<J, WHOLE>(a.logits + t * a.E, a.E, l, y);
    on = a.mask ? a.mask[t] : 1;
    e = l < a.k ? a.topk_idx[t * a.k + l] : -1;
  };
  if (lo + row < hi) fetch(lo + row, x, live, pick);
  for (int e = tid; e < 256; e += 64 * BAL_WAVES) hist[e] = 0;
  __syncthreads();
  float acc[J][4] = {};
  double z = 0.0;
  int n = 0;
  for (int64_t t = lo + row; t < hi; t += 4 * BAL_WAVES) {   // a row's 16 lanes go together
    Logits<J> next;
    int next_live = 1, next_pick = -1;
    if (t + 4 * BAL_WAVES < hi) fetch(t + 4 * BAL_WAVES, next, next_live, next_pick);
    if (live) {
      Scores<J, SIG> q;
      scores<J, SIG>(x, q);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] += q.p[j][i];
      if (pick >= 0 && pick < a.E) atomicAdd(&hist[pick], 1);
      z += (double)q.lse * (double)q.lse;
      ++n;
    }
    x = next;
    live = next_live;
    pick = next_pick;
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
  double pe = 0.0, ze = 0.0;
  int ne = 0;
#pragma unroll
  for (int u = 0; u < BAL_WAVES; ++u) {
    if (tid < 64 * J) pe += part[u][tid];
    ze += zpart[u];
    ne += npart[u];
  }
  if constexpr (!ONE) {
    if (tid < a.E) {
      ws.p[(int64_t)slot * a.E + tid] = (float)pe;
      ws.c[(int64_t)slot * a.E + tid] = hist[tid];
    }
    if (tid == 0) {
      ws.z[slot] = ze;
      ws.n[slot] = ne;
    }
  } else {
    double w = 0.0;
    if (tid < a.E) {
      const double mean = ne ? pe / ne : 0.0;
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
__device__ __forceinline__ V wave_add(V v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// A sequence per workgroup: its parts' sums; 1024 threads are EP experts by
// slices of the parts.  With several sequences, the workgroup that ends last
// joins their losses, in the sequences' order (a launch of its own takes 4 us).
// A chain of dependent loads: 9.4 us for 13 sequences of 20 parts.
template <int EP>
__global__ __launch_bounds__(1024) void balance_seq_kernel(BalanceArgs a, BalanceWs ws, int per) {
  constexpr int SL = 1024 / EP;
  __shared__ double sums[1024];
  __shared__ int cs[1024];
  __shared__ double zs[16], wsum[16], ns[16], some[16];
  __shared__ int is[16], last;
  const int tid = threadIdx.x, e = tid % EP, sl = tid / EP, s = blockIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t lo = seq_begin(a, s), hi = seq_end(a, s);
  const int64_t b0 = lo / per, b1 = hi > lo ? (hi - 1) / per + 1 : b0;   // its workgroups
  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  for (int64_t b = b0 + tid; b < b1; b += 1024) {
    z += ws.z[b + s];
    n += ws.n[b + s];
  }
  if (e < a.E) {
#pragma unroll 8
    for (int64_t b = b0 + sl; b < b1; b += SL) {
      p += (double)ws.p[(b + s) * a.E + e];
      c += ws.c[(b + s) * a.E + e];
    }
  }
  z = wave_add(z);
  n = wave_add(n);
  sums[tid] = p;
  cs[tid] = c;
  if (lane == 0) {
    zs[wave] = z;
    is[wave] = n;
  }
  __syncthreads();
  z = 0.0;
  n = 0;
  for (int u = 0; u < 16; ++u) {
    z += zs[u];
    n += is[u];
  }
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
  if (tid < EP) w = wave_add(w);
  if (lane == 0) wsum[wave] = w;
  __syncthreads();
  if (tid == 0) {
    w = 0.0;
    for (int u = 0; u < EP / 64; ++u) w += wsum[u];
    w = w * a.E / (a.k * div);
    a.tokens[s] = n;
    if (a.S == 1) {
      a.losses[0] = (float)w;
      a.losses[1] = (float)(z / div);
    } else {
      ws.seq[2 * s] = w;
      ws.seq[2 * s + 1] = z;
      // what this workgroup wrote is seen by whoever sees the count
      last = __hip_atomic_fetch_add(ws.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == a.S - 1;
    }
  }
  if (a.S == 1) return;
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  double some_ = 0.0, n_ = 0.0;
  w = z = 0.0;
  for (int i = tid; i < a.S; i += 1024) {
    const int t = a.tokens[i];
    w += ws.seq[2 * i];   // 0 without tokens
    z += ws.seq[2 * i + 1];
    n_ += t;
    some_ += t > 0;
  }
  w = wave_add(w);
  z = wave_add(z);
  n_ = wave_add(n_);
  some_ = wave_add(some_);
  if (lane == 0) {
    wsum[wave] = w;
    zs[wave] = z;
    ns[wave] = n_;
    some[wave] = some_;
  }
  __syncthreads();
  if (tid) return;
  for (int u = 1; u < 16; ++u) {
    w += wsum[u];
    z += zs[u];
    n_ += ns[u];
    some_ += some[u];
  }
  a.losses[0] = (float)(some_ > 0.0 ? w / some_ : 0.0);
  a.losses[1] = (float)(n_ > 0.0 ? z / n_ : 0.0);
}

// 8192 x 128, softmax, added to another gradient: 5.1 us, 2.5 TB/s.
//
// dlogits: 16 tokens at a time in a workgroup, `per` in all.  A wave looks its
// first token's sequence up, and those of the rows whose tokens lie behind it.
// add may be dlogits: a lane reads its elements before it writes them.
template <int J, bool SIG, bool WHOLE>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceArgs a, const float* __restrict__ dlosses,
                                                          const float* add, float* dlogits, int per) {
  __shared__ int all[4], some[4];
  const int tid = threadIdx.x, l = tid & 15, row = tid >> 4;
  const int64_t first = (int64_t)blockIdx.x * per, t1 = min(first + per, a.T);
  // the first token's logits are under way while the sequences are counted
  Logits<J> x;
  if (first + row < t1) logits16<J, WHOLE>(a.logits + (first + row) * a.E, a.E, l, x);
  int n_ = 0, some_ = 0;   // N <= T < 2^26
  for (int s = tid; s < a.S; s += 256) {
    const int n = a.tokens[s];
    n_ += n;
    some_ += n > 0;
  }
  n_ = wave_add(n_);
  some_ = wave_add(some_);
  if ((tid & 63) == 0) {
    all[tid >> 6] = n_;
    some[tid >> 6] = some_;
  }
  auto after = [&](int from, int64_t t) {   // the first sequence that ends behind token t
    return first_of(from, a.S, [&](int i) { return seq_end(a, i) > t; });
  };
  const int wrow = row & ~3;   // the wave's first row
  int s = a.offsets ? after(0, first + wrow) : 0;
  __syncthreads();
  n_ = all[0] + all[1] + all[2] + all[3];
  some_ = some[0] + some[1] + some[2] + some[3];
  const float da = dlosses[0] * (float)a.E / (float)a.k, db = n_ > 0 ? 2.0f * dlosses[1] / (float)n_ : 0.0f;
  for (int64_t base = first; base < t1; base += 16) {   // uniform
    const int64_t t = base + row;
    if (a.offsets) {
      uint64_t gone = __ballot(t < t1 && s < a.S && seq_end(a, s) <= t);
      while (gone) {   // one row after the other
        const int r = __builtin_ctzll(gone) >> 4;
        const int found = after(__builtin_amdgcn_readlane(s, 16 * r), base + wrow + r);
        if ((tid >> 4 & 3) == r) s = found;
        gone &= ~(0xFFFFull << 16 * r);
      }
    }
    if (t >= t1) continue;
    if (base > first) logits16<J, WHOLE>(a.logits + t * a.E, a.E, l, x);
    const bool live = s < a.S && seq_begin(a, s) <= t && !(a.mask && !a.mask[t]);
    float d[J][4] = {};
    if (live) {
      Scores<J, SIG> q;
      scores<J, SIG>(x, q);
      const float n = (float)a.tokens[s], f = n > 0.0f ? da / (n * n * (float)some_) : 0.0f;
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
      if (add) v += four<WHOLE>(add + t * a.E, e, a.E, 0.0f);
      float* o = dlogits + t * a.E + e;
      if (WHOLE || e + 4 <= a.E) {
        *reinterpret_cast<f32x4_any*>(o) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (e + i < a.E) o[i] = v[i];
      }
    }
  }
}

// ------------------------------------------------------------------ launchers

// Tokens of a workgroup: its 32 at a time, and more of them while workgroups
// are many, whose parts are read again.
static int balance_per(int64_t T) {
  int per = 32;
  while (per < 1024 && (T + per - 1) / per > 256) per *= 2;
  return per;
}
// One sequence of few tokens: a launch less, while one CU takes less time for
// them (256 x 256: 15.2 us against 9.3).
static int lane_experts(int E) { return E <= 64 ? 64 : E <= 128 ? 128 : 256; }
static bool balance_one(int64_t T, int E, int S) { return S == 1 && T * lane_experts(E) <= 16384; }

static size_t balance_layout(int64_t T, int E, int S, void* base, BalanceWs* ws) {
  const int per = balance_per(T);
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
  w.done = reinterpret_cast<int32_t*>(take(4));
  w.p = reinterpret_cast<float*>(take(slots * E * 4));
  w.c = reinterpret_cast<int32_t*>(take(slots * E * 4));
  w.z = reinterpret_cast<double*>(take(slots * 8));
  w.n = reinterpret_cast<int32_t*>(take(slots * 4));
  if (ws) *ws = w;
  return at;
}
size_t balance_ws_bytes(int64_t T, int E, int S) {
  return balance_one(T, E, S) ? 0 : balance_layout(T, E, S, nullptr, nullptr);
}
int balance_launches(int64_t T, int E, int S) { return balance_one(T, E, S) ? 1 : 2; }

template <int J, bool ONE>
static void part(const BalanceArgs& a, const BalanceWs& ws, int per, hipStream_t s) {
  // one sequence of all tokens has a slot for each block
  const dim3 grid(ONE ? 1 : (unsigned)((a.T + per - 1) / per + (a.offsets ? a.S : 0))), block(64 * BAL_WAVES);
  if (a.sigmoid) {
    if (a.E % 4 == 0)
      hipLaunchKernelGGL((balance_part_kernel<J, true, true, ONE>), grid, block, 0, s, a, ws, per);
    else
      hipLaunchKernelGGL((balance_part_kernel<J, true, false, ONE>), grid, block, 0, s, a, ws, per);
  } else {
    if (a.E % 4 == 0)
      hipLaunchKernelGGL((balance_part_kernel<J, false, true, ONE>), grid, block, 0, s, a, ws, per);
    else
      hipLaunchKernelGGL((balance_part_kernel<J, false, false, ONE>), grid, block, 0, s, a, ws, per);
  }
}

hipError_t launch_balance(const BalanceArgs& a, int which, void* base, hipStream_t s) {
  BalanceWs ws{};
  if (balance_one(a.T, a.E, a.S)) {
    if (a.E <= 64)
      part<1, true>(a, ws, (int)a.T, s);
    else if (a.E <= 128)
      part<2, true>(a, ws, (int)a.T, s);
    else
      part<4, true>(a, ws, (int)a.T, s);
    return hipGetLastError();
  }
  if (!base) return hipErrorInvalidValue;
  balance_layout(a.T, a.E, a.S, base, &ws);
  const int per = balance_per(a.T);
  if (which == 0) {
    if (a.E <= 64)
      part<1, false>(a, ws, per, s);
    else if (a.E <= 128)
      part<2, false>(a, ws, per, s);
    else
      part<4, false>(a, ws, per, s);
  } else {
    if (a.E <= 64)
      hipLaunchKernelGGL(balance_seq_kernel<64>, dim3(a.S), dim3(1024), 0, s, a, ws, per);
    else if (a.E <= 128)
      hipLaunchKernelGGL(balance_seq_kernel<128>, dim3(a.S), dim3(1024), 0, s, a, ws, per);
    else
      hipLaunchKernelGGL(balance_seq_kernel<256>, dim3(a.S), dim3(1024), 0, s, a, ws, per);
  }
  return hipGetLastError();
}

template <int J>
static void bwd(const BalanceArgs& a, const float* dlosses, const float* add, float* dlogits, int per, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + per - 1) / per)), block(256);
  if (a.sigmoid) {
    if (a.E % 4 == 0)
      hipLaunchKernelGGL((balance_bwd_kernel<J, true, true>), grid, block, 0, s, a, dlosses, add, dlogits, per);
    else
      hipLaunchKernelGGL((balance_bwd_kernel<J, true, false>), grid, block, 0, s, a, dlosses, add, dlogits, per);
  } else {
    if (a.E % 4 == 0)
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
