// Routing from logits (gfx950): softmax or sigmoid scores, a selection bias,
// groups of experts, top-k, weights and the permutation plan; and the
// gradient of the weights with respect to the logits.
//
// A token belongs to a wave, lane l with experts NQ l .. NQ l + NQ - 1 (NQ =
// ceil(E / 64)), or to a row of 16 lanes, four tokens in a wave (NQ =
// ceil(E / 16)).  Scores are formed in fp64 and the choice is taken on
// c = fp32(s + bias), so that neighbours in the order do not change places
// with the rounding of an fp32 exponential.  The k largest come from k
// rounds of a wave maximum over integer keys.
#include <type_traits>

#include "common.hpp"
#include "gate.hpp"
#include "launch.hpp"

// Sums and products are rounded one by one: a score is the same number where
// its bias is added and where the weights are formed, and every layout of the
// choice and of the gradient gives the same bits.
#pragma clang fp contract(off)

namespace mxmoe {

// Total-order key of a choice value: larger key = larger value, -0.0 equal
// to +0.0, NaN below every number; INT32_MIN is left for experts that may
// not be chosen.
__device__ __forceinline__ int32_t choice_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u << 1) == 0u) u = 0u;
  const int32_t b = (int32_t)u;
  return (f != f) ? INT32_MIN + 1 : (b ^ ((b >> 31) & 0x7FFFFFFF));
}

// Exchanges within rows of 16 lanes by DPP: lanes xor 1, xor 2, mirrored
// within 8, mirrored within 16 (a mirror does as an xor once the lanes below
// agree); a chain of LDS shuffles takes several times the time.
template <int STEP>
__device__ __forceinline__ int32_t dpp_swap(int32_t v) {
  constexpr int CTRL = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ int32_t row_max(int32_t v) {
  v = max(v, dpp_swap<1>(v));
  v = max(v, dpp_swap<2>(v));
  v = max(v, dpp_swap<4>(v));
  return max(v, dpp_swap<8>(v));
}
// Largest value over the wave, as a scalar: the rows joined by broadcasts
// (row_bcast:15 into rows 1 and 3, row_bcast:31 into rows 2 and 3).
__device__ __forceinline__ int32_t wave_max(int32_t v) {
  v = row_max(v);
  v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x143, 0xC, 0xF, false));
  return __builtin_amdgcn_readlane(v, 63);
}
// The number a choice key stands for (a NaN key gives a NaN).
__device__ __forceinline__ float key_number(int32_t k) {
  return __uint_as_float((uint32_t)(k ^ ((k >> 31) & 0x7FFFFFFF)));
}
// The largest of the wave's floats, NaN below every number.
__device__ __forceinline__ float wave_max(float v) {
  const int32_t k = wave_max(choice_key(v));
  return k == INT32_MIN + 1 ? -INFINITY : key_number(k);
}
// Sum of the first 8 lanes' values, in each of them.
template <int STEP>
__device__ __forceinline__ double dpp_swap(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp_swap<STEP>((int32_t)(uint32_t)b);
  const uint32_t hi = (uint32_t)dpp_swap<STEP>((int32_t)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double sum8(double v) {
  v += dpp_swap<1>(v);
  v += dpp_swap<2>(v);
  return v + dpp_swap<4>(v);
}
// Sum over the wave, in every lane.
__device__ __forceinline__ double wave_sum(double v) {
  v = sum8(v);
  v += dpp_swap<8>(v);
  auto bcast = [](double x, auto ctrl, auto rows) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, decltype(ctrl)::value,
                                                              decltype(rows)::value, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), decltype(ctrl)::value,
                                                              decltype(rows)::value, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
  };
  v += bcast(v, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
  v += bcast(v, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

// A result, with one NaN for all: the layouts reach a NaN by different
// operands, whose signs and payloads it would keep.
__device__ __forceinline__ float one_nan(float v) {
  return (__float_as_uint(v) & 0x7FFFFFFFu) > 0x7F800000u ? __uint_as_float(0x7FC00000u) : v;
}

// LDS of one wave's token.
struct TokenLds {
  double score[256];
  float c[256];
};

// Scores of a token's experts in fp64 (0 past E): v holds the logits.
template <int NQ>
__device__ __forceinline__ void token_scores(const float (&v)[NQ], int E, int lane, int sigmoid,
                                             double (&s)[NQ]) {
  if (sigmoid) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) s[q] = 1.0 / (1.0 + exp(-(double)v[q]));
    return;
  }
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    if (NQ * lane + q < E) m = fmaxf(m, v[q]);
  m = wave_max(m);
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    // a row of -inf alone has no finite maximum: scores 0
    s[q] = NQ * lane + q < E && !(v[q] == -INFINITY) ? exp((double)v[q] - (double)m) : 0.0;
    sum += s[q];
  }
  sum = wave_sum(sum);
  const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
  for (int q = 0; q < NQ; ++q) s[q] *= inv;
}

// Which groups are open to the choice, as a bit mask over groups.  `share`
// (a power of two, share * groups <= 64) lanes value a group from the token's
// choice values in LDS: each takes every share-th expert, the two largest
// are merged over the lanes, and a group is open if fewer than top_groups
// groups beat it.
__device__ __forceinline__ unsigned long long open_groups(const RouteArgs& a, const float* c,
                                                          int lane) {
  const int per = a.E / a.groups, share = a.share;
  const int g = lane / share;
  int32_t k1 = INT32_MIN, k2 = INT32_MIN;
  float c1 = 0.0f, c2 = 0.0f;
  auto take = [&](int32_t kv, float v) {
    const bool first = kv > k1, second = kv > k2;
    k2 = first ? k1 : second ? kv : k2;
    c2 = first ? c1 : second ? v : c2;
    k1 = first ? kv : k1;
    c1 = first ? v : c1;
  };
  if (g < a.groups)
    for (int i = lane % share; i < per; i += share) {
      const float v = c[g * per + i];
      take(choice_key(v), v);
    }
  for (int m = 1; m < share; m <<= 1) {
    const int32_t o1 = __shfl_xor(k1, m), o2 = __shfl_xor(k2, m);
    const float v1 = __shfl_xor(c1, m), v2 = __shfl_xor(c2, m);
    take(o1, v1);
    take(o2, v2);
  }
  const int32_t key = choice_key(a.top2 && per > 1 ? c1 + c2 : c1);
  int beaten = 0;
  for (int o = 0; o < a.groups; ++o) {
    const int32_t ok = __builtin_amdgcn_readlane(key, o * share);
    beaten += ok > key || (ok == key && o < g);
  }
  const unsigned long long lanes =
      __ballot(lane % share == 0 && g < a.groups && beaten < a.top_groups);
  if (share == 1) return lanes;
  unsigned long long open = 0;
  for (int o = 0; o < a.groups; ++o) open |= ((lanes >> (o * share)) & 1ull) << o;
  return open;
}

template <int NQ>
using Floats = float __attribute__((ext_vector_type(NQ)));

template <int NQ>
struct Lane {          // what a lane holds of its experts, whatever the token
  float bias[NQ];
  int group[NQ];
};
template <int NQ>
__device__ __forceinline__ Lane<NQ> lane_of(const RouteArgs& a, int lane) {
  Lane<NQ> l;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = min(NQ * lane + q, a.E - 1);
    l.bias[q] = a.bias ? a.bias[e] : 0.0f;
    l.group[q] = e / (a.E / a.groups);
  }
  return l;
}
// A lane's logits of token t (past E: some of the row's).
template <int NQ>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int lane, float (&v)[NQ]) {
  const float* row = a.logits + t * a.E;
  if (a.wide) {   // whole vectors: E % NQ == 0
    const auto x = *reinterpret_cast<const Floats<NQ>*>(row + min(NQ * lane, a.E - NQ));
#pragma unroll
    for (int q = 0; q < NQ; ++q) v[q] = x[q];
    return;
  }
#pragma unroll
  for (int q = 0; q < NQ; ++q) v[q] = row[min(NQ * lane + q, a.E - 1)];
}

// Whether this lane's group is open, where a group is `lanes` whole lanes (a
// power of two): k1 and k2 are the largest and second keys of the lane's
// experts.  The two largest are merged over the group's lanes, then each
// lane counts the groups that beat its own.
__device__ __forceinline__ bool lane_group_open(const RouteArgs& a, int lanes, int lane, int32_t k1,
                                                int32_t k2) {
  auto merge = [&](int32_t o1, int32_t o2) {
    k2 = max(min(k1, o1), max(k2, o2));
    k1 = max(k1, o1);
  };
  if (lanes > 1) merge(dpp_swap<1>(k1), dpp_swap<1>(k2));
  if (lanes > 2) merge(dpp_swap<2>(k1), dpp_swap<2>(k2));
  if (lanes > 4) merge(dpp_swap<4>(k1), dpp_swap<4>(k2));
  if (lanes > 8) merge(dpp_swap<8>(k1), dpp_swap<8>(k2));
  if (lanes > 16) merge(__shfl_xor(k1, 16), __shfl_xor(k2, 16));
  const int32_t key =
      a.top2 && a.E > a.groups ? choice_key(key_number(k1) + key_number(k2)) : k1;
  const int g = lane / lanes;
  int beaten = 0;
  for (int o = 0; o < a.groups; ++o) {
    const int32_t ok = __builtin_amdgcn_readlane(key, o * lanes);
    beaten += ok >= key + (o >= g);   // an equal key of a lower group beats too
  }
  return beaten < a.top_groups;
}

// Chooses token t's experts: lane j < k returns slot j's expert (others 0)
// and writes the slot's index and weight.  A lane's keys are sorted once
// (stably, so that ties stay in index order); a round takes the wave's
// largest head, from the lowest lane that has it, and that lane moves on.
template <int NQ>
__device__ __forceinline__ int choose(const RouteArgs& a, const Lane<NQ>& mine_of, int64_t t, int lane,
                                      const float (&v)[NQ], TokenLds& lds) {
  double s[NQ];
  token_scores<NQ>(v, a.E, lane, a.sigmoid, s);
  const bool grouped = a.top_groups < a.groups;
  int32_t key[NQ];
  int at[NQ];
  wave_lds_sync();   // the previous token's reads are done
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = NQ * lane + q;
    const float c = (float)(s[q] + (double)mine_of.bias[q]);
    key[q] = e < a.E ? choice_key(c) : INT32_MIN;
    at[q] = e;
    if (e < a.E) {
      lds.score[e] = s[q];
      if (grouped && !a.group_lanes) lds.c[e] = c;
    }
  }
  wave_lds_sync();
  if (grouped && !a.group_lanes) {
    const unsigned long long open = open_groups(a, lds.c, lane);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (!((open >> mine_of.group[q]) & 1)) key[q] = INT32_MIN;
  }
#pragma unroll
  for (int n = NQ - 1; n > 0; --n)
#pragma unroll
    for (int q = 0; q < n; ++q) {
      const bool swap = key[q] < key[q + 1];
      const int32_t kq = key[q];
      const int aq = at[q];
      key[q] = swap ? key[q + 1] : kq;
      at[q] = swap ? at[q + 1] : aq;
      key[q + 1] = swap ? kq : key[q + 1];
      at[q + 1] = swap ? aq : at[q + 1];
    }
  if (grouped && a.group_lanes &&
      !lane_group_open(a, a.group_lanes, lane, key[0], NQ > 1 ? key[NQ > 1] : INT32_MIN)) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) key[q] = INT32_MIN;
  }
  int mine = 0, k = a.k, l = lane;
  // compared in the rounds, not in registers kept (and spilled) for all tokens
  asm volatile("" : "+s"(k), "+v"(l));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= k) break;
    const int32_t top = wave_max(key[0]);
    const int owner = (int)__builtin_ctzll(__ballot(key[0] == top));
    const int e = __builtin_amdgcn_readlane(at[0], owner);
    if (l == j) mine = e;
    if (l == owner) {
#pragma unroll
      for (int q = 0; q + 1 < NQ; ++q) {
        key[q] = key[q + 1];
        at[q] = at[q + 1];
      }
      key[NQ - 1] = INT32_MIN;
    }
  }
  // weights: the chosen scores, over their sum
  const double sc = lane < a.k ? lds.score[mine] : 0.0;
  const double total = a.renorm ? sum8(sc) : 1.0;
  if (lane < a.k) {
    a.topk_idx[t * a.k + lane] = mine;
    a.topk_w[t * a.k + lane] = one_nan((float)(total == 0.0 ? 0.0 : sc / total * (double)a.scale));
  }
  return mine;
}

// The choice of `per_block` tokens by one workgroup of 16 waves, and the
// workgroup's histogram of experts.  This form takes what rows of 16 lanes do
// not (gate_rows_kernel): groups that are not whole lanes of a row, E % 4,
// unaligned logits.  Bound by vector instructions (about 550 a token): 16384
// tokens x 256 experts, k = 8 in 25 us.
constexpr int GATE_W = 16;
template <int NQ>
__global__ __launch_bounds__(64 * GATE_W) void gate_kernel(RouteArgs a, int per_block,
                                                           int32_t* __restrict__ hist_out) {
  __shared__ TokenLds lds[GATE_W];
  __shared__ int32_t hist[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < 256) hist[tid] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * per_block;
  const int n = (int)min((int64_t)per_block, a.T - t0);
  const Lane<NQ> mine = lane_of<NQ>(a, lane);
  float v[NQ], next[NQ];
  load_logits<NQ>(a, t0 + min(wave, n - 1), lane, v);
  for (int i = wave; i < n; i += GATE_W) {
    load_logits<NQ>(a, t0 + min(i + GATE_W, n - 1), lane, next);   // the next token's, under this one's choice
    const int e = choose<NQ>(a, mine, t0 + i, lane, v, lds[wave]);
#pragma unroll
    for (int q = 0; q < NQ; ++q) v[q] = next[q];
    if (lane < a.k) atomicAdd(&hist[e], 1);   // counts only: order does not matter
  }
  __syncthreads();
  if (tid < a.E) hist_out[(int64_t)blockIdx.x * a.E + tid] = hist[tid];
}

// Four tokens at a time in a wave, a row of 16 lanes each, lane r with experts
// NQ r .. NQ r + NQ - 1.  A round of the choice is then eight DPP steps for
// four tokens instead of six and three scalar reads for each; what it costs
// more is the sorting of a lane's 4, 8 or 16 experts (networks of 5 and 19
// comparisons; of two sorted eights the larger halves are merged).  Entries
// are (key, 255 - expert) in 64 bits, so ties sort by index.  Whole routing,
// one token a wave against this (us): 16384 x 256, k 8 28.2, 23.7; 65536 x
// 64, k 6 47.3, 28.9; 2048 x 32, k 4 8.6, 7.6; 100 x 256 10.6, 10.4.
template <int I, int J, int N>
__device__ __forceinline__ void exchange(int64_t (&x)[N]) {   // the larger to I
  const int64_t a = x[I], b = x[J];
  const bool swap = a < b;
  x[I] = swap ? b : a;
  x[J] = swap ? a : b;
}
template <int O, int N>
__device__ __forceinline__ void sort4(int64_t (&x)[N]) {
  exchange<O, O + 1>(x), exchange<O + 2, O + 3>(x);
  exchange<O, O + 2>(x), exchange<O + 1, O + 3>(x);
  exchange<O + 1, O + 2>(x);
}
template <int O, int N>
__device__ __forceinline__ void sort8(int64_t (&x)[N]) {
  exchange<O, O + 2>(x), exchange<O + 1, O + 3>(x), exchange<O + 4, O + 6>(x), exchange<O + 5, O + 7>(x);
  exchange<O, O + 4>(x), exchange<O + 1, O + 5>(x), exchange<O + 2, O + 6>(x), exchange<O + 3, O + 7>(x);
  exchange<O, O + 1>(x), exchange<O + 2, O + 3>(x), exchange<O + 4, O + 5>(x), exchange<O + 6, O + 7>(x);
  exchange<O + 2, O + 4>(x), exchange<O + 3, O + 5>(x);
  exchange<O + 1, O + 4>(x), exchange<O + 3, O + 6>(x);
  exchange<O + 1, O + 2>(x), exchange<O + 3, O + 4>(x), exchange<O + 5, O + 6>(x);
}
// The eight largest (all, if there are fewer), descending, in x[0] ..
template <int N>
__device__ __forceinline__ void sort_heads(int64_t (&x)[N]) {
  if constexpr (N == 4) {
    sort4<0>(x);
  } else {
    sort8<0>(x);
    if constexpr (N == 16) {
      sort8<8>(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] < x[15 - i] ? x[15 - i] : x[i];
      exchange<0, 4>(x), exchange<1, 5>(x), exchange<2, 6>(x), exchange<3, 7>(x);
      exchange<0, 2>(x), exchange<1, 3>(x), exchange<4, 6>(x), exchange<5, 7>(x);
      exchange<0, 1>(x), exchange<2, 3>(x), exchange<4, 5>(x), exchange<6, 7>(x);
    }
  }
}
__device__ __forceinline__ int32_t key_of(int64_t x) { return (int32_t)(x >> 32); }

// A lane's NQ logits of its row's token (E % 4 == 0).
template <int NQ>
__device__ __forceinline__ void load_row(const float* row, int E, int r, float (&v)[NQ]) {
#pragma unroll
  for (int q = 0; q < NQ; q += 4) {
    const auto y = *reinterpret_cast<const Floats<4>*>(row + min(NQ * r + q, E - 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[q + i] = y[i];
  }
}
// Softmax over a row of 16 lanes: s = exp(v - m) in fp64, 0 past E, and the
// inverse of their sum, added in token_scores()'s order.
template <int NQ>
__device__ __forceinline__ double row_softmax(const float (&v)[NQ], int E, int r, float& m, double (&s)[NQ]) {
  double part[4];
  m = -INFINITY;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    if (NQ * r + q < E) m = fmaxf(m, v[q]);
  const int32_t top = row_max(choice_key(m));
  m = key_number(top);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    part[p] = 0.0;
#pragma unroll
    for (int q = p * NQ / 4; q < (p + 1) * NQ / 4; ++q) {
      s[q] = NQ * r + q < E && !(v[q] == -INFINITY) ? exp((double)v[q] - (double)m) : 0.0;
      part[p] += s[q];
      // interleaved further, the exponentials of 16 experts do not fit the
      // registers of four waves a SIMD
      if (NQ > 8 && q % 2) __builtin_amdgcn_sched_barrier(0);
    }
  }
  double sum = sum8((part[0] + part[1]) + (part[2] + part[3]));
  sum += dpp_swap<8>(sum);
  return sum == 0.0 ? 0.0 : 1.0 / sum;
}
// One logit's score, by the same steps.
__device__ __forceinline__ double one_score(int sigmoid, float l, float m, double inv) {
  if (sigmoid) return 1.0 / (1.0 + exp(-(double)l));
  return (l == -INFINITY ? 0.0 : exp((double)l - (double)m)) * inv;
}

// Chooses token t's experts, as choose() does; t per row of 16 lanes, r the
// lane in it.
template <int NQ>
__device__ __forceinline__ int choose_row(const RouteArgs& a, const float* bias, int64_t t, bool on,
                                          int lane) {
  constexpr int HEADS = NQ < 8 ? NQ : 8;
  const int r = lane & 15;
  const float* row = a.logits + t * a.E;
  float v[NQ];
  load_row<NQ>(row, a.E, r, v);
  int64_t x[NQ];
  auto enter = [&](int q, double s) {
    const int e = NQ * r + q;
    const int32_t key = e < a.E ? choice_key((float)(s + (double)bias[e])) : INT32_MIN;
    x[q] = (int64_t)((uint64_t)(uint32_t)key << 32 | (uint32_t)(255 - e));
  };
  double inv = 0.0;
  float m = 0.0f;
  if (a.sigmoid) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      enter(q, one_score(1, v[q], 0.0f, 0.0));
      if (NQ > 8 && q % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // registers, as above
    }
  } else {
    double s[NQ];
    inv = row_softmax<NQ>(v, a.E, r, m, s);
#pragma unroll
    for (int q = 0; q < NQ; ++q) enter(q, s[q] * inv);
  }
  sort_heads(x);
  if (a.top_groups < a.groups) {
    // as lane_group_open, the groups' values from lanes of the token's row
    int32_t k1 = key_of(x[0]), k2 = key_of(x[1]);
    auto merge = [&](int32_t o1, int32_t o2) {
      k2 = max(min(k1, o1), max(k2, o2));
      k1 = max(k1, o1);
    };
    if (a.row_lanes > 1) merge(dpp_swap<1>(k1), dpp_swap<1>(k2));
    if (a.row_lanes > 2) merge(dpp_swap<2>(k1), dpp_swap<2>(k2));
    if (a.row_lanes > 4) merge(dpp_swap<4>(k1), dpp_swap<4>(k2));
    const int32_t key = a.top2 && a.E > a.groups ? choice_key(key_number(k1) + key_number(k2)) : k1;
    const int g = r / a.row_lanes;
    int beaten = 0;
    for (int o = 0; o < a.groups; ++o)
      beaten += __shfl(key, (lane & 48) + o * a.row_lanes) >= key + (o >= g);
    if (beaten >= a.top_groups) {
#pragma unroll
      for (int q = 0; q < HEADS; ++q) x[q] = (int64_t)((uint64_t)0x80000000u << 32 | (uint32_t)x[q]);
    }
  }
  int mine = 0, k = a.k;
  asm volatile("" : "+s"(k));   // compared in the rounds
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= k) break;
    const int32_t top = row_max(key_of(x[0]));
    const int32_t low = row_max(key_of(x[0]) == top ? (int32_t)x[0] : -1);
    if (r == j) mine = 255 - low;
    if ((int32_t)x[0] == low) {
#pragma unroll
      for (int q = 0; q + 1 < HEADS; ++q) x[q] = x[q + 1];
      x[HEADS - 1] = (int64_t)((uint64_t)0x80000000u << 32 | 0xFFFFFFFFu);
    }
  }
  // the chosen scores again from their logits
  const double sc = r < k ? one_score(a.sigmoid, row[mine], m, inv) : 0.0;
  const double total = a.renorm ? sum8(sc) : 1.0;
  if (r < k && on) {
    a.topk_idx[t * k + r] = mine;
    a.topk_w[t * k + r] = one_nan((float)(total == 0.0 ? 0.0 : sc / total * (double)a.scale));
  }
  return mine;
}

// gate_kernel's work in rows of 16 lanes.  Bound by vector instructions, of
// which the fp64 scores are about half: 16384 x 256, k 8 in 17.6 us, 2048 x 32
// in 4.2.  With 16 experts a lane two registers are spilled.
template <int NQ>
__global__ __launch_bounds__(64 * GATE_W) void gate_rows_kernel(RouteArgs a, int per_block,
                                                                int32_t* __restrict__ hist_out) {
  __shared__ int32_t hist[256];
  __shared__ __align__(16) float bias[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15;
  if (tid < 256) {
    hist[tid] = 0;
    bias[tid] = a.bias && tid < a.E ? a.bias[tid] : 0.0f;
  }
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * per_block;
  const int n = (int)min((int64_t)per_block, a.T - t0);
  for (int b = 4 * wave; b < n; b += 4 * GATE_W) {
    const int i = b + (lane >> 4);
    const int e = choose_row<NQ>(a, bias, t0 + min(i, n - 1), i < n, lane);
    if (r < a.k && i < n) atomicAdd(&hist[e], 1);   // counts only: order does not matter
  }
  __syncthreads();
  if (tid < a.E) hist_out[(int64_t)blockIdx.x * a.E + tid] = hist[tid];
}

// Few tokens (T <= GATE_ONE_TOKENS): choice, offsets and permutation in one
// workgroup.  A chain of dependent steps, so bound by latency: one token of
// 256 experts, k = 8 in 5.5 us, against three launches of 3 us and more.
constexpr int GATE_ONE_TOKENS = 32;
template <int NQ>
__global__ __launch_bounds__(64 * GATE_W) void gate_one_kernel(RouteArgs a) {
  __shared__ TokenLds lds[GATE_W];
  __shared__ int32_t ex[GATE_ONE_TOKENS * 8];
  __shared__ int32_t off[257];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Lane<NQ> mine = lane_of<NQ>(a, lane);
  for (int t = wave; t < (int)a.T; t += GATE_W) {
    float v[NQ];
    load_logits<NQ>(a, t, lane, v);
    const int e = choose<NQ>(a, mine, t, lane, v, lds[wave]);
    if (lane < a.k) ex[t * a.k + lane] = e;
  }
  __syncthreads();
  const int R = (int)a.T * a.k;
  // rows of lower experts are before expert tid's: its offset
  if (tid <= a.E) {
    int n = 0;
    for (int f = 0; f < R; ++f) n += ex[f] < tid;
    off[tid] = n;
    a.offsets[tid] = n;
  }
  __syncthreads();
  if (tid < R) {
    int rank = 0;
    for (int f = 0; f < tid; ++f) rank += ex[f] == ex[tid];
    a.sorted_rows[off[ex[tid]] + rank] = tid;
  }
}

// Expert e = blockIdx.x: in place, hist[b][e] becomes the number of rows of
// e in workgroups before b; total[e] their sum.  Latency (a scan of 256
// numbers): 4.0 us for 256 workgroups x 256 experts.
__global__ __launch_bounds__(256) void gate_prefix_kernel(int32_t* __restrict__ hist, int nblk,
                                                          int E, int32_t* __restrict__ total) {
  __shared__ int32_t part[256];
  const int e = blockIdx.x, tid = threadIdx.x;
  const int per = (nblk + 255) / 256;
  const int b0 = min(tid * per, nblk), b1 = min(b0 + per, nblk);
  int32_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += hist[(int64_t)b * E + e];
  part[tid] = sum;
  __syncthreads();
  for (int d = 1; d < 256; d <<= 1) {
    const int32_t o = tid >= d ? part[tid - d] : 0;
    __syncthreads();
    part[tid] += o;
    __syncthreads();
  }
  int32_t run = part[tid] - sum;
  if (tid == 255) total[e] = part[255];
  for (int b = b0; b < b1; ++b) {
    const int32_t v = hist[(int64_t)b * E + e];
    hist[(int64_t)b * E + e] = run;
    run += v;
  }
}

// Offsets from the totals, and each workgroup's rows to their places:
// offsets[e] + rows of e in earlier workgroups + earlier rows of e here.  A
// chunk of 256 rows at a time: within a wave, the rows of the same expert
// come from eight ballots on the bits of its number; over the waves, from
// counts in LDS.  base and total are gate_prefix_kernel's, or with total ==
// nullptr base holds the workgroups' histograms and every workgroup adds up
// the few there are (2048 tokens: one launch less, 3 us of host time).
// 131072 rows of 256 experts in 4.1 us.
__global__ __launch_bounds__(256) void gate_scatter_kernel(RouteArgs a, int per_block,
                                                           const int32_t* __restrict__ base,
                                                           const int32_t* __restrict__ total) {
  __shared__ int32_t off[256];
  __shared__ int32_t cnt[4][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t mine = 0, before = 0;
  if (total) {
    mine = tid < a.E ? total[tid] : 0;
    before = tid < a.E ? base[(int64_t)blockIdx.x * a.E + tid] : 0;
  } else {
    // thread (c, e) adds workgroups c, c + C, ... of expert e
    const int C = 256 / a.E, c = tid / a.E, e = tid % a.E, nblk = gridDim.x;
    cnt[0][tid] = cnt[1][tid] = 0;
    __syncthreads();
    if (c < C) {
      int32_t all = 0, early = 0;
      int b0 = c;
      auto add = [&](auto loads) {   // of so many workgroups, all under way at once
        constexpr int N = decltype(loads)::value;
        int32_t v[N];
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = base[(int64_t)min(b0 + u * C, nblk - 1) * a.E + e];
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const int b = b0 + u * C;
          all += b < nblk ? v[u] : 0;
          early += b < (int)blockIdx.x ? v[u] : 0;
        }
        b0 += N * C;
      };
      while (b0 + 16 * C < nblk) add(std::integral_constant<int, 32>{});
      while (b0 < nblk) add(std::integral_constant<int, 8>{});
      atomicAdd(&cnt[0][e], all);   // whole numbers: order does not matter
      atomicAdd(&cnt[1][e], early);
    }
    __syncthreads();
    mine = cnt[0][tid];
    before = cnt[1][tid];
    __syncthreads();
  }
  // exclusive sum of the totals: within a wave by shuffles, over waves by LDS
  int32_t inc = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) cnt[0][wave] = inc;
  __syncthreads();
  int32_t start = inc - mine;
  for (int w = 0; w < wave; ++w) start += cnt[0][w];
  if (blockIdx.x == 0) {
    if (tid < a.E) a.offsets[tid] = start;
    if (tid == a.E - 1) a.offsets[a.E] = start + mine;
  }
  off[tid] = start + before;
  const int64_t f0 = (int64_t)blockIdx.x * per_block * a.k;
  const int n = (int)min((int64_t)per_block * a.k, a.T * a.k - f0);
  for (int c0 = 0; c0 < n; c0 += 256) {
    const int i = c0 + tid;
    const bool live = i < n;
    const int e = live ? a.topk_idx[f0 + i] : 0;
    unsigned long long same = __ballot(live);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const unsigned long long m = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? m : ~m;
    }
    __syncthreads();   // off is there; the counts of the chunk before are used up
#pragma unroll
    for (int w = 0; w < 4; ++w) cnt[w][tid] = 0;
    __syncthreads();
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    if (live && rank == 0) cnt[wave][e] = __popcll(same);
    __syncthreads();
    if (live) {
      int32_t p = off[e] + rank;
      for (int w = 0; w < wave; ++w) p += cnt[w][e];
      a.sorted_rows[p] = (int32_t)(f0 + i);
    }
    __syncthreads();
    off[tid] += cnt[0][tid] + cnt[1][tid] + cnt[2][tid] + cnt[3][tid];
  }
}

// A slot's share of the gradient.  With w = scale * s the chosen scores'
// gradients are ds_j = scale dw_j; sigmoid dl = ds s (1 - s), softmax dl_e =
// s_e (ds_e - sum_j ds_j s_j).  Renormalised weights w_j = s_j / S take p_j =
// ds_j s_j = scale w_j (dw_j - sum_i dw_i w_i) instead: ds_j itself has a
// division by S and is infinite where the chosen scores are below 2^-1022
// though the weights are ordinary.  Sigmoid dl = p (1 - s), softmax dl_e = p_e
// - s_e sum_j p_j, and that sum is 0 since the w_j add up to 1.  Returns ds_j,
// or p_j with renorm (0 in slots that are not `on`); slots are the first 8
// lanes of a row.
__device__ __forceinline__ double slot_gradient(const RouteArgs& a, bool on, double sc, float dw) {
  const double d = on ? (double)a.scale * (double)dw : 0.0;
  if (!a.renorm) return d;
  const double total = sum8(sc), w = total == 0.0 ? 0.0 : sc / total, dot = sum8(d * w);
  return on ? w * (d - dot) : 0.0;
}
// The gradient of an expert with score s and slot sum g; mean = sum_j ds_j s_j,
// 0 with renorm.  A NaN score's gradient is NaN, chosen or not.  (g = 0: s
// (0 - mean) in both forms.)
template <bool RENORM>
__device__ __forceinline__ float expert_gradient(int sigmoid, double g, double s, double mean) {
  if (RENORM) return (float)(sigmoid ? g * (1.0 - s) : g - s * mean);
  return (float)(sigmoid ? g * s * (1.0 - s) : s * (g - mean));
}

// dlogits of one token per wave.  Scores in fp64, as in the choice, which
// bounds it: 2048 tokens x 256 experts in 4.5 us, 16384 in 17.7 (1.9 TB/s).
template <int NQ>
__global__ __launch_bounds__(256) void gate_bwd_kernel(RouteArgs a, const int32_t* __restrict__ idx,
                                                       const float* __restrict__ dw,
                                                       float* __restrict__ dlogits) {
  __shared__ TokenLds lds[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  float v[NQ];
  load_logits<NQ>(a, t, lane, v);
  const int e = lane < a.k ? idx[t * a.k + lane] : -1;   // all loads at the start
  const float d = lane < a.k ? dw[t * a.k + lane] : 0.0f;
  double s[NQ];
  token_scores<NQ>(v, a.E, lane, a.sigmoid, s);
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    if (NQ * lane + q < a.E) lds[wave].score[NQ * lane + q] = s[q];
  wave_lds_sync();
  const bool on = e >= 0 && e < a.E;
  const double sc = on ? lds[wave].score[e] : 0.0;
  const double ds = slot_gradient(a, on, sc, d);
  const double mean = a.sigmoid || a.renorm ? 0.0 : wave_sum(ds * sc);   // 0 past the slots
  double g[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) g[q] = 0.0;
  const int ej_of = on ? e : -1;
  const uint64_t ds_bits = __builtin_bit_cast(uint64_t, ds);
  for (int j = 0; j < a.k; ++j) {
    const int ej = __builtin_amdgcn_readlane(ej_of, j);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)ds_bits, j);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(ds_bits >> 32), j);
    const double dj = __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
#pragma unroll
    for (int q = 0; q < NQ; ++q) g[q] += NQ * lane + q == ej ? dj : 0.0;
  }
  Floats<NQ> o;
  if (a.renorm) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) o[q] = expert_gradient<true>(a.sigmoid, g[q], s[q], mean);
  } else {
#pragma unroll
    for (int q = 0; q < NQ; ++q) o[q] = expert_gradient<false>(a.sigmoid, g[q], s[q], mean);
  }
  float any = o[0];
#pragma unroll
  for (int q = 1; q < NQ; ++q) any += o[q];
  if (any != any) {   // hardly ever
#pragma unroll
    for (int q = 0; q < NQ; ++q) o[q] = one_nan(o[q]);
  }
  float* out = dlogits + t * a.E + NQ * lane;
  if (a.wide) {
    if (NQ * lane < a.E) *reinterpret_cast<Floats<NQ>*>(out) = o;
    return;
  }
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    if (NQ * lane + q < a.E) out[q] = o[q];
}

// The same, four tokens at a time in a wave, a row of 16 lanes each (E % 4 ==
// 0).  All that a choice changes is at the chosen experts: a lane writes its
// experts' gradients as if none were chosen to LDS, the slots' lanes put
// theirs over them.  A sigmoid is needed at the chosen experts alone.  8192 x
// 128 in 5.7 us (softmax), 16384 x 256 in 12.8 (2.6 TB/s), by sigmoids 7.8
// (4.3 TB/s, the memory's rate).
template <int NQ>
__global__ __launch_bounds__(256) void gate_bwd_rows_kernel(RouteArgs a, const int32_t* __restrict__ idx,
                                                            const float* __restrict__ dw,
                                                            float* __restrict__ dlogits) {
  __shared__ __align__(16) float lds[16][16 * NQ];
  const int lane = threadIdx.x & 63, r = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4), t = min(t0, a.T - 1);
  const float* row = a.logits + t * a.E;
  float v[NQ], *mine = lds[threadIdx.x >> 4];
  load_row<NQ>(row, a.E, r, v);
  const int e = r < a.k ? idx[t * a.k + r] : -1;
  const float d = r < a.k ? dw[t * a.k + r] : 0.0f;
  const bool on = e >= 0 && e < a.E;
  const float l = on ? row[e] : 0.0f;
  double s[NQ], inv = 0.0;
  float m = 0.0f;
  if (!a.sigmoid) inv = row_softmax<NQ>(v, a.E, r, m, s);
  const double sc = on ? one_score(a.sigmoid, l, m, inv) : 0.0;
  const double ds = slot_gradient(a, on, sc, d);
  double mean = 0.0;
  if (!a.sigmoid && !a.renorm) {
    mean = sum8(ds * sc);
    mean += dpp_swap<8>(mean);   // 0 past the slots
  }
  double g = 0.0;   // of all slots with this lane's expert
  for (int j = 0; j < a.k; ++j) {
    const double dj = __shfl(ds, (lane & 48) + j);
    g += __shfl(e, (lane & 48) + j) == e ? dj : 0.0;
  }
#pragma unroll
  for (int q = 0; q < NQ; q += 4) {
    Floats<4> o;
#pragma unroll
    for (int i = 0; i < 4; ++i)   // a NaN's derivative is NaN, chosen or not
      o[i] = a.sigmoid ? (v[q + i] != v[q + i] ? __uint_as_float(0x7FC00000u) : 0.0f) : (float)(s[q + i] * inv * (0.0 - mean));
    *reinterpret_cast<Floats<4>*>(mine + NQ * r + q) = o;
  }
  if (!(inv - inv == 0.0 && mean - mean == 0.0))   // softmax: a row of NaN, or with some
#pragma unroll
    for (int q = 0; q < NQ; ++q) mine[NQ * r + q] = one_nan(mine[NQ * r + q]);
  wave_lds_sync();
  if (on)
    mine[e] = one_nan(a.renorm ? expert_gradient<true>(a.sigmoid, g, sc, mean)
                               : expert_gradient<false>(a.sigmoid, g, sc, mean));
  wave_lds_sync();
  if (t0 >= a.T) return;
  float* out = dlogits + t * a.E;
#pragma unroll
  for (int q = 0; q < NQ; q += 4) {   // whole rows of 256 bytes at a time
    const int x = 4 * r + 16 * q;
    if (x < a.E) *reinterpret_cast<Floats<4>*>(out + x) = *reinterpret_cast<const Floats<4>*>(mine + x);
  }
}

// Tokens per workgroup of the choice, which has a histogram row for each: 16
// for every 4096 tokens of the batch or part of them, at most 256, so 1 to 16 a
// wave.  gate_kernel takes them one by one; gate_rows_kernel four at a time, so
// that up to 4096 tokens four of its 16 waves have some, and from 12289 on all.
// Whole routing with 1, 2, 4, 8, 16 a wave (us): 16384 tokens x 256
// experts 38.4, 27.3, 23.7 (taken), 35.4, 57.8; 4096 x 256 14.6 (taken), 16.3,
// 20.5, 31.8, 56.5; 65536 x 256 134, 93, 72, 65, 65 (taken).  Fewer leave the
// two later launches more histograms, more leave SIMDs empty.
static int gate_tokens(int64_t T) {
  const int64_t per_wave = (T + 4095) / 4096;
  return GATE_W * (int)(per_wave < 16 ? per_wave : 16);
}

int64_t gate_blocks(int64_t T) { return (T + gate_tokens(T) - 1) / gate_tokens(T); }
bool gate_adds(int64_t T) { return gate_blocks(T) <= 128; }
bool gate_in_one(int64_t T) { return T <= GATE_ONE_TOKENS; }

#define GATE_LAUNCH(kernel, ...)                         \
  do {                                                   \
    if (a.E <= 64)                                       \
      hipLaunchKernelGGL(kernel<1>, __VA_ARGS__);        \
    else if (a.E <= 128)                                 \
      hipLaunchKernelGGL(kernel<2>, __VA_ARGS__);        \
    else                                                 \
      hipLaunchKernelGGL(kernel<4>, __VA_ARGS__);        \
    return hipGetLastError();                            \
  } while (0)

hipError_t launch_gate_one(const RouteArgs& a, hipStream_t s) {
  GATE_LAUNCH(gate_one_kernel, dim3(1), dim3(64 * GATE_W), 0, s, a);
}

hipError_t launch_gate(const RouteArgs& a, int32_t* hist, hipStream_t s) {
  if (a.row_lanes) {
    const dim3 grid((unsigned)gate_blocks(a.T)), block(64 * GATE_W);
    if (a.E <= 64)
      hipLaunchKernelGGL(gate_rows_kernel<4>, grid, block, 0, s, a, gate_tokens(a.T), hist);
    else if (a.E <= 128)
      hipLaunchKernelGGL(gate_rows_kernel<8>, grid, block, 0, s, a, gate_tokens(a.T), hist);
    else
      hipLaunchKernelGGL(gate_rows_kernel<16>, grid, block, 0, s, a, gate_tokens(a.T), hist);
    return hipGetLastError();
  }
  GATE_LAUNCH(gate_kernel, dim3((unsigned)gate_blocks(a.T)), dim3(64 * GATE_W), 0, s, a,
              gate_tokens(a.T), hist);
}

hipError_t launch_gate_prefix(const RouteArgs& a, int32_t* hist, int32_t* total, hipStream_t s) {
  hipLaunchKernelGGL(gate_prefix_kernel, dim3((unsigned)a.E), dim3(256), 0, s, hist,
                     (int)gate_blocks(a.T), a.E, total);
  return hipGetLastError();
}

hipError_t launch_gate_scatter(const RouteArgs& a, const int32_t* base, const int32_t* total,
                               hipStream_t s) {
  hipLaunchKernelGGL(gate_scatter_kernel, dim3((unsigned)gate_blocks(a.T)), dim3(256), 0, s, a,
                     gate_tokens(a.T), base, total);
  return hipGetLastError();
}

hipError_t launch_gate_bwd(const RouteArgs& a, const int32_t* idx, const float* dw, float* dlogits,
                           hipStream_t s) {
  // four tokens a wave from 4096 tokens on (softmax, 256 experts, us: 2048
  // tokens 4.5 with one a wave, 6.2 with four; 6000: 8.1, 7.9; 16384: 17.7,
  // 12.8; sigmoid 4.0, 4.0; 7.4, 4.9; 16.0, 7.8)
  if (a.rows && a.T >= 4096) {
    const dim3 grid((unsigned)((a.T + 15) / 16)), block(256);
    if (a.E <= 64)
      hipLaunchKernelGGL(gate_bwd_rows_kernel<4>, grid, block, 0, s, a, idx, dw, dlogits);
    else if (a.E <= 128)
      hipLaunchKernelGGL(gate_bwd_rows_kernel<8>, grid, block, 0, s, a, idx, dw, dlogits);
    else
      hipLaunchKernelGGL(gate_bwd_rows_kernel<16>, grid, block, 0, s, a, idx, dw, dlogits);
    return hipGetLastError();
  }
  // a launch has 2^32 - 1 threads, a token takes 64
  constexpr int64_t PART = int64_t(1) << 25;
  if (a.T > PART) {
    RouteArgs b = a, rest = a;
    b.T = PART;
    rest.T = a.T - PART;
    rest.logits += PART * a.E;
    const hipError_t e = launch_gate_bwd(b, idx, dw, dlogits, s);
    if (e != hipSuccess) return e;
    return launch_gate_bwd(rest, idx + PART * a.k, dw + PART * a.k, dlogits + PART * a.E, s);
  }
  GATE_LAUNCH(gate_bwd_kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a, idx, dw, dlogits);
}

}  // namespace mxmoe
