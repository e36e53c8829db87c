// Routing from logits (gfx950): softmax or sigmoid scores, a selection bias,
// groups of experts, top-k, weights and the permutation plan; and the
// gradient of the weights with respect to the logits.
//
// One wave owns a token: lane l holds experts NQ l .. NQ l + NQ - 1 (NQ =
// ceil(E / 64)).  Scores are formed in fp64 and the choice is taken on
// c = fp32(s + bias), so that neighbours in the order do not change places
// with the rounding of an fp32 exponential.  The k largest come from k
// rounds of a wave maximum over integer keys.
#include "common.hpp"
#include "gate.hpp"
#include "launch.hpp"

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

__device__ __forceinline__ int32_t wave_max(int32_t v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = max(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
template <class F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
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

// Which groups are open to the choice, as a bit mask: lane g < groups
// values group g from the token's choice values in LDS and counts the
// groups that beat it.
__device__ __forceinline__ unsigned long long open_groups(const RouteArgs& a, const float* c,
                                                          int lane) {
  const int per = a.E / a.groups;
  int32_t key = INT32_MIN;
  if (lane < a.groups) {
    const float* p = c + lane * per;
    int32_t k1 = INT32_MIN, k2 = INT32_MIN;
    float c1 = 0.0f, c2 = 0.0f;
    for (int i = 0; i < per; ++i) {
      const float v = p[i];
      const int32_t kv = choice_key(v);
      if (kv > k1) {
        k2 = k1;
        c2 = c1;
        k1 = kv;
        c1 = v;
      } else if (kv > k2) {
        k2 = kv;
        c2 = v;
      }
    }
    key = choice_key(a.top2 && per > 1 ? c1 + c2 : c1);
  }
  int beaten = 0;
  for (int g = 0; g < a.groups; ++g) {
    const int32_t o = __shfl(key, g);
    beaten += o > key || (o == key && g < lane);
  }
  return __ballot(lane < a.groups && beaten < a.top_groups);
}

// Chooses token t's experts: lane j < k returns slot j's expert (others 0)
// and writes the slot's index and weight.
template <int NQ>
__device__ __forceinline__ int choose(const RouteArgs& a, int64_t t, int lane, TokenLds& lds) {
  const float* row = a.logits + t * a.E;
  float v[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) v[q] = row[min(NQ * lane + q, a.E - 1)];
  double s[NQ];
  token_scores<NQ>(v, a.E, lane, a.sigmoid, s);
  int32_t key[NQ];
  wave_lds_sync();   // the previous token's reads are done
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = NQ * lane + q;
    const float c = (float)(a.bias ? s[q] + (double)a.bias[min(e, a.E - 1)] : s[q]);
    key[q] = e < a.E ? choice_key(c) : INT32_MIN;
    if (e < a.E) {
      lds.score[e] = s[q];
      lds.c[e] = c;
    }
  }
  wave_lds_sync();
  if (a.top_groups < a.groups) {
    const unsigned long long open = open_groups(a, lds.c, lane);
    const int per = a.E / a.groups;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (!((open >> min((NQ * lane + q) / per, 63)) & 1)) key[q] = INT32_MIN;
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    int32_t best = key[0];
#pragma unroll
    for (int q = 1; q < NQ; ++q) best = max(best, key[q]);
    const int32_t top = wave_max(best);
    // the lowest lane that holds it, and its lowest such expert
    const int owner = __builtin_ctzll(__ballot(best == top));
    int at = 0;
#pragma unroll
    for (int q = NQ - 1; q >= 0; --q)
      if (key[q] == top) at = q;
    const int e = __builtin_amdgcn_readlane(NQ * lane + at, owner);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (NQ * lane + q == e) key[q] = INT32_MIN;
    if (lane == j) mine = e;
  }
  // weights: scores of the chosen experts, summed in slot order
  const double sc = lane < a.k ? lds.score[mine] : 0.0;
  double total = 1.0;
  if (a.renorm) {
    total = 0.0;
    for (int j = 0; j < a.k; ++j) total += __shfl(sc, j);
  }
  if (lane < a.k) {
    a.topk_idx[t * a.k + lane] = mine;
    a.topk_w[t * a.k + lane] = (float)(total == 0.0 ? 0.0 : sc / total * (double)a.scale);
  }
  return mine;
}

// The choice of `per_block` tokens by one workgroup of 4 waves, and the
// workgroup's histogram of experts.
template <int NQ>
__global__ __launch_bounds__(256) void gate_kernel(RouteArgs a, int per_block,
                                                   int32_t* __restrict__ hist_out) {
  __shared__ TokenLds lds[4];
  __shared__ int32_t hist[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  hist[tid] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * per_block;
  const int n = (int)min((int64_t)per_block, a.T - t0);
  for (int i = wave; i < n; i += 4) {
    const int e = choose<NQ>(a, t0 + i, lane, lds[wave]);
    if (lane < a.k) atomicAdd(&hist[e], 1);   // counts only: order does not matter
  }
  __syncthreads();
  if (tid < a.E) hist_out[(int64_t)blockIdx.x * a.E + tid] = hist[tid];
}

// Expert e = blockIdx.x: in place, hist[b][e] becomes the number of rows of
// e in workgroups before b; total[e] their sum.
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
// offsets[e] + rows of e in earlier workgroups + earlier rows of e here.
__global__ __launch_bounds__(256) void gate_scatter_kernel(RouteArgs a, int per_block,
                                                           const int32_t* __restrict__ base,
                                                           const int32_t* __restrict__ total) {
  __shared__ int32_t off[256];
  __shared__ int32_t ex[256];
  const int tid = threadIdx.x;
  const int32_t mine = tid < a.E ? total[tid] : 0;
  off[tid] = mine;
  __syncthreads();
  for (int d = 1; d < 256; d <<= 1) {
    const int32_t o = tid >= d ? off[tid - d] : 0;
    __syncthreads();
    off[tid] += o;
    __syncthreads();
  }
  const int32_t start = off[tid] - mine;
  if (blockIdx.x == 0) {
    if (tid < a.E) a.offsets[tid] = start;
    if (tid == a.E - 1) a.offsets[a.E] = off[tid];
  }
  __syncthreads();
  if (tid < a.E) off[tid] = start + base[(int64_t)blockIdx.x * a.E + tid];
  const int64_t f0 = (int64_t)blockIdx.x * per_block * a.k;
  const int n = (int)min((int64_t)per_block * a.k, a.T * a.k - f0);
  for (int c0 = 0; c0 < n; c0 += 256) {
    const int i = c0 + tid;
    const int e = i < n ? a.topk_idx[f0 + i] : -1;
    __syncthreads();
    ex[tid] = e;
    __syncthreads();
    if (e >= 0) {
      int rank = 0;
      for (int j = 0; j < tid; ++j) rank += ex[j] == e;
      a.sorted_rows[off[e] + rank] = (int32_t)(f0 + i);
    }
    __syncthreads();
    // the chunk's counts move the places on (one thread per expert)
    if (c0 + 256 < n && tid < a.E) {
      int cnt = 0;
      for (int j = 0; j < 256; ++j) cnt += ex[j] == tid;
      off[tid] += cnt;
    }
  }
}

// dlogits of one token per wave.  With w = scale * s / S (renorm) the
// chosen scores' gradients are ds_j = scale (dw_j - sum_i dw_i s_i / S) / S,
// else ds_j = scale dw_j; sigmoid dl = ds s (1 - s), softmax dl_e =
// s_e (ds_e - sum_j ds_j s_j).  Scores in fp64, as in the choice.
template <int NQ>
__global__ __launch_bounds__(256) void gate_bwd_kernel(RouteArgs a, const int32_t* __restrict__ idx,
                                                       const float* __restrict__ dw,
                                                       float* __restrict__ dlogits) {
  __shared__ TokenLds lds[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  float v[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) v[q] = a.logits[t * a.E + min(NQ * lane + q, a.E - 1)];
  double s[NQ];
  token_scores<NQ>(v, a.E, lane, a.sigmoid, s);
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    if (NQ * lane + q < a.E) lds[wave].score[NQ * lane + q] = s[q];
  wave_lds_sync();
  const int e = lane < a.k ? idx[t * a.k + lane] : -1;
  const bool on = e >= 0 && e < a.E;
  const double sc = on ? lds[wave].score[e] : 0.0;
  double ds = on ? (double)a.scale * (double)dw[t * a.k + lane] : 0.0;
  if (a.renorm) {
    const double total = wave_sum(sc), dot = wave_sum(ds * sc);
    ds = on && total != 0.0 ? (ds - dot / total) / total : 0.0;
  }
  const double mean = a.sigmoid ? 0.0 : wave_sum(ds * sc);
  double g[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) g[q] = 0.0;
  for (int j = 0; j < a.k; ++j) {
    const int ej = __shfl(on ? e : -1, j);
    const double dj = __shfl(ds, j);
#pragma unroll
    for (int q = 0; q < NQ; ++q) g[q] += NQ * lane + q == ej ? dj : 0.0;
  }
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int x = NQ * lane + q;
    if (x < a.E)
      dlogits[t * a.E + x] = (float)(a.sigmoid ? g[q] * s[q] * (1.0 - s[q]) : s[q] * (g[q] - mean));
  }
}

// Tokens per workgroup: the plan has one histogram row for each workgroup.
static int gate_tokens(int64_t T) { return T <= 4096 ? 16 : 64; }

int64_t gate_blocks(int64_t T) { return (T + gate_tokens(T) - 1) / gate_tokens(T); }

hipError_t launch_gate(const RouteArgs& a, int32_t* hist, hipStream_t s) {
  const int per = gate_tokens(a.T);
  const dim3 grid((unsigned)gate_blocks(a.T)), block(256);
  if (a.E <= 64)
    hipLaunchKernelGGL(gate_kernel<1>, grid, block, 0, s, a, per, hist);
  else if (a.E <= 128)
    hipLaunchKernelGGL(gate_kernel<2>, grid, block, 0, s, a, per, hist);
  else
    hipLaunchKernelGGL(gate_kernel<4>, grid, block, 0, s, a, per, hist);
  return hipGetLastError();
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
  const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
  if (a.E <= 64)
    hipLaunchKernelGGL(gate_bwd_kernel<1>, grid, block, 0, s, a, idx, dw, dlogits);
  else if (a.E <= 128)
    hipLaunchKernelGGL(gate_bwd_kernel<2>, grid, block, 0, s, a, idx, dw, dlogits);
  else
    hipLaunchKernelGGL(gate_bwd_kernel<4>, grid, block, 0, s, a, idx, dw, dlogits);
  return hipGetLastError();
}

}  // namespace mxmoe
