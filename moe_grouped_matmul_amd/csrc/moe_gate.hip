// Router of a mixture-of-experts layer for gfx950: from logits l[T][E] the k
// experts of each token, their weights, the experts' loads and the balance
// loss, and the gradient.
//
//   p = softmax(l);  S = the k largest logits of a row (equal ones: the lower
//   expert first; -inf and NaN are never chosen)
//   w_j = scale * p_j / sum_S p (renorm) or scale * p_j
//   c_e = choices of expert e, n = tokens with a choice, C = sum_e c_e,
//   P_e = sum_t p_te,  loss = coef * E / (C n) * sum_e c_e P_e
//
// A token that `valid` marks 0 or whose logits are all -inf has no expert
// (idx -1, w 0) and enters no sum.  A row that holds a NaN or +inf has NaN
// probabilities, and so NaN weights and a NaN loss.
//
// The gradient of sum(dw * w) + dloss * loss, the counts being constants:
//   dl_e = p_e (g_e - sum p g - [not renorm] sum_j w_j dw_j) + [e = S_j] w_j (dw_j - [renorm] sum_i w_i dw_i / scale),
//   g_e = dloss * coef * E c_e / (C n).
//
// A row is held by LPT lanes, VPL consecutive experts each, so the lowest lane
// with the largest value holds the lowest expert.  Each of k rounds takes the
// maximum over the lanes' own maxima (float bits ordered as integers) and
// removes it.  Probabilities are summed per lane over the tokens it handles,
// per workgroup in LDS, and over workgroups in a fixed order, so results do
// not depend on scheduling.

#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

constexpr int kGateThreads = 256;
constexpr int kGateMaxBlocks = 256;
constexpr int kGateMaxE = 1024;

// order-preserving integer of a float, 0 for values that are never chosen (-inf, NaN)
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 becomes +0: equal logits, equal keys
  const uint32_t key = u & 0x80000000u ? ~u : u | 0x80000000u;
  return f > -__builtin_inff() ? key : 0u;  // false for NaN too
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
}

template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) {
    const uint32_t u = __shfl_xor(v, o);
    v = u > v ? u : v;
  }
  return v;
}

// workspace of a launch of `blocks` workgroups: counts [blocks][E + 1], then sums [blocks][E]
template <int LPT, int VPL, bool BF16>
__global__ void __launch_bounds__(kGateThreads) gate_kernel(GateParams p) {
  constexpr int GPB = kGateThreads / LPT;  // tokens at a time
  __shared__ int cnt[kGateMaxE + 1];
  __shared__ float psum[kGateThreads / 64][kGateMaxE];
  const int E = p.E;
  const int sub = threadIdx.x % LPT;
  const int grp = threadIdx.x / LPT;
  for (int e = threadIdx.x; e <= E; e += kGateThreads) cnt[e] = 0;
  __syncthreads();
  float sum[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) sum[v] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < p.T; t0 += (int64_t)gridDim.x * GPB) {
    const int64_t t = t0 + grp;
    const bool live = t < p.T && (!p.valid || p.valid[t] != 0);
    float l[VPL];
    uint32_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = sub * VPL + v;
      l[v] = live && e < E ? load_logit<BF16>(p.logits, t * E + e) : -__builtin_inff();
      key[v] = order_key(l[v]);
    }
    uint32_t mkey = 0;
    int my_idx = -1;       // lane j < k: the j-th choice
    uint32_t my_key = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0;
      int bv = 0;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (key[v] > best) {
          best = key[v];
          bv = v;
        }
      const uint32_t top = group_max<LPT>(best);
      if (j == 0) mkey = top;
      // the lowest lane of the group that holds it
      unsigned long long who = __ballot(best == top && top != 0);
      if constexpr (LPT < 64) who = (who >> ((threadIdx.x & 63) / LPT * LPT)) & ((1ull << LPT) - 1ull);
      const int win = who ? __builtin_ctzll(who) : 0;
      const int e = __shfl(sub * VPL + bv, ((threadIdx.x & 63) / LPT) * LPT + win);
      if (who && sub == win) {
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          if (v == bv) key[v] = 0;
      }
      if (who && sub == j) {
        my_idx = e;
        my_key = top;
      }
    }
    const float m = mkey ? key_value(mkey) : 0.f;
    float ex[VPL];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      ex[v] = expf(l[v] - m);
      s += ex[v];
    }
    s = group_sum<LPT>(s);
    const float mine = my_idx >= 0 ? expf(key_value(my_key) - m) : 0.f;
    const float chosen = group_sum<LPT>(mine);
    const float inv = s > 0.f ? 1.0f / s : (s == s ? 0.f : s);  // no choice: 0; NaN stays NaN
#pragma unroll
    for (int v = 0; v < VPL; ++v) sum[v] += ex[v] * inv;
    if (t < p.T && sub < p.k) {
      // a NaN sum makes the weights NaN in either form
      const float den = p.renorm ? (s == s ? chosen : s) : s;
      p.idx[t * p.k + sub] = my_idx;
      p.w[t * p.k + sub] = s != s ? s : (my_idx >= 0 ? p.w_scale * (mine / den) : 0.f);
      if (my_idx >= 0) atomicAdd(&cnt[my_idx], 1);
      if (sub == 0 && my_idx >= 0) atomicAdd(&cnt[E], 1);
    }
  }
  // lanes of a wave that hold the same experts, then waves, in order
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
#pragma unroll
    for (int o = LPT; o < 64; o <<= 1) sum[v] += __shfl_xor(sum[v], o);
    const int e = sub * VPL + v;
    if ((threadIdx.x & 63) < LPT && e < E) psum[threadIdx.x >> 6][e] = sum[v];
  }
  __syncthreads();
  int* wc = static_cast<int*>(p.ws) + (int64_t)blockIdx.x * (E + 1);
  float* wp = reinterpret_cast<float*>(static_cast<int*>(p.ws) + (int64_t)gridDim.x * (E + 1)) + (int64_t)blockIdx.x * E;
  for (int e = threadIdx.x; e <= E; e += kGateThreads) {
    wc[e] = cnt[e];
    if (e < E) wp[e] = (psum[0][e] + psum[1][e]) + (psum[2][e] + psum[3][e]);
  }
}

// one workgroup: sums over the blocks in order, and the loss
__global__ void __launch_bounds__(1024) gate_reduce_kernel(GateParams p, int blocks) {
  __shared__ float part[16], part_c[16];
  const int E = p.E;
  const int* wc = static_cast<const int*>(p.ws);
  const float* wp = reinterpret_cast<const float*>(wc + (int64_t)blocks * (E + 1));
  const int e = threadIdx.x;
  float s = 0.f;
  int c = 0, n = 0;
  if (e < E)
    for (int b = 0; b < blocks; ++b) {
      s += wp[(int64_t)b * E + e];
      c += wc[(int64_t)b * (E + 1) + e];
    }
  for (int b = 0; b < blocks; ++b) n += wc[(int64_t)b * (E + 1) + E];
  if (e < E) {
    p.prob_sum[e] = s;
    p.counts[e] = c;
  }
  if (e == 0) p.counts[E] = n;
  float x = (float)c * s, y = (float)c;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    x += __shfl_xor(x, o);
    y += __shfl_xor(y, o);
  }
  if ((e & 63) == 0) {
    part[e >> 6] = x;
    part_c[e >> 6] = y;
  }
  __syncthreads();
  if (e == 0) {
    float a = 0.f, C = 0.f;
    for (int i = 0; i < 16; ++i) {
      a += part[i];
      C += part_c[i];
    }
    *p.loss = n > 0 ? p.coef * (float)E * (a / (C * (float)n)) : a;  // nothing routed: 0 (or NaN)
  }
}

template <int LPT, int VPL, bool BF16>
__global__ void __launch_bounds__(kGateThreads) gate_bwd_kernel(GateBwdParams p) {
  constexpr int GPB = kGateThreads / LPT;
  __shared__ float part[4];
  const int E = p.E;
  const int sub = threadIdx.x % LPT;
  const int grp = threadIdx.x / LPT;
  // C = sum of the counts
  float C = 0.f;
  for (int e = threadIdx.x; e < E; e += kGateThreads) C += (float)p.counts[e];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) C += __shfl_xor(C, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = C;
  __syncthreads();
  C = (part[0] + part[1]) + (part[2] + part[3]);
  const float n = (float)p.counts[E];
  const float f = p.dloss && n > 0.f ? *p.dloss * p.coef * (float)E / (C * n) : 0.f;
  float g[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = sub * VPL + v;
    g[v] = e < E ? f * (float)p.counts[e] : 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < p.T; t0 += (int64_t)gridDim.x * GPB) {
    const int64_t t = t0 + grp;
    const bool in = t < p.T;
    const bool have = in && sub < p.k;
    const int idx = have ? p.idx[t * p.k + sub] : -1;
    const bool live = __shfl(idx, ((threadIdx.x & 63) / LPT) * LPT) >= 0;  // the first choice exists
    const float w = have && idx >= 0 ? p.w[t * p.k + sub] : 0.f;
    const float dw = have && idx >= 0 && p.dw ? p.dw[t * p.k + sub] : 0.f;
    float l[VPL];
    float m = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = sub * VPL + v;
      l[v] = live && e < E ? load_logit<BF16>(p.logits, t * E + e) : -__builtin_inff();
      m = fmaxf(m, l[v]);
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (!live) m = 0.f;
    float ex[VPL];
    float s = 0.f, pg = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      ex[v] = expf(l[v] - m);
      s += ex[v];
      pg = __builtin_fmaf(ex[v], g[v], pg);
    }
    s = group_sum<LPT>(s);
    pg = group_sum<LPT>(pg);
    const float dot = group_sum<LPT>(w * dw);
    const float inv = live ? 1.0f / s : 0.f;
    const float base = pg * inv + (p.renorm ? 0.f : dot);
    const float own = p.renorm ? w * (dw - dot / p.w_scale) : w * dw;
    float d[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] = ex[v] * inv * (g[v] - base);
    for (int j = 0; j < p.k; ++j) {
      const int src = ((threadIdx.x & 63) / LPT) * LPT + j;
      const int e = __shfl(idx, src) - sub * VPL;
      const float a = __shfl(own, src);
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (v == e) d[v] += a;
    }
    if (in) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int e = sub * VPL + v;
        if (e < E) {
          if constexpr (BF16) static_cast<uint16_t*>(p.dlogits)[t * E + e] = f32_to_bf16_rne(d[v]);
          else static_cast<float*>(p.dlogits)[t * E + e] = d[v];
        }
      }
    }
  }
}

// lanes per token and values per lane of E experts
#define DG_GATE_SHAPES(X)            \
  if (p.E <= 64) { X(16, 4); }       \
  else if (p.E <= 128) { X(16, 8); } \
  else if (p.E <= 256) { X(16, 16); } \
  else if (p.E <= 512) { X(64, 8); } \
  else { X(64, 16); }

int gate_blocks(int64_t T, int64_t E) {
  const int64_t per = kGateThreads / (E <= 256 ? 16 : 64);
  const int64_t b = (T + per - 1) / per;
  return (int)(b < 1 ? 1 : (b < kGateMaxBlocks ? b : kGateMaxBlocks));
}

}  // namespace

size_t gate_workspace_bytes(int64_t T, int64_t E) { return (size_t)gate_blocks(T, E) * (size_t)(2 * E + 1) * 4; }

hipError_t launch_gate(const GateParams& p, bool bf16, hipStream_t stream) {
  const int blocks = gate_blocks(p.T, p.E);
#define X(L, V)                                                                                                   \
  if (bf16) hipLaunchKernelGGL((gate_kernel<L, V, true>), dim3(blocks), dim3(kGateThreads), 0, stream, p);        \
  else hipLaunchKernelGGL((gate_kernel<L, V, false>), dim3(blocks), dim3(kGateThreads), 0, stream, p)
  DG_GATE_SHAPES(X)
#undef X
  hipLaunchKernelGGL(gate_reduce_kernel, dim3(1), dim3(1024), 0, stream, p, blocks);
  return hipGetLastError();
}

hipError_t launch_gate_bwd(const GateBwdParams& p, bool bf16, hipStream_t stream) {
  const int64_t per = kGateThreads / (p.E <= 256 ? 16 : 64);
  const int64_t b = (p.T + per - 1) / per;
  const int blocks = (int)(b < 4096 ? b : 4096);
#define X(L, V)                                                                                                   \
  if (bf16) hipLaunchKernelGGL((gate_bwd_kernel<L, V, true>), dim3(blocks), dim3(kGateThreads), 0, stream, p);    \
  else hipLaunchKernelGGL((gate_bwd_kernel<L, V, false>), dim3(blocks), dim3(kGateThreads), 0, stream, p)
  DG_GATE_SHAPES(X)
#undef X
  return hipGetLastError();
}

}  // namespace dg
