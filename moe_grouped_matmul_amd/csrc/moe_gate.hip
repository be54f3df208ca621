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
// A row is held by LPT lanes (16 up to 256 experts, else 64), each with VPL of
// its values in 16-byte pieces, so every load and store is contiguous across
// lanes.  A logit and its expert become one unique ordered key (bf16: 16 + 16
// bits as an integer; fp32: 32 + 10 bits in the mantissa of a double, whose
// maximum and minimum are single instructions), larger for larger logits and,
// of equal ones, for the lower expert.  Every lane sorts its keys once; a round
// takes the maximum of the lanes' first keys over the row (DPP, no LDS) and its
// owner drops it.
//
// Probabilities are summed per lane over the tokens it handles, per workgroup
// in LDS, then over groups of 16 workgroups and over the groups, each by the
// last workgroup to arrive (agent-scope counters, coherent partials) and in a
// fixed order, so results do not depend on scheduling.
//
// Bounds.  Forward, 32768 x 256 fp32, k = 8: 23 us, of which the logits' bytes
// at the copy rate are 7 and the tail over workgroups about 6.  The vector units
// (sorting and k rounds over 16 values per lane) are busy 0.67 of the cycles; a
// CU holds one workgroup of 16 waves in phase, so a pass's loads and the tail
// have no other work under them, and a wave waits 0.60 of its cycles (131 us
// with a wave per token and no sorted keys, 26 with 16 lanes; 22-bit keys in 32
// bits with the expert in the low ones and a second comparison 29).  64 x 256
// bf16: 7.3 us, all 64 tokens in one workgroup, four waves a SIMD one after
// another through a chain of dependent steps.  Gradient: memory, 17 us for 67
// MB (3.9 TB/s).

#include "dg_internal.hpp"
#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

constexpr int kGateThreads = 1024;
constexpr int kGateWaves = kGateThreads / 64;
constexpr int kGateFan = 16;  // workgroups per group, groups
constexpr int kGateMaxBlocks = kGateFan * kGateFan;
constexpr int kBwdThreads = 256;

// ---- keys.  -inf and NaN (read as -inf) sort below every number; 0 is an
// empty place; neither is ever chosen: some(key) is false for both.
template <bool BF16>
struct Keys;

// order-preserving bits of a float, -0 as +0 (equal logits, equal keys), NaN as -inf
__device__ __forceinline__ uint32_t ordered(float f) {
  const int32_t u = (int32_t)__float_as_uint(fmaxf(f + 0.0f, -__builtin_inff()));
  return (uint32_t)(u ^ ((u >> 31) | (int32_t)0x80000000));
}

template <>
struct Keys<true> {
  typedef uint32_t T;
  static __device__ __forceinline__ T make(float f, int e) {
    return (ordered(f) & 0xffff0000u) | (0xffffu - (uint32_t)e);
  }
  static __device__ __forceinline__ bool some(T k) { return k >= 0x00800000u; }
  static __device__ __forceinline__ float value(T k) {
    const uint32_t o = k >> 16;
    return __uint_as_float((o & 0x8000u ? o & 0x7fffu : ~o & 0xffffu) << 16);
  }
  static __device__ __forceinline__ int expert(T k) { return (int)(0xffffu - (k & 0xffffu)); }
  static __device__ __forceinline__ T max(T a, T b) { return a > b ? a : b; }
  static __device__ __forceinline__ T min(T a, T b) { return a < b ? a : b; }
  template <int C>
  static __device__ __forceinline__ T dpp(T a) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, C, 0xf, 0xf, true);
  }
  static __device__ __forceinline__ T far(T a, int o) { return __shfl_xor(a, o); }
};

template <>
struct Keys<false> {
  typedef double T;
  static __device__ __forceinline__ T make(float f, int e) {
    const uint32_t o = ordered(f);
    const uint32_t hi = __builtin_amdgcn_alignbit(0x3ff00000u >> 10, o, 22);  // exponent of 1.0, then o's upper 10 bits
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | ((o << 10) | (uint32_t)(1023 - e)));
  }
  static __device__ __forceinline__ bool some(T k) {
    return k >= __builtin_bit_cast(double, 0x3ff0000000000000ull | ((uint64_t)0x00800000u << 10));
  }
  static __device__ __forceinline__ float value(T k) {
    const uint32_t o = (uint32_t)(__builtin_bit_cast(uint64_t, k) >> 10);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
  }
  static __device__ __forceinline__ int expert(T k) { return 1023 - (int)(__builtin_bit_cast(uint64_t, k) & 1023u); }
  // no NaN among the keys
  static __device__ __forceinline__ T max(T a, T b) { return __builtin_fmax(a, b); }
  static __device__ __forceinline__ T min(T a, T b) { return __builtin_fmin(a, b); }
  template <int C>
  static __device__ __forceinline__ T dpp(T a) {
    const uint64_t b = __builtin_bit_cast(uint64_t, a);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, C, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), C, 0xf, 0xf, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  }
  static __device__ __forceinline__ T far(T a, int o) { return __shfl_xor(a, o); }
};

// DPP controls that exchange lanes inside a row of 16: pairs, pairs of pairs,
// the quads of a half row, the half rows (each step's partner group is uniform
// inside, so mirroring serves as well as an exclusive-or)
constexpr int kDpp1 = 0xB1, kDpp2 = 0x4E, kDpp4 = 0x141, kDpp8 = 0x140;

template <int LPT, bool BF16>
__device__ __forceinline__ typename Keys<BF16>::T group_max(typename Keys<BF16>::T v) {
  typedef Keys<BF16> K;
  v = K::max(v, K::template dpp<kDpp1>(v));
  v = K::max(v, K::template dpp<kDpp2>(v));
  v = K::max(v, K::template dpp<kDpp4>(v));
  v = K::max(v, K::template dpp<kDpp8>(v));
  if constexpr (LPT == 64) {
    v = K::max(v, K::far(v, 16));
    v = K::max(v, K::far(v, 32));
  }
  return v;
}
// sum over the four rows of 16 lanes
__device__ __forceinline__ float rows_sum(float v) {
  const uint32_t a = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);  // each pair of rows: the even one, the odd one
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const uint32_t b = __float_as_uint(v);
  const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
template <int C>
__device__ __forceinline__ float dppf(float a) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(a), C, 0xf, 0xf, true));
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  v += dppf<kDpp1>(v);
  v += dppf<kDpp2>(v);
  v += dppf<kDpp4>(v);
  v += dppf<kDpp8>(v);
  if constexpr (LPT == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_fmax(float v) {
  v = fmaxf(v, dppf<kDpp1>(v));
  v = fmaxf(v, dppf<kDpp2>(v));
  v = fmaxf(v, dppf<kDpp4>(v));
  v = fmaxf(v, dppf<kDpp8>(v));
  if constexpr (LPT == 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
}

// e^x for x <= 0 (NaN stays NaN): 2^n 2^f with n the integer nearest x log2 e
// and f = x log2 e - n, with log2 e in two parts: f is off by two roundings of
// a number of at most a half, 2^-24, wherever x lies, and e^x by 3 x 2^-24
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kHigh = 1.44269502f, kLow = 1.92596303e-8f;  // log2 e
  x = __builtin_elementwise_maximum(x, -200.f);
  const float n = __builtin_rintf(x * kHigh);
  const float f = __builtin_fmaf(x, kLow, __builtin_fmaf(x, kHigh, -n));
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

template <bool BF16, int M>
__device__ __forceinline__ void cmp_swap(typename Keys<BF16>::T (&a)[M], int i, int j) {  // the larger first
  const typename Keys<BF16>::T x = Keys<BF16>::max(a[i], a[j]), y = Keys<BF16>::min(a[i], a[j]);
  a[i] = x;
  a[j] = y;
}
// odd-even merge sort of a[LO .. LO + N), descending; merge: of the elements
// LO, LO + R, ... whose odd and even halves are sorted
template <bool BF16, int LO, int N, int R, int M>
__device__ __forceinline__ void merge_desc(typename Keys<BF16>::T (&a)[M]) {
  if constexpr (2 * R < N) {
    merge_desc<BF16, LO, N, 2 * R>(a);
    merge_desc<BF16, LO + R, N, 2 * R>(a);
#pragma unroll
    for (int i = LO + R; i + R < LO + N; i += 2 * R) cmp_swap<BF16>(a, i, i + R);
  } else {
    cmp_swap<BF16>(a, LO, LO + R);
  }
}
template <bool BF16, int LO, int N, int M>
__device__ __forceinline__ void sort_desc(typename Keys<BF16>::T (&a)[M]) {
  if constexpr (N > 1) {
    sort_desc<BF16, LO, N / 2>(a);
    sort_desc<BF16, LO + N / 2, N / 2>(a);
    merge_desc<BF16, LO, N, 1>(a);
  }
}

// the row values of this lane: value v is expert ((v / VEC) LPT + sub) VEC + v % VEC; out of range: -inf
template <int LPT, int VPL, bool BF16>
struct Row {
  static constexpr int VEC = BF16 ? 8 : 4;
  static __device__ __forceinline__ int expert(int sub, int v) { return ((v / VEC) * LPT + sub) * VEC + v % VEC; }
  // whole: E is a multiple of VEC, so every piece is inside or outside the row and 16-byte aligned
  static __device__ __forceinline__ void load(const void* p, int64_t t, int E, int sub, bool live, bool whole, float* l) {
#pragma unroll
    for (int c = 0; c < VPL / VEC; ++c) {
      const int e = expert(sub, c * VEC);
      float* o = l + c * VEC;
      // values outside the row (or of no token) are read at element 0 instead and replaced
      if (whole) {
        const bool in = live && e < E;
        const int64_t at = in ? t * E + e : 0;
        if constexpr (BF16) {
          const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
          o[0] = __uint_as_float(w.x << 16); o[1] = __uint_as_float(w.x & 0xffff0000u);
          o[2] = __uint_as_float(w.y << 16); o[3] = __uint_as_float(w.y & 0xffff0000u);
          o[4] = __uint_as_float(w.z << 16); o[5] = __uint_as_float(w.z & 0xffff0000u);
          o[6] = __uint_as_float(w.w << 16); o[7] = __uint_as_float(w.w & 0xffff0000u);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
          o[0] = w.x; o[1] = w.y; o[2] = w.z; o[3] = w.w;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = in ? o[i] : -__builtin_inff();
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const bool in = live && e + i < E;
          const int64_t at = in ? t * E + e + i : 0;
          float x;
          if constexpr (BF16) x = __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[at] << 16);
          else x = static_cast<const float*>(p)[at];
          o[i] = in ? x : -__builtin_inff();
        }
      }
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t t, int E, int sub, bool whole, const float* d) {
#pragma unroll
    for (int c = 0; c < VPL / VEC; ++c) {
      const int e = expert(sub, c * VEC);
      const int64_t at = t * E + e;
      const float* o = d + c * VEC;
      if (whole) {
        if (e < E) {
          if constexpr (BF16)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = uint4{
                pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
          else
            *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(o[0], o[1], o[2], o[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (e + i < E) {
            if constexpr (BF16) static_cast<uint16_t*>(p)[at + i] = f32_to_bf16_rne(o[i]);
            else static_cast<float*>(p)[at + i] = o[i];
          }
      }
    }
  }
};

// One arrival at `counter`; true for the whole workgroup that is the last of
// n.  Every wave's coherent stores are acknowledged before the arrival, and
// the last workgroup reads only after it; the counter is left at zero.
__device__ __forceinline__ bool last_arrival(unsigned int* counter, unsigned int n, int* flag) {
  wait_vmcnt<0>();
  __syncthreads();
  if (threadIdx.x == 0) {
    *flag = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
    if (*flag) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *flag != 0;
}

// workspace: counters (the root's, then one per group) in the bytes that every
// operator keeps its counters in, [blocks][2 E + 1] partials of workgroups
// (sums, then counts), [groups][2 E + 1] of groups
template <int LPT, int VPL, int KCAP, bool BF16>
__global__ void __launch_bounds__(kGateThreads) gate_kernel(GateParams p) {
  typedef Keys<BF16> KT;
  typedef typename KT::T Key;
  typedef Row<LPT, VPL, BF16> R;
  constexpr int GPB = kGateThreads / LPT;  // tokens at a time
  constexpr int EMAX = LPT * VPL;
  constexpr int L = VPL < KCAP ? VPL : KCAP;  // keys a lane may lose
  __shared__ int cnt[EMAX + 1];
  __shared__ float psum[kGateWaves][EMAX];
  __shared__ float red[2][kGateWaves];
  __shared__ int flag;
  const int E = p.E;
  const int sub = threadIdx.x % LPT;
  const int grp = threadIdx.x / LPT;
  const int wave = threadIdx.x >> 6;
  const bool whole = E % R::VEC == 0;
  for (int e = threadIdx.x; e <= E; e += kGateThreads) cnt[e] = 0;
  __syncthreads();
  float sum[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) sum[v] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < p.T; t0 += (int64_t)gridDim.x * GPB) {
    const int64_t t = t0 + grp;
    const bool live = t < p.T && (!p.valid || p.valid[t] != 0);
    float l[VPL];
    int row = E;
    asm volatile("" : "+s"(row));  // compared anew for each token: kept across the loop, the masks of the values spill
    R::load(p.logits, t, row, sub, live, whole, l);
    Key key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) key[v] = KT::make(l[v], R::expert(sub, v));
    if constexpr (L < VPL) {  // 16 values, 8 wanted: sort the halves, keep the larger 8, merge
      static_assert(VPL == 16 && L == 8, "shapes of the kernel");
      sort_desc<BF16, 0, 8>(key);
      sort_desc<BF16, 8, 8>(key);
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = KT::max(key[i], key[15 - i]);
#pragma unroll
      for (int h = 4; h >= 1; h /= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((i & h) == 0) cmp_swap<BF16>(key, i, i + h);
    } else {
      sort_desc<BF16, 0, VPL>(key);
    }
    float m = 0.f;
    Key mine = 0;  // lane j < k: the j-th choice
#pragma unroll
    for (int j = 0; j < KCAP; ++j) {
      if (j < p.k) {  // uniform
        const Key top = group_max<LPT, BF16>(key[0]);
        const bool win = key[0] == top;
        // what round j leaves at place i > KCAP - 2 - j no later round reads
#pragma unroll
        for (int i = 0; i < L && i < KCAP - 1 - j; ++i) {  // values first: a choice of array elements would be a variable index
          const Key a = key[i], b = i + 1 < L ? key[i + 1 < L ? i + 1 : 0] : Key(0);
          key[i] = win ? b : a;
        }
        if (j == 0 && KT::some(top)) m = KT::value(top);
        if (sub == j) mine = top;
      }
    }
    float ex[VPL];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      ex[v] = exp_neg(l[v] - m);
      s += ex[v];
    }
    s = group_sum<LPT>(s);
    const bool have = KT::some(mine);
    const float em = have ? exp_neg(KT::value(mine) - m) : 0.f;
    const float den = p.renorm ? group_sum<LPT>(em) : s;
    const float inv = s > 0.f ? 1.0f / s : (s == s ? 0.f : s);  // no choice: 0; NaN stays NaN
#pragma unroll
    for (int v = 0; v < VPL; ++v) sum[v] = __builtin_fmaf(ex[v], inv, sum[v]);
    if (t < p.T && sub < p.k) {
      const int e = have ? KT::expert(mine) : -1;
      p.idx[t * p.k + sub] = e;
      p.w[t * p.k + sub] = s != s ? s : (have ? p.w_scale * (em / den) : 0.f);
      if (have) atomicAdd(&cnt[e], 1);
      if (have && sub == 0) atomicAdd(&cnt[E], 1);
    }
  }
  // lanes of a wave that hold the same experts, then waves, in order
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float x = sum[v];
    if constexpr (LPT == 16) x = rows_sum(x);
    if ((threadIdx.x & 63) < LPT) psum[wave][R::expert(sub, v)] = x;
  }
  __syncthreads();
  if (threadIdx.x < E) {  // E <= 1024 = kGateThreads
    float x = psum[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kGateWaves; ++w) x += psum[w][threadIdx.x];
    psum[0][threadIdx.x] = x;
  }
  __syncthreads();
  const int blocks = (int)gridDim.x;
  if (blocks > 1) {
    // item i: sum of expert i (i < E), else count i - E (the last: tokens)
    const int items = 2 * E + 1;
    const int groups = (blocks + kGateFan - 1) / kGateFan;
    unsigned int* root = static_cast<unsigned int*>(p.ws);
    uint32_t* part = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.ws) + kWsCounterBytes);
    uint32_t* gpart = part + (int64_t)blocks * items;
    const int g = (int)blockIdx.x / kGateFan;
    const int members = blocks - g * kGateFan < kGateFan ? blocks - g * kGateFan : kGateFan;
    auto put = [&](uint32_t* to) {
      for (int i = threadIdx.x; i < items; i += kGateThreads)
        __hip_atomic_store(to + i, i < E ? __float_as_uint(psum[0][i]) : (uint32_t)cnt[i - E], __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    };
    auto take = [&](const uint32_t* from, int n) {  // sums of n partials into LDS, in order
      for (int i = threadIdx.x; i < items; i += kGateThreads) {
        uint32_t u[kGateFan];
#pragma unroll
        for (int b = 0; b < kGateFan; ++b)
          u[b] = b < n ? __hip_atomic_load(from + (int64_t)b * items + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
        float f = 0.f;
        uint32_t c = 0;
#pragma unroll
        for (int b = 0; b < kGateFan; ++b) {
          f += __uint_as_float(u[b]);
          c += u[b];
        }
        if (i < E) psum[0][i] = f;
        else cnt[i - E] = (int)c;
      }
      __syncthreads();
    };
    put(part + (int64_t)blockIdx.x * items);
    if (!last_arrival(root + 1 + g, (unsigned)members, &flag)) return;
    take(part + (int64_t)g * kGateFan * items, members);
    if (groups > 1) {
      put(gpart + (int64_t)g * items);
      if (!last_arrival(root, (unsigned)groups, &flag)) return;
      take(gpart, groups);
    }
  }
  const int e = threadIdx.x;
  const float P = e < E ? psum[0][e] : 0.f;
  const int c = e < E ? cnt[e] : 0;
  if (e < E) {
    p.prob_sum[e] = P;
    p.counts[e] = c;
  }
  float x = (float)c * P, y = (float)c;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    x += __shfl_xor(x, o);
    y += __shfl_xor(y, o);
  }
  if ((threadIdx.x & 63) == 0) {
    red[0][wave] = x;
    red[1][wave] = y;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int n = cnt[E];
    p.counts[E] = n;
    float a = 0.f, C = 0.f;
    for (int i = 0; i < kGateWaves; ++i) {
      a += red[0][i];
      C += red[1][i];
    }
    *p.loss = n > 0 ? p.coef * (float)E * (a / (C * (float)n)) : a;  // nothing routed: 0 (or NaN)
  }
}

// The choices' own terms reach the lanes that hold their experts through a
// per-token row of LDS that is zero between tokens.
template <int LPT, int VPL, bool BF16>
__global__ void __launch_bounds__(kBwdThreads) gate_bwd_kernel(GateBwdParams p) {
  typedef Row<LPT, VPL, BF16> R;
  constexpr int GPB = kBwdThreads / LPT;
  constexpr int EMAX = LPT * VPL;
  __shared__ __attribute__((aligned(16))) float own[GPB][EMAX];
  __shared__ float part[kBwdThreads / 64];
  const int E = p.E;
  const int sub = threadIdx.x % LPT;
  const int grp = threadIdx.x / LPT;
  const bool whole = E % R::VEC == 0;
  // C = sum of the counts
  float C = 0.f;
  for (int e = threadIdx.x; e < E; e += kBwdThreads) C += (float)p.counts[e];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) C += __shfl_xor(C, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = C;
  for (int i = threadIdx.x; i < GPB * EMAX; i += kBwdThreads) (&own[0][0])[i] = 0.f;
  __syncthreads();
  C = (part[0] + part[1]) + (part[2] + part[3]);
  const float n = (float)p.counts[E];
  const float f = p.dloss && n > 0.f ? *p.dloss * p.coef * (float)E / (C * n) : 0.f;
  float g[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = R::expert(sub, v);
    g[v] = e < E ? f * (float)p.counts[e] : 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < p.T; t0 += (int64_t)gridDim.x * GPB) {
    const int64_t t = t0 + grp;
    const bool in = t < p.T;
    const int idx = in && sub < p.k ? p.idx[t * p.k + sub] : -1;
    const bool live = in && p.idx[t * p.k] >= 0;  // the first choice exists
    const bool have = idx >= 0 && idx < E;
    const float w = have ? p.w[t * p.k + sub] : 0.f;
    const float dw = have && p.dw ? p.dw[t * p.k + sub] : 0.f;
    float l[VPL];
    R::load(p.logits, t, E, sub, live, whole, l);
    float m = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < VPL; ++v) m = fmaxf(m, l[v]);
    m = group_fmax<LPT>(m);
    if (!live) m = 0.f;
    float s = 0.f, pg = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      l[v] = exp_neg(l[v] - m);
      s += l[v];
      pg = __builtin_fmaf(l[v], g[v], pg);
    }
    s = group_sum<LPT>(s);
    pg = group_sum<LPT>(pg);
    const float dot = group_sum<LPT>(w * dw);
    const float inv = live ? 1.0f / s : 0.f;
    const float base = pg * inv + (p.renorm ? 0.f : dot);
    if (have) own[grp][idx] = p.renorm ? w * (dw - dot / p.w_scale) : w * dw;
    __builtin_amdgcn_wave_barrier();  // a row belongs to lanes of one wave: LDS accesses are in order
    float d[VPL];
#pragma unroll
    for (int c = 0; c < VPL / 4; ++c) {
      const float4 a = *reinterpret_cast<const float4*>(&own[grp][R::expert(sub, 4 * c)]);
      d[4 * c] = a.x; d[4 * c + 1] = a.y; d[4 * c + 2] = a.z; d[4 * c + 3] = a.w;
    }
    __builtin_amdgcn_wave_barrier();
    if (have) own[grp][idx] = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] += l[v] * inv * (g[v] - base);
    if (in) R::store(p.dlogits, t, E, sub, whole, d);
  }
}

// lanes per token and values per lane of E experts (bf16 pieces hold 8 values)
#define DG_GATE_SHAPES(X)                                  \
  if (bf16) {                                              \
    if (p.E <= 128) { X(16, 8, true); }                    \
    else if (p.E <= 256) { X(16, 16, true); }              \
    else if (p.E <= 512) { X(64, 8, true); }               \
    else { X(64, 16, true); }                              \
  } else {                                                 \
    if (p.E <= 64) { X(16, 4, false); }                    \
    else if (p.E <= 128) { X(16, 8, false); }              \
    else if (p.E <= 256) { X(16, 16, false); }             \
    else if (p.E <= 512) { X(64, 8, false); }              \
    else { X(64, 16, false); }                             \
  }

int gate_blocks(int64_t T, int64_t E) {
  const int64_t per = kGateThreads / (E <= 256 ? 16 : 64);
  const int64_t b = (T + per - 1) / per;
  return (int)(b < 1 ? 1 : (b < kGateMaxBlocks ? b : kGateMaxBlocks));
}

}  // namespace

size_t gate_workspace_bytes(int64_t T, int64_t E) {
  const int blocks = gate_blocks(T, E);
  return kWsCounterBytes + (size_t)(blocks + kGateFan) * (size_t)(2 * E + 1) * 4;
}

hipError_t launch_gate(const GateParams& p, bool bf16, hipStream_t stream) {
  const int blocks = gate_blocks(p.T, p.E);
#define X(L, V, B)                                                                                                       \
  if (p.k <= 8) hipLaunchKernelGGL((gate_kernel<L, V, 8, B>), dim3(blocks), dim3(kGateThreads), 0, stream, p);           \
  else hipLaunchKernelGGL((gate_kernel<L, V, 16, B>), dim3(blocks), dim3(kGateThreads), 0, stream, p)
  DG_GATE_SHAPES(X)
#undef X
  return hipGetLastError();
}

hipError_t launch_gate_bwd(const GateBwdParams& p, bool bf16, hipStream_t stream) {
  const int64_t per = kBwdThreads / (p.E <= 256 ? 16 : 64);
  const int64_t b = (p.T + per - 1) / per;
  // three workgroups a CU: the counts and the zeroed row are set up once for several rounds of tokens (32768 x 256 fp32:
  // 512, 768, 1024, 2048 workgroups 18, 17, 18, 22 us; bf16 17, 16, 18, 26 us)
  const int blocks = (int)(b < 768 ? b : 768);
#define X(L, V, B) hipLaunchKernelGGL((gate_bwd_kernel<L, V, B>), dim3(blocks), dim3(kBwdThreads), 0, stream, p)
  DG_GATE_SHAPES(X)
#undef X
  return hipGetLastError();
}

}  // namespace dg
