// The experts of a mixture-of-experts layer for a few tokens, in two kernels:
//   h[c] = silu(W1g_e x_t) * (W1u_e x_t)          for each choice c = (t, j) of an expert e held here
//   y[t] = sum_j w[t, j] W2_e h[(t, j)]
// x and y are bf16, weights block-scaled e4m3 or microscaled 4-bit floats.  The
// weights are widened to bf16 (exactly: e4m3 has 4 significant bits, e2m1 two and
// a power of two) and multiplied with bf16 activations in the matrix cores, fp32
// sums; the block scales are applied to each 128-deep product.  h is rounded to
// bf16 once, as the matrix cores take it; y once at the end.
//
// Bound by the weights of the experts that were chosen, which are read once,
// straight into registers: no two waves share a weight, so staging them in LDS
// would only add a hop.  16 weight rows are the matrix cores' row operand and up
// to 16 tokens the column operand, so one token costs what sixteen do.

#include "activation.hpp"
#include "block_internal.hpp"
#include "gemm_common.hpp"

namespace dg {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOOB = 0xFFFFFF00u;  // an offset past every buffer range used here
constexpr int kStream = 2;              // nt
constexpr int kCoherent = 16;           // sc1: coherent across the XCDs' L2 caches

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

enum Format { kFp8 = 0, kFp4 = 1 };

// A lane's 32 consecutive weights of one row (a quarter of a 128-deep step)
template <int FMT>
struct Weights {
  u32x4 v[FMT == kFp8 ? 2 : 1];
};

template <int FMT, bool NT>
__device__ __forceinline__ Weights<FMT> load_weights(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t step) {
  Weights<FMT> w;
  if constexpr (FMT == kFp8) {
    w.v[0] = __builtin_amdgcn_raw_buffer_load_b128(r, off, step * 128u, NT ? kStream : 0);
    w.v[1] = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16u, step * 128u, NT ? kStream : 0);
  } else {
    w.v[0] = __builtin_amdgcn_raw_buffer_load_b128(r, off, step * 64u, NT ? kStream : 0);
  }
  return w;
}

// The i-th 8 of them as bf16.  e4m3 as it is; e2m1 times the power of two in byte 0 of `code`.
template <int FMT>
__device__ __forceinline__ bf16x8 widened(const Weights<FMT>& w, int i, float scale) {
  typedef __bf16 bf16x2_ __attribute__((ext_vector_type(2)));
  union {
    bf16x8 v;
    bf16x2_ p[4];
  } r;
  if constexpr (FMT == kFp8) {
    const int a = (int)w.v[i >> 1][2 * (i & 1)], b = (int)w.v[i >> 1][2 * (i & 1) + 1];
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
  } else {
    const uint32_t a = w.v[0][i];
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 0);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 1);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 2);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 3);
  }
  return r.v;
}

// fp32 whose exponent is byte q of a scale word (the conversion reads the exponent alone: 255 gives NaN, 0 2^-127)
__device__ __forceinline__ float exponent_of(uint32_t word, int q) { return __uint_as_float(((word >> (8 * q)) & 0xffu) << 23); }

__device__ __forceinline__ f32x4 mfma(bf16x8 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---- gate and up projection.  A workgroup takes 16 columns of h of one chosen expert (16 rows of the gate and of the up
// weights), its four waves a quarter of H each.  The expert's choices share a pass over the weights, up to 32 of them (most
// experts have few: 16 keep four steps in flight, 32 two).

// the chosen experts of [first, first + G) as bits, and each choice's (-1: not here), in LDS
struct Chosen {
  uint32_t bits[kExpertsMaxGroups / 32];
  int before[kExpertsMaxGroups / 32 + 1];  // experts before each word's
  int16_t expert[kExpertsMaxChoices];
};

__device__ __forceinline__ void read_choices(const ExpertsParams& p, Chosen& s) {
  const int n = p.T * p.k;
  if (threadIdx.x < 32) s.bits[threadIdx.x] = 0;
  __syncthreads();
  for (int c = threadIdx.x; c < n; c += 256) {
    const int64_t e = (int64_t)p.idx[c] - p.first;
    const bool here = e >= 0 && e < p.G;
    s.expert[c] = here ? (int16_t)e : -1;
    if (here) atomicOr(&s.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (threadIdx.x < 64) {  // one wave
    const int lane = threadIdx.x;
    int v = lane < 32 ? __popc(s.bits[lane]) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up(v, o);
      if (lane >= o) v += u;
    }
    if (lane == 0) s.before[0] = 0;
    if (lane < 32) s.before[lane + 1] = v;
  }
  __syncthreads();
}

// the a-th chosen expert (a < s.before[32])
__device__ __forceinline__ int nth_expert(const Chosen& s, int a) {
  int lo = 0, hi = 31;  // the last word with before[] <= a
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.before[mid] <= a) lo = mid;
    else hi = mid - 1;
  }
  uint32_t b = s.bits[lo];
  for (int i = a - s.before[lo]; i > 0; --i) b &= b - 1;
  return __builtin_amdgcn_readfirstlane(lo * 32 + __ffs(b) - 1);
}

// what the passes of a wave share
struct UpWave {
  const uint8_t* wbase;
  const void* sbase;
  uint32_t w_bytes, s_bytes;
  uint32_t g_off, u_off;    // of the lane's gate and up row
  float beta_g, beta_u;     // e4m3: block scales of the wave's steps, one to a lane
  int lo, hi;               // steps
  int i0, lane, wave, q, n16;
};

// rows [m0, m0 + 16 MG) of the expert's choices
template <int FMT, int MG, bool NT>
__device__ __forceinline__ void up_pass(const ExpertsParams& p, const UpWave& s, const int16_t* rows, int m, int m0,
                                        f32x4 (*part)[4][64]) {
  constexpr int D = MG == 1 ? 4 : 2;  // steps in flight
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, (uint32_t)p.T * (uint32_t)p.H * 2u);
  const uint32_t two_i = 2u * (uint32_t)p.I;
  uint32_t x_off[MG];
#pragma unroll
  for (int g = 0; g < MG; ++g) {
    const int r = m0 + 16 * g + s.n16;
    x_off[g] = r < m ? (uint32_t)(rows[r] / p.k) * (uint32_t)p.H * 2u + 64u * s.q : kOOB;
  }
  Weights<FMT> wg[D], wu[D];
  uint32_t sg[D], su[D];
  u32x4 xr[D][MG][4];
  f32x4 cg[MG], cu[MG];
#pragma unroll
  for (int g = 0; g < MG; ++g) cg[g] = cu[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  // past the wave's last step the ranges are empty: zeros, and no traffic
  auto load = [&](int d, int kb) {
    const bool in = kb < s.hi;
    const uint32_t k = in ? (uint32_t)kb : 0u;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(s.wbase, in ? s.w_bytes : 0u);
    const __amdgpu_buffer_rsrc_t ry = in ? rx : make_rsrc(p.x, 0u);
    wg[d] = load_weights<FMT, NT>(rw, s.g_off, k);
    wu[d] = load_weights<FMT, NT>(rw, s.u_off, k);
    if constexpr (FMT == kFp4) {  // a word of four codes a row and step
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(s.sbase, in ? s.s_bytes : 0u);
      sg[d] = __builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(s.i0 + s.n16) * 4u, k * 4u * two_i, 0);
      su[d] = __builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(p.I + s.i0 + s.n16) * 4u, k * 4u * two_i, 0);
    }
#pragma unroll
    for (int g = 0; g < MG; ++g)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        xr[d][g][t] = __builtin_amdgcn_raw_buffer_load_b128(ry, x_off[g] == kOOB ? kOOB : x_off[g] + 16u * t, k * 256u, 0);
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, s.lo + d);
  for (int k0 = s.lo; k0 < s.hi; k0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      __builtin_amdgcn_sched_barrier(0);
      const float eg = FMT == kFp4 ? exponent_of(sg[d], s.q) : 1.f, eu = FMT == kFp4 ? exponent_of(su[d], s.q) : 1.f;
      bf16x8 ag[4], au[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        ag[t] = widened<FMT>(wg[d], t, eg);
        au[t] = widened<FMT>(wu[d], t, eu);
      }
      const int i = k0 + d - s.lo;  // a lane's: a quarter of a row is at most 64 steps, and lanes past it hold zeros
      const float bg = FMT == kFp8 ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s.beta_g), i)) : 1.f;
      const float bu = FMT == kFp8 ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s.beta_u), i)) : 1.f;
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        const f32x4 zero = f32x4{0.f, 0.f, 0.f, 0.f};
        f32x4 pg = FMT == kFp8 ? zero : cg[g], pu = FMT == kFp8 ? zero : cu[g];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          pg = mfma(ag[t], xr[d][g][t], pg);
          pu = mfma(au[t], xr[d][g][t], pu);
        }
        if constexpr (FMT == kFp8) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            cg[g][v] = __builtin_fmaf(pg[v], bg, cg[g][v]);
            cu[g][v] = __builtin_fmaf(pu[v], bu, cu[g][v]);
          }
        } else {
          cg[g] = pg;
          cu[g] = pu;
        }
      }
      load(d, k0 + d + D);
    }
  }
  // the waves' sums, in order
  __syncthreads();  // (the last pass' reads of part are done)
  if (s.wave > 0) {
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      part[s.wave - 1][2 * g][s.lane] = cg[g];
      part[s.wave - 1][2 * g + 1][s.lane] = cu[g];
    }
  }
  __syncthreads();
  if (s.wave > 0) return;
#pragma unroll
  for (int g = 0; g < MG; ++g) {
#pragma unroll
    for (int o = 0; o < 3; ++o) {
      cg[g] += part[o][2 * g][s.lane];
      cu[g] += part[o][2 * g + 1][s.lane];
    }
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = activate<kActSilu>(cg[g][j]) * cu[g][j];
    const int r = m0 + 16 * g + s.n16;
    if (r < m)
      *reinterpret_cast<uint2*>(p.h + (int64_t)rows[r] * p.I + s.i0 + 4 * s.q) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

template <int FMT, bool NT>
__global__ void __launch_bounds__(256) experts_up_kernel(ExpertsParams p) {
  __shared__ Chosen s;
  __shared__ int16_t rows[kExpertsMaxChoices];
  __shared__ int n_rows;
  __shared__ __attribute__((aligned(16))) f32x4 part[3][4][64];
  const int H = p.H, I = p.I;
  const int tiles = I >> 4;
  const int a = (int)blockIdx.x / tiles;
  UpWave u;
  u.i0 = ((int)blockIdx.x - a * tiles) * 16;
  u.lane = threadIdx.x & 63;
  u.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  u.q = u.lane >> 4;
  u.n16 = u.lane & 15;
  if (threadIdx.x == 0) n_rows = 0;
  read_choices(p, s);
  if (a >= s.before[kExpertsMaxGroups / 32]) return;  // fewer experts were chosen than could be
  const int e = nth_expert(s, a);
  for (int c = threadIdx.x; c < p.T * p.k; c += 256)  // (which column of the products a choice takes does not matter)
    if (s.expert[c] == e) rows[atomicAdd(&n_rows, 1)] = (int16_t)c;
  __syncthreads();
  const int m = __builtin_amdgcn_readfirstlane(n_rows);

  const int KB = H >> 7;
  const int per = (KB + 3) >> 2;
  u.lo = u.wave * per < KB ? u.wave * per : KB;
  u.hi = u.lo + per < KB ? u.lo + per : KB;
  const uint32_t row_bytes = FMT == kFp8 ? (uint32_t)H : (uint32_t)H / 2;
  u.w_bytes = 2u * (uint32_t)I * row_bytes;
  u.wbase = p.w1 + (int64_t)e * u.w_bytes;
  u.g_off = (uint32_t)(u.i0 + u.n16) * row_bytes + (FMT == kFp8 ? 32u * u.q : 16u * u.q);
  u.u_off = u.g_off + (uint32_t)I * row_bytes;
  u.beta_g = u.beta_u = 0.f;
  u.s_bytes = FMT == kFp8 ? 0u : (uint32_t)KB * 2u * (uint32_t)I * 4u;
  u.sbase = FMT == kFp8 ? p.s1 : static_cast<const int32_t*>(p.s1) + (int64_t)e * KB * 2 * I;
  if constexpr (FMT == kFp8) {
    const float* b = static_cast<const float*>(p.s1) + (int64_t)e * (I >> 6) * KB;  // [2 I / 128][KB]
    if (u.lo + u.lane < u.hi) {
      u.beta_g = b[(int64_t)(u.i0 >> 7) * KB + u.lo + u.lane];
      u.beta_u = b[(int64_t)((I + u.i0) >> 7) * KB + u.lo + u.lane];
    }
  }
  int m0 = 0;
  for (; m - m0 > 16; m0 += 32) up_pass<FMT, 2, NT>(p, u, rows, m, m0, part);
  if (m0 < m) up_pass<FMT, 1, NT>(p, u, rows, m, m0, part);
}

// ---- down projection and weighted sum.  A workgroup takes 16 columns of y for all tokens; its eight waves, and those of all
// p.splits workgroups of the columns, take equal runs of the 128-deep steps of all chosen experts, one expert after the other,
// with the next steps' loads in flight across experts.  The tokens of an expert share its steps, 16 at a time; a product goes
// into the accumulator times its block scale and the token's weight, and from there, when the expert (or its 16 tokens) change,
// into the wave's sums of the tokens in LDS, so that a token's experts are added in the order of their numbers.
struct Members {
  int16_t expert[kExpertsMaxChoices];   // of each choice, -1: not here
  int count[kExpertsMaxGroups];         // tokens of each expert
  int16_t rank[kExpertsMaxGroups];      // of a chosen expert among the chosen
  int16_t list[kExpertsMaxGroups];      // chosen experts
  int16_t start[kExpertsMaxGroups + 1]; // first of its entries below
  int16_t group[kExpertsMaxGroups + 1]; // groups of 16 tokens before it
  int16_t choice[kExpertsMaxChoices];   // entries: a choice whose row of h is the token's, and its weight
  float weight[kExpertsMaxChoices];
  int n;                                // chosen experts
};

__device__ __forceinline__ void read_members(const ExpertsParams& p, Members& s) {
  const int n = p.T * p.k;
  for (int e = threadIdx.x; e < p.G; e += 512) s.count[e] = 0;
  for (int c = threadIdx.x; c < n; c += 512) {
    const int64_t e = (int64_t)p.idx[c] - p.first;
    s.expert[c] = e >= 0 && e < p.G ? (int16_t)e : -1;
  }
  __syncthreads();
  // a token that names an expert twice is one entry, of the first of the choices, with the sum of their weights
  int mine[kExpertsMaxChoices / 512], place[kExpertsMaxChoices / 512];
  float w[kExpertsMaxChoices / 512];
#pragma unroll
  for (int i = 0; i < kExpertsMaxChoices / 512; ++i) {
    const int c = threadIdx.x + 512 * i;
    mine[i] = -1;
    place[i] = 0;
    w[i] = 0.f;
    if (c >= n) continue;
    const int e = s.expert[c];
    if (e < 0) continue;
    const int t0 = c - c % p.k;
    bool first = true;
    for (int j = t0; j < t0 + p.k; ++j)
      if (s.expert[j] == e) {
        if (j < c) first = false;
        else w[i] += p.w[j];
      }
    if (!first) continue;
    mine[i] = e;
    place[i] = atomicAdd(&s.count[e], 1);  // (which column a token takes does not matter)
  }
  __syncthreads();
  if (threadIdx.x < 64) {  // one wave: ranks, and sums over the chosen experts of their tokens and groups
    const int lane = threadIdx.x;
    int chosen = 0, tokens = 0, groups = 0;
    for (int e0 = 0; e0 < p.G; e0 += 64) {
      const int e = e0 + lane;
      const int m = e < p.G ? s.count[e] : 0;
      int v = m | (((m + 15) >> 4) << 16);  // both sums at once: at most 1024 tokens and 1024 groups
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
      }
      const unsigned long long mask = __ballot(m > 0);
      if (m > 0) {
        const int a = chosen + __popcll(mask & ((1ull << lane) - 1));
        s.rank[e] = (int16_t)a;
        s.list[a] = (int16_t)e;
        s.start[a] = (int16_t)(tokens + (v & 0xffff) - m);
        s.group[a] = (int16_t)(groups + (v >> 16) - ((m + 15) >> 4));
      }
      chosen += __popcll(mask);
      const int all = __shfl(v, 63);
      tokens += all & 0xffff;
      groups += all >> 16;
    }
    if (lane == 0) {
      s.n = chosen;
      s.start[chosen] = (int16_t)tokens;
      s.group[chosen] = (int16_t)groups;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kExpertsMaxChoices / 512; ++i)
    if (mine[i] >= 0) {
      const int at = s.start[s.rank[mine[i]]] + place[i];
      s.choice[at] = (int16_t)(threadIdx.x + 512 * i);
      s.weight[at] = w[i];
    }
  __syncthreads();
}

template <int FMT, bool NT>
__global__ void __launch_bounds__(512) experts_down_kernel(ExpertsParams p) {
  constexpr int D = 3;  // steps in flight
  constexpr int W = 8;
  __shared__ Members s;
  __shared__ __attribute__((aligned(16))) f32x4 sums[W][kExpertsMaxTokens * 4];  // [token][quarter of the columns]
  __shared__ int last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, n16 = lane & 15;
  const int H = p.H, I = p.I;
  const int tile = (int)blockIdx.x / p.splits, split = (int)blockIdx.x - tile * p.splits;
  const int c0 = tile * 16;
  for (int i = lane; i < p.T * 4; i += 64) sums[wave][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  read_members(p, s);
  const int KB = I >> 7;
  const int chosen = __builtin_amdgcn_readfirstlane(s.n);
  const int steps = chosen * KB;  // (a step of all of an expert's groups: which of them a token is in changes no sum)
  const int slots = W * p.splits;
  const int per = (steps + slots - 1) / slots;
  const int lo = (split * W + wave) * per < steps ? (split * W + wave) * per : steps;
  const int hi = lo + per < steps ? lo + per : steps;

  const uint32_t row_bytes = FMT == kFp8 ? (uint32_t)I : (uint32_t)I / 2;
  const uint32_t w_bytes = (uint32_t)H * row_bytes;
  const uint32_t w_off = (uint32_t)(c0 + n16) * row_bytes + (FMT == kFp8 ? 32u * q : 16u * q);
  // scales: e4m3 [ceil(H / 128)][KB] fp32, e2m1 words [KB][H]
  const uint32_t s_bytes = FMT == kFp8 ? (uint32_t)((H + 127) >> 7) * (uint32_t)KB * 4u : (uint32_t)KB * (uint32_t)H * 4u;
  const uint32_t s_off = FMT == kFp8 ? (uint32_t)(c0 >> 7) * (uint32_t)KB * 4u : (uint32_t)(c0 + n16) * 4u;
  const uint32_t s_step = FMT == kFp8 ? 4u : 4u * (uint32_t)H;
  const uint32_t h_bytes = (uint32_t)p.T * (uint32_t)p.k * (uint32_t)I * 2u;

  if (lo < hi) {
    // what is being loaded: expert ld_a of the list, step ld_k, group ld_g of its ld_n; the lane's row of h, weight and token
    int ld_a = lo / KB, ld_k = lo - ld_a * KB;
    int ld_g = 0, ld_n = 1, first = 0, members = 0;
    // loads of the run: a step's groups one after the other
    auto loads_before = [&](int step) {
      const int a = step / KB;
      const int g = __builtin_amdgcn_readfirstlane((int)s.group[a]);
      const int n = a < chosen ? __builtin_amdgcn_readfirstlane((int)s.group[a + 1]) - g : 0;
      return g * KB + (step - a * KB) * n;
    };
    const int loads = loads_before(hi) - loads_before(lo);
    const uint8_t* wbase = p.w2;
    const uint8_t* sbase = static_cast<const uint8_t*>(p.s2);
    uint32_t h_off = kOOB;
    float fac = 0.f;
    int token = -1;
    auto enter_expert = [&]() {
      const int e = __builtin_amdgcn_readfirstlane((int)s.list[ld_a]);
      wbase = p.w2 + (int64_t)e * w_bytes;
      sbase = static_cast<const uint8_t*>(p.s2) + (int64_t)e * s_bytes;
      first = __builtin_amdgcn_readfirstlane((int)s.start[ld_a]);
      members = __builtin_amdgcn_readfirstlane((int)s.start[ld_a + 1]) - first;
      ld_n = (members + 15) >> 4;
    };
    auto enter_group = [&]() {
      const int r = 16 * ld_g + n16;
      h_off = kOOB;
      fac = 0.f;
      token = -1;
      if (r < members) {
        const int c = s.choice[first + r];
        h_off = (uint32_t)c * (uint32_t)I * 2u + 64u * q;
        fac = s.weight[first + r];
        token = c / p.k;
      }
    };
    enter_expert();
    enter_group();
    bool fresh = true;  // the next load begins a group of tokens

    Weights<FMT> wr[D];
    uint32_t sr[D];
    u32x4 hr[D][4];
    float fr[D];
    int tr[D];
    bool nr[D];
    auto load = [&](int d, int j) {
      const bool in = j < loads;
      if (in && ld_k == KB) {
        ++ld_a;
        ld_k = ld_g = 0;
        enter_expert();
        enter_group();
        fresh = true;
      }
      const __amdgpu_buffer_rsrc_t rw = make_rsrc(wbase, in ? w_bytes : 0u);
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(sbase, in ? s_bytes : 0u);
      const __amdgpu_buffer_rsrc_t rh = make_rsrc(p.h, in ? h_bytes : 0u);
      const uint32_t k = in ? (uint32_t)ld_k : 0u;
      wr[d] = load_weights<FMT, NT>(rw, w_off, k);
      sr[d] = __builtin_amdgcn_raw_buffer_load_b32(rs, s_off, k * s_step, 0);
#pragma unroll
      for (int t = 0; t < 4; ++t) hr[d][t] = __builtin_amdgcn_raw_buffer_load_b128(rh, h_off == kOOB ? kOOB : h_off + 16u * t, k * 256u, 0);
      fr[d] = in ? fac : 0.f;  // (an infinite weight times the padding's zero would be NaN)
      tr[d] = token;
      nr[d] = in && fresh;
      fresh = false;
      if (in) {
        if (ld_n == 1) {
          ++ld_k;
        } else {
          if (++ld_g == ld_n) {
            ld_g = 0;
            ++ld_k;
          }
          enter_group();
          fresh = true;
        }
      }
    };
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    int to = -1;
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int j0 = 0; j0 < loads; j0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        __builtin_amdgcn_sched_barrier(0);
        if (nr[d]) {  // uniform
          if (to >= 0) sums[wave][to * 4 + q] += acc;
          acc = f32x4{0.f, 0.f, 0.f, 0.f};
          to = tr[d];
        }
        const float ex = FMT == kFp4 ? exponent_of(sr[d], q) : 1.f;
        f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 4; ++t) o = mfma(widened<FMT>(wr[d], t, ex), hr[d][t], o);
        const float f = FMT == kFp8 ? fr[d] * __uint_as_float(sr[d]) : fr[d];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(o[v], f, acc[v]);
        load(d, j0 + d + D);
      }
    }
    if (to >= 0) sums[wave][to * 4 + q] += acc;
  }
  __syncthreads();
  // the waves' sums in order: a thread takes four columns of a token
  const int u = threadIdx.x;
  const bool live = u < p.T * 4;
  f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
  if (live)
#pragma unroll
    for (int o = 0; o < W; ++o) y += sums[o][u];
  if (p.splits > 1) {
    // The workgroups' sums meet in the workspace: sc1 stores and loads are coherent across the XCDs' L2 caches; every wave's
    // stores are acknowledged (vmcnt 0) before the barrier that precedes the relaxed counter increment, and the last
    // workgroup loads only after its own increment has returned.  It adds them in order and leaves the counter at zero.
    const uint32_t one = (uint32_t)p.T * 64u;
    const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.partials, (uint32_t)(p.splits * (H >> 4)) * one);
    const uint32_t off = live ? (uint32_t)tile * (uint32_t)p.splits * one + (uint32_t)u * 16u : kOOB;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), rp, off, (uint32_t)split * one, kCoherent);
    wait_vmcnt<0>();
    __syncthreads();
    if (threadIdx.x == 0)
      last = __hip_atomic_fetch_add(&p.counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned int)(p.splits - 1);
    __syncthreads();
    if (!last) return;
    y = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < p.splits; ++i)
      y += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rp, off, (uint32_t)i * one, kCoherent));
    if (threadIdx.x == 0) __hip_atomic_store(&p.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (live)
    *reinterpret_cast<uint2*>(p.y + (int64_t)(u >> 2) * H + c0 + 4 * (u & 3)) = uint2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

template <int FMT, bool NT>
hipError_t launch_format(const ExpertsParams& p, hipStream_t stream) {
  const int most = p.G < p.T * p.k ? p.G : p.T * p.k;  // experts that can have been chosen
  hipLaunchKernelGGL((experts_up_kernel<FMT, NT>), dim3((unsigned)(most * (p.I / 16))), dim3(256), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((experts_down_kernel<FMT, NT>), dim3((unsigned)(p.H / 16 * p.splits)), dim3(512), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

// Workgroups that share 16 columns of the down projection: as many as give the chip sixteen waves a CU, with two steps a wave
int experts_splits(int64_t choices, int64_t H, int64_t I, int64_t G, int cus) {
  const int64_t tiles = H / 16;
  if (tiles > 1024) return 1;  // counters
  const int64_t steps = (G < choices ? G : choices) * (I / 128);
  int64_t s = 2 * (int64_t)cus / tiles;
  if (s > steps / 16) s = steps / 16;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

size_t experts_h_bytes(int64_t choices, int64_t I) { return ((size_t)choices * (size_t)I * 2 + 255) / 256 * 256; }

hipError_t launch_moe_experts(const ExpertsParams& p, bool fp4, bool stream_weights, hipStream_t stream) {
  if (fp4) return stream_weights ? launch_format<kFp4, true>(p, stream) : launch_format<kFp4, false>(p, stream);
  return stream_weights ? launch_format<kFp8, true>(p, stream) : launch_format<kFp8, false>(p, stream);
}

}  // namespace dg
