// The experts of a mixture-of-experts layer for a few tokens, in two kernels:
//   h[c] = silu(W1g_e x_t) * (W1u_e x_t)          for each choice c = (t, j) of an expert e held here
//   y[t] = sum_j w[t, j] W2_e h[(t, j)]
// x and y are bf16, weights block-scaled e4m3 or microscaled 4-bit floats.  The
// weights are widened to bf16 (exactly: e4m3 has 4 significant bits, e2m1 two and
// a power of two) and multiplied with bf16 activations in the matrix cores, fp32
// sums; the block scales are applied to each 128-deep product.  h is rounded to
// bf16 once, as the matrix cores take it; y once at the end.
//
// Bound by the weights of the experts that were chosen, which are read straight
// into registers: no two waves share a weight, so staging them in LDS would only
// add a hop.  They are read once for as many tokens of an expert as share a pass:
// gate and up 16 (calls of up to 16 tokens) or 32; down 8, 16 or 32, one size
// for the whole call by the tokens an expert has on average.  So an expert of
// many tokens among cold ones is read more than once (64 tokens x 2 of 32, 4096
// x 2048 e4m3: 133 us even, 143 with one expert of 32 tokens, 154 with one of 64;
// e2m1 96, 103, 115).  An instruction loads whole cache lines, 8 rows of 128
// bytes, streamed past the caches (8 rows x 128 bytes 6.3 TB/s of 224 MB,
// 16 rows x 64 bytes, where a line is taken in two halves, 5.1).  So a lane has
// 16 bytes (a chunk) of one of 8 rows, row lane % 8, chunk lane / 16 + 4 (lane /
// 8 % 2), and the matrix cores' 16 x 16 product takes the 8 rows twice, in its
// upper and lower half with different chunks; 8 tokens are its columns, twice
// too.  The products of unlike halves are of no use, those of like halves are
// two sums over K that meet at the end: one token costs what eight do.  Where an
// expert has more, two such loads are turned into whole products of 16 rows and
// 16 tokens, one half of the chunks after the other.
//
// Rates (both kernels, weights alone): one token, 8 of 32 experts, 7168 x 2048
// e4m3 (352 MB) 62 us, 6.1 and 5.0 TB/s; 48 tokens x 8 of 256, 32 of them here,
// e2m1 (430 MB of the 17 to 19 that were chosen) 77-103 us, where a step's four
// loads of activations and two of scales keep the data path behind the address
// units busy 0.9 of the cycles; 64 tokens x 2 of 8, 4096 x 2048 e4m3 (202 MB)
// 53-67 us, busy 0.8: the activations, read from the L2 caches by every workgroup
// that needs them, take as long as the weights, e2m1 (107 MB) 42-45; 1, 8 and 16
// tokens x 8 of 64, 7168 x 2048 e2m1 (187, 983 and 1217 MB) 50, 199 and 247 us,
// 3.8-4.9 TB/s, e4m3 of 8 and 16 tokens 6.7 and 6.3; one token, 4 of 16 experts, 1024
// x 512 (6 MB) 11.4 us, two launches and the order of the choices.

#include "activation.hpp"
#include "block_internal.hpp"
#include "gemm_common.hpp"

namespace dg {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOOB = 0xFFFFFF00u;  // an offset past every buffer range used here
constexpr int kStream = 2;              // nt
constexpr int kCoherent = 16;           // sc1: coherent across the XCDs' L2 caches

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

enum Format { kFp8 = 0, kFp4 = 1 };

// The t-th 8 weights of a lane's chunk as bf16: of 16 e4m3 as they are (t < 2), of 32 e2m1 times the power of two `scale` (t < 4)
template <int FMT>
__device__ __forceinline__ bf16x8 widened(u32x4 w, int t, float scale) {
  typedef __bf16 bf16x2_ __attribute__((ext_vector_type(2)));
  union {
    bf16x8 v;
    bf16x2_ p[4];
  } r;
  if constexpr (FMT == kFp8) {
    const int a = (int)w[2 * t], b = (int)w[2 * t + 1];
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
  } else {
    const uint32_t a = w[t];
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 0);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 1);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 2);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 3);
  }
  return r.v;
}
template <int FMT>
constexpr int kParts = FMT == kFp8 ? 2 : 4;  // 8-deep parts of a chunk: products of a step, and 16-byte loads of its activations
template <int FMT>
constexpr uint32_t kStepDepth = FMT == kFp8 ? 128 : 256;  // weights of a row in a step's 128 bytes

// fp32 whose exponent is byte q of a scale word (the conversion reads the exponent alone: 255 gives NaN, 0 2^-127)
__device__ __forceinline__ float exponent_of(uint32_t word, int q) { return __uint_as_float(((word >> (8 * q)) & 0xffu) << 23); }

// 16 bytes of each lane to where the products want them: loaded so that four neighbouring lanes have 64 consecutive bytes (row
// lane / 8, chunk lane % 8, which the address unit takes as one access and not as four), used by the lane of row lane % 8 and
// chunk lane / 16 + 4 (lane / 8 % 2).  They go through 1 KB of the wave's own LDS, a row's chunks turned about by its number, so
// that neither side meets another lane's banks: a wave's LDS accesses happen in order, and no wait stands between the two (16
// cycles of the LDS; four rotations of a register between lanes took 23).  Slots in turn leave the next ones free to be written.
constexpr int kSpreadSlots = 2;
// what other lanes of the wave put into the LDS before this is seen after it: an order for the compiler, no instruction
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local"); }
struct Spread {
  u32x4* put;
  const u32x4* get;
  const u32x4* get16;  // of two slots together: row lane % 16, chunk lane / 16, and from those of the upper half the chunks past 4
  int upper;
};
__device__ __forceinline__ Spread spread_of(u32x4* slots) {
  const int lane = threadIdx.x & 63;
  const int r8 = lane & 7, chunk = (lane >> 4) + 4 * ((lane >> 3) & 1);
  const int row = 64 * ((lane >> 3) & 1) + 8 * r8, low = (lane >> 4) ^ r8;
  return Spread{slots + (lane & ~7) + ((lane & 7) ^ (lane >> 3)), slots + 8 * r8 + (chunk ^ r8), slots + row + low,
                (low ^ 4) - low};
}
__device__ __forceinline__ u32x4 spread(const Spread& s, int turn, u32x4 v) {
  s.put[64 * (turn % kSpreadSlots)] = v;
  wave_fence();  // (and the slot's last reads are before the fence of the turn between)
  return s.get[64 * (turn % kSpreadSlots)];
}

// the sum of both like halves of a product, in both
__device__ __forceinline__ f32x4 halves(f32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], 40);
  return v;
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// two registers of 8 rows each as both halves of the chunks of 16 rows
__device__ __forceinline__ void spread16(const Spread& s, u32x4 rows0, u32x4 rows8, u32x4 (&out)[2]) {
  wave_fence();  // the last reads of both slots
  s.put[0] = rows0;
  s.put[64] = rows8;
  wave_fence();
  out[0] = s.get16[0];
  out[1] = s.get16[s.upper];
}

// ---- who chose what.  Every workgroup of the first kernel sorts the choices by expert; its first leaves the result for the second.
struct Members {
  int16_t expert[kExpertsMaxChoices];  // of each choice, -1: not here
  float weight[kExpertsMaxChoices];
  int count[kExpertsMaxGroups];        // tokens of each expert
  int start[kExpertsMaxGroups];        // its first entry
  ExpertsTable table;
};
// a chosen expert's number, tokens and first entry in one word
__device__ __forceinline__ uint32_t run_word(int expert, int count, int start) {
  return (uint32_t)expert | (uint32_t)(count - 1) << 10 | (uint32_t)start << 16;
}
__device__ __forceinline__ int expert_of(uint32_t r) { return (int)(r & 1023u); }
__device__ __forceinline__ int count_of(uint32_t r) { return (int)((r >> 10) & 63u) + 1; }
__device__ __forceinline__ int start_of(uint32_t r) { return (int)(r >> 16); }
static_assert(kExpertsMaxGroups <= 1024 && kExpertsMaxTokens <= 64 && kExpertsMaxChoices <= 65536, "the words of the table");

// the tokens of all chosen experts
__device__ __forceinline__ int entries_of(const ExpertsTable& s) {
  const int n = __builtin_amdgcn_readfirstlane(s.n);
  const uint32_t end = n > 0 ? __builtin_amdgcn_readfirstlane(s.run[n - 1]) : 0u;
  return n > 0 ? start_of(end) + count_of(end) : 0;
}

constexpr int kUpThreads = 256;
// Tokens of an expert on average past which neighbouring units are taken together, in both kernels.  64 tokens, 4096 x 2048, every
// expert as many, apart and together: e4m3 of 32 experts with 4 tokens 132.6 and 137.4 us, 6: 135.8 and 138.7, 8: 141.2 and 140.1,
// 10: 183 and 142; e2m1 91 and 86, 103 and 92, 118 and 101, 148 and 102
constexpr int kPairTokens = 6;

__device__ __forceinline__ void read_members(const ExpertsParams& p, Members& s) {
  constexpr int EACH = kExpertsMaxChoices / kUpThreads;
  const int n = p.T * p.k;
  for (int e = threadIdx.x; e < p.G; e += kUpThreads) s.count[e] = 0;
  for (int c = threadIdx.x; c < n; c += kUpThreads) {
    const int64_t e = (int64_t)p.idx[c] - p.first;
    s.expert[c] = e >= 0 && e < p.G ? (int16_t)e : -1;
    s.weight[c] = p.w[c];
  }
  __syncthreads();
  // a token that names an expert twice is one entry, of the first of the choices, with the sum of their weights
  int mine[EACH], place[EACH];
  float w[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int c = threadIdx.x + kUpThreads * i;
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
        else w[i] += s.weight[j];
      }
    if (!first) continue;
    mine[i] = e;
    place[i] = atomicAdd(&s.count[e], 1);  // (which column of the products a token takes does not matter)
  }
  __syncthreads();
  if (threadIdx.x < 64) {  // one wave: the chosen experts in order
    const int lane = threadIdx.x;
    int chosen = 0, tokens = 0;
    for (int e0 = 0; e0 < p.G; e0 += 64) {
      const int e = e0 + lane;
      const int m = e < p.G ? s.count[e] : 0;
      int v = m;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
      }
      const unsigned long long mask = __ballot(m > 0);
      if (m > 0) {
        s.start[e] = tokens + v - m;
        s.table.run[chosen + __popcll(mask & ((1ull << lane) - 1))] = run_word(e, m, tokens + v - m);
      }
      chosen += __popcll(mask);
      tokens += __shfl(v, 63);
    }
    if (lane == 0) s.table.n = chosen;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < EACH; ++i)
    if (mine[i] >= 0) {
      const int c = threadIdx.x + kUpThreads * i, at = s.start[mine[i]] + place[i];
      s.table.entry[at] = (uint32_t)c | (uint32_t)(c / p.k) << 16;
      s.table.weight[at] = w[i];
    }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < n; i += kUpThreads) {  // (what lies past the experts and entries is not looked at)
      p.table->run[i] = s.table.run[i];
      p.table->entry[i] = s.table.entry[i];
      p.table->weight[i] = s.table.weight[i];
    }
    if (threadIdx.x == 0) p.table->n = s.table.n;
  }
}

// ---- gate and up projection.  A unit is 16 columns of h of one chosen expert (16 rows of the gate and of the up weights); a
// workgroup takes a run of units (or every so-manyth), its four waves a quarter of H each, and the next pass' first steps are in
// flight while the current one ends.  An expert's tokens share a pass over the weights, up to 8 MAXMG of them.  Where there are
// more than 8, two neighbouring units of a run are one pass: the tokens' activations, which the address unit takes as long for as
// for the weights, are loaded for both (8 experts, 64 tokens, 4096 x 2048: 34.8
// -> 33.4 us of this kernel).  Fewer are taken unit by unit, neighbouring workgroups on neighbouring units (48 tokens of 1.5 an
// expert 61.5 us, 68 in runs).

// steps in flight: (weights and activations of) a step take 16 + 8 registers for every 8 tokens of e4m3, 20 + 16 of e2m1, twice
// those of the weights for two units.  More are no faster: a wave has few steps of a row, padded to whole turns (16 to 32 tokens
// of 4096 x 2048, three in place of two: 36.0 -> 36.8 us)
template <int FMT>
constexpr int up_depth(int mg, int c, int maxmg) {
  if (c == 2) return FMT == kFp8 ? 2 : mg == 2 ? 2 : 1;
  if (FMT == kFp8) return maxmg == 2 ? 2 : mg == 1 ? 4 : mg == 2 ? 3 : 2;
  return maxmg == 2 ? (mg == 1 ? 3 : 1) : (mg == 1 ? 2 : 1);
}

template <int MAXMG>
struct __attribute__((aligned(16))) UpShared {
  Members members;
  f32x4 part[2][3][4 * MAXMG][16];  // [turn][wave - 1][accumulator][lane]
  u32x4 spread[kUpThreads / 64][64 * kSpreadSlots];
};

// A pass of 8 MG tokens, from m0 on, of unit u (all uniform)
struct UpItem {
  int u, m0;
  int expert, start, m, i0;
};
__device__ __forceinline__ UpItem up_item(const Members& s, int u, int m0, int tiles) {
  UpItem r;
  const int a = u / tiles;
  const uint32_t w = __builtin_amdgcn_readfirstlane(s.table.run[a]);
  r.u = u;
  r.m0 = m0;
  r.expert = expert_of(w);
  r.start = start_of(w);
  r.m = count_of(w);
  r.i0 = (u - a * tiles) * 16;
  return r;
}
// groups of 8 that share the pass: 1, 2 or 4.  One and more than one add in different orders, and which tokens a last pass has is
// not the same in every run: so an expert of more than 8 tokens takes none of one group.
template <int MAXMG>
__device__ __forceinline__ int up_groups(const UpItem& it) {
  return it.m - it.m0 > 8 * 2 && MAXMG > 2 ? 4 : it.m > 8 ? 2 : 1;
}
// units of the pass: two that share their block scales
struct UpRun {
  int end, step;  // the workgroup's units are every `step`th before `end`
};
template <int MAXMG>
__device__ __forceinline__ int up_units(const UpItem& it, const UpRun& run) {
  return MAXMG > 2 && run.step == 1 && it.m > 8 && it.u % 2 == 0 && it.u + 1 < run.end ? 2 : 1;
}

// the passes of this workgroup from `it` on, as long as they are of MG groups and C units; returns whether one is left, which is in `it`
template <int FMT, int MG, int C, int MAXMG, bool NT>
__device__ __forceinline__ bool up_passes(const ExpertsParams& p, UpShared<MAXMG>& sh, UpItem& it, const UpRun& run, int& turn) {
  constexpr int D = up_depth<FMT>(MG, C, MAXMG);
  constexpr int P = kParts<FMT>;
  const Members& s = sh.members;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r8 = lane & 7, half = (lane >> 3) & 1, q = lane >> 4;
  const uint32_t H = (uint32_t)p.H, I = (uint32_t)p.I;
  const int tiles = p.I >> 4;
  const uint32_t row_bytes = FMT == kFp8 ? H : H / 2;
  const uint32_t w_bytes = 2u * I * row_bytes;
  const int KB = p.H >> 7;
  const uint32_t s_bytes = FMT == kFp8 ? (I >> 6) * (uint32_t)KB * 4u : (uint32_t)KB * 2u * I * 4u;
  // this wave's steps [lo, lo + n) of a row, `per` a wave, padded to whole turns of the stages with empty ones
  const int steps = (int)((row_bytes + 127) >> 7);
  const int per = (steps + 3) >> 2;
  const int lo = wave * per;
  const int n = lo >= steps ? 0 : steps - lo < per ? steps - lo : per;
  const int padded = (per + D - 1) / D * D;
  // loads: row (or token) lane / 8, chunk lane % 8; weight rows 2 (lane / 8) + a: neighbours, whose scale words are loaded together
  const int l8 = lane >> 3, ch = lane & 7;
  const Spread sp = spread_of(sh.spread[wave]);
  uint32_t w_off[2 * C];
#pragma unroll
  for (int a = 0; a < 2 * C; ++a) w_off[a] = (uint32_t)(MG == 1 ? 2 * l8 + a : 8 * a + l8) * row_bytes + 16u * ch;
  const uint32_t s_off = (MG == 1 ? half * 2 * I + 2 * r8 : (uint32_t)(lane & 15)) * 4u;

  // a pass' own: where its weights and tokens are, and the block scales of the wave's steps, one to a lane (e4m3)
  struct Own {
    bool there;
    int expert, i0;
    uint32_t x_off[MG];
    float beta[2];
  };
  auto own_of = [&](const UpItem& t, bool there) {
    Own o;
    o.there = there;
    o.expert = there ? t.expert : 0;
    o.i0 = t.i0;
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const int r = t.m0 + 8 * g + l8;
      o.x_off[g] = there && r < t.m ? (s.table.entry[t.start + r] >> 16) * H * 2u + 16u * P * ch : kOOB;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      o.beta[b] = 0.f;
      if constexpr (FMT == kFp8) {  // [2 I / 128][KB] fp32
        const __amdgpu_buffer_rsrc_t r = make_rsrc(static_cast<const uint8_t*>(p.s1) + (int64_t)o.expert * s_bytes, there ? s_bytes : 0u);
        o.beta[b] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            r, lane < n ? (uint32_t)(lo + lane) * 4u : kOOB, (uint32_t)((b * p.I + o.i0) >> 7) * (uint32_t)KB * 4u, 0));
      }
    }
    return o;
  };

  u32x4 w[D][2][2 * C];
  u32x2 sc[D][2][C];
  u32x4 xr[D][MG][P];
  // step i of a pass into stage d; empty ranges past its last step: zeros, and no traffic; so are the upper chunks of a last
  // half step of e2m1
  auto load = [&](int d, const Own& o, int i) {
    const bool in = o.there && i < n;
    const uint32_t k = in ? (uint32_t)(lo + i) : 0u;
    const bool over = FMT == kFp4 && (k + 1) * 256u > H;
    const bool cut = over && ch >= 4;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w1 + (int64_t)o.expert * w_bytes, in ? w_bytes : 0u);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, in ? (uint32_t)p.T * H * 2u : 0u);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int a = 0; a < 2 * C; ++a)
        w[d][b][a] = __builtin_amdgcn_raw_buffer_load_b128(rw, cut ? kOOB : w_off[a], (b * I + (uint32_t)o.i0) * row_bytes + k * 128u, NT ? kStream : 0);
    if constexpr (FMT == kFp4) {  // the words of step k are 2 k and 2 k + 1 of a row
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(static_cast<const uint8_t*>(p.s1) + (int64_t)o.expert * s_bytes, in ? s_bytes : 0u);
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if constexpr (MG == 1) {
          sc[d][b][0] = __builtin_amdgcn_raw_buffer_load_b64(rs, over && half ? kOOB : s_off, (k * 4u * I + b * I + (uint32_t)o.i0) * 4u, 0);
        } else {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const uint32_t at = (k * 4u * I + b * I + (uint32_t)o.i0) * 4u;
            sc[d][b][c][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, s_off + 64u * c, at, 0);
            sc[d][b][c][1] = __builtin_amdgcn_raw_buffer_load_b32(rs, over ? kOOB : s_off + 64u * c, at + 8u * I, 0);
          }
        }
    }
#pragma unroll
    for (int g = 0; g < MG; ++g)
#pragma unroll
      for (int t = 0; t < P; ++t)
        xr[d][g][t] = __builtin_amdgcn_raw_buffer_load_b128(rx, cut || o.x_off[g] == kOOB ? kOOB : o.x_off[g] + 16u * t, k * 2u * kStepDepth<FMT>, 0);
  };

  Own cur = own_of(it, true);
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, cur, d);
  for (;;) {
    UpItem next = it;
    bool left = true;
    if (it.m0 + 8 * MG < it.m) next.m0 += 8 * MG;
    else if (it.u + C * run.step < run.end) next = up_item(s, it.u + C * run.step, 0, tiles);
    else left = false;
    const bool on = left && up_groups<MAXMG>(next) == MG && up_units<MAXMG>(next, run) == C;
    const Own then = own_of(next, on);
    constexpr int Q = MG == 1 ? 2 : MG / 2;  // accumulators of 16 rows: of the rows 2 i and 2 i + 1, or of 16 tokens each
    f32x4 c[C][2][Q];
#pragma unroll
    for (int n2 = 0; n2 < C; ++n2)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int a = 0; a < Q; ++a) c[n2][b][a] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < padded; k0 += D) {
      const bool ahead = k0 + D >= padded;  // the loads of this turn are the next pass'
      Own o = cur;
      if (ahead) o = then;
#pragma unroll
      for (int d = 0; d < D; ++d) {
        __builtin_amdgcn_sched_barrier(0);
        // a lane's: a wave has at most 64 steps, and past them lanes hold zero, or the step's products are zero
        const int i = k0 + d < 63 ? k0 + d : 63;
        float beta[2] = {1.f, 1.f};
        if constexpr (FMT == kFp8)
#pragma unroll
          for (int b = 0; b < 2; ++b) beta[b] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(cur.beta[b]), i));
        auto add = [&](int n2, int b, int a, f32x4 z) {
          if constexpr (FMT == kFp8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[n2][b][a][e] = __builtin_fmaf(z[e], beta[b], c[n2][b][a][e]);
          } else {
            c[n2][b][a] = z;
          }
        };
        if constexpr (MG == 1) {
          u32x4 y[P];
#pragma unroll
          for (int t = 0; t < P; ++t) y[t] = spread(sp, t, xr[d][0][t]);
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              const float ex = FMT == kFp4 ? exponent_of(sc[d][b][0][a], q) : 1.f;
              const u32x4 chunk = spread(sp, a, w[d][b][a]);
              f32x4 z = FMT == kFp8 ? f32x4{0.f, 0.f, 0.f, 0.f} : c[0][b][a];
#pragma unroll
              for (int t = 0; t < P; ++t) z = mfma(widened<FMT>(chunk, t, ex), y[t], z);
              add(0, b, a, z);
            }
        } else {
          u32x4 y[MG / 2][P][2];
#pragma unroll
          for (int g = 0; g < MG; g += 2)
#pragma unroll
            for (int t = 0; t < P; ++t) spread16(sp, xr[d][g][t], xr[d][g + 1][t], y[g / 2][t]);
#pragma unroll
          for (int n2 = 0; n2 < C; ++n2)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              u32x4 chunk[2];
              spread16(sp, w[d][b][2 * n2], w[d][b][2 * n2 + 1], chunk);
              f32x4 z[Q];
#pragma unroll
              for (int a = 0; a < Q; ++a) z[a] = FMT == kFp8 ? f32x4{0.f, 0.f, 0.f, 0.f} : c[n2][b][a];
#pragma unroll
              for (int s2 = 0; s2 < 2; ++s2) {
                const float ex = FMT == kFp4 ? exponent_of(sc[d][b][n2][s2], q) : 1.f;
#pragma unroll
                for (int t = 0; t < P; ++t) {
                  const bf16x8 v = widened<FMT>(chunk[s2], t, ex);
#pragma unroll
                  for (int a = 0; a < Q; ++a) z[a] = mfma(v, y[a][t][s2], z[a]);
                }
              }
#pragma unroll
              for (int a = 0; a < Q; ++a) add(n2, b, a, z[a]);
            }
        }
        load(d, o, ahead ? d : k0 + D + d);
      }
    }
    // the waves' sums, in order: `part` has four places of 16 lanes for every 16 accumulators of a column
    const int at = MG == 1 ? r8 | (q << 3) : lane & 15;
    const bool mine = MG > 1 || (!half && q < 2);  // one row of tokens: lanes (token r8, q < 2) of the lower half have weight rows 8 q + 2 e + a
    auto place = [&](int b, int a) { return MG == 1 ? b * 2 + a : (a * 2 + b) * 4 + q; };
#pragma unroll
    for (int n2 = 0; n2 < C; ++n2) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int a = 0; a < Q; ++a) {
          if constexpr (MG == 1) c[n2][b][a] = halves(c[n2][b][a]);
          if (wave > 0 && mine) sh.part[turn][wave - 1][place(b, a)][at] = c[n2][b][a];
        }
      __syncthreads();  // (the other half of `part` is what the next pass writes)
      if (wave == 0 && mine) {
        f32x4 v[Q];
#pragma unroll
        for (int a = 0; a < Q; ++a) {
          f32x4 z[2] = {c[n2][0][a], c[n2][1][a]};
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int u = 0; u < 3; ++u) z[b] += sh.part[turn][u][place(b, a)][at];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[a][e] = activate<kActSilu>(z[0][e]) * z[1][e];
        }
        if constexpr (MG == 1) {
          const int r = it.m0 + r8;
          if (r < it.m)
            *reinterpret_cast<uint4*>(p.h + (int64_t)(s.table.entry[it.start + r] & 0xffffu) * p.I + it.i0 + 8 * q) =
                uint4{pack_bf16x2(v[0][0], v[1][0]), pack_bf16x2(v[0][1], v[1][1]), pack_bf16x2(v[0][2], v[1][2]), pack_bf16x2(v[0][3], v[1][3])};
        } else {
#pragma unroll
          for (int a = 0; a < Q; ++a) {
            const int r = it.m0 + 16 * a + (lane & 15);
            if (r < it.m)
              *reinterpret_cast<uint2*>(p.h + (int64_t)(s.table.entry[it.start + r] & 0xffffu) * p.I + it.i0 + 16 * n2 + 4 * q) =
                  uint2{pack_bf16x2(v[a][0], v[a][1]), pack_bf16x2(v[a][2], v[a][3])};
          }
        }
      }
      turn ^= 1;
    }
    it = next;
    if (!on) return left;
    cur = then;
  }
}

template <int FMT, int MAXMG, bool NT>
__global__ void __launch_bounds__(kUpThreads) experts_up_kernel(ExpertsParams p) {
  __shared__ UpShared<MAXMG> sh;
  read_members(p, sh.members);
  const int tiles = p.I >> 4;
  const int units = __builtin_amdgcn_readfirstlane(sh.members.table.n) * tiles;
  int first = (int)blockIdx.x;
  UpRun run{units, 0};
  if (units == 0) return;
  if (MAXMG > 2 && entries_of(sh.members.table) > kPairTokens * sh.members.table.n) {  // a run of neighbouring units, one more for some workgroups than for others
    const int n = units < (int)gridDim.x ? units : (int)gridDim.x;
    if (first >= n) return;
    run.end = (int)((int64_t)(first + 1) * units / n);
    first = (int)((int64_t)first * units / n);
    run.step = 1;
  } else {  // as many workgroups as give each the same number of units, or one less
    const int rounds = (units + (int)gridDim.x - 1) / (int)gridDim.x;
    run.step = (units + rounds - 1) / rounds;
    if (first >= run.step) return;
  }
  UpItem it = up_item(sh.members, first, 0, tiles);
  int turn = 0;
  for (bool left = true; left;) {
    const int g = up_groups<MAXMG>(it), c = up_units<MAXMG>(it, run);
    if (g == 1) left = up_passes<FMT, 1, 1, MAXMG, NT>(p, sh, it, run, turn);
    else if (g == 2 && c == 1) left = up_passes<FMT, 2, 1, MAXMG, NT>(p, sh, it, run, turn);
    else if constexpr (MAXMG > 2) {
      if (g == 2) left = up_passes<FMT, 2, 2, MAXMG, NT>(p, sh, it, run, turn);
      else if (c == 1) left = up_passes<FMT, 4, 1, MAXMG, NT>(p, sh, it, run, turn);
      else left = up_passes<FMT, 4, 2, MAXMG, NT>(p, sh, it, run, turn);
    }
  }
}

// ---- down projection and weighted sum.  A workgroup takes 16 columns of y for all tokens (where experts have many tokens 32, and
// twice as many workgroups share them: h is loaded half as often); its waves, and those of all workgroups of the columns, take equal runs of the steps of all chosen experts, one expert after the other, with the
// next steps' loads in flight across experts.  The tokens of an expert share its steps, 8 MG at a time (one group).  When the
// group changes, the accumulators times the tokens' weights are added to the wave's sums of the tokens in LDS, so that a
// token's experts are added in the order of their numbers.
constexpr int kDownCols = 16;
// waves of a workgroup: eight, two workgroups to a CU, where 8 tokens at most leave the registers for it; else four of twice the
// registers
template <bool FEW>
constexpr int kDownWaves = FEW ? 8 : 4;

// Steps in flight.  128 registers leave room for two workgroups of eight waves a CU, 256 for two of four.
template <int FMT, bool FEW>
constexpr int down_depth(int mg, int c) {
  if (c == 2) return FMT == kFp8 ? (mg == 2 ? 3 : 2) : mg == 2 ? 2 : 1;
  if (FMT == kFp8) return FEW ? 4 : mg == 1 ? 5 : mg == 2 ? 3 : 2;
  return FEW ? 2 : mg == 1 ? 3 : mg == 2 ? 2 : 1;
}

// the wave's part: its run of the steps, into its sums of 16 C columns
template <int FMT, int MG, int C, bool FEW, bool NT>
__device__ __forceinline__ void down_run(const ExpertsParams& p, const ExpertsTable& s, f32x4* sums, u32x4* slots_of_wave, int c0, int slot, int slots) {
  constexpr int D = down_depth<FMT, FEW>(MG, C);
  constexpr int P = kParts<FMT>;
  const int lane = threadIdx.x & 63;
  const int r8 = lane & 7, half = (lane >> 3) & 1, q = lane >> 4;
  const uint32_t H = (uint32_t)p.H, I = (uint32_t)p.I;
  const uint32_t row_bytes = FMT == kFp8 ? I : I / 2;
  const int KS = (int)((row_bytes + 127) >> 7);  // steps of an expert
  const int steps = __builtin_amdgcn_readfirstlane(s.n) * KS;  // (a step of all of an expert's groups: which of them a token is in changes no sum)
  const int per = (steps + slots - 1) / slots;
  const int lo = slot * per < steps ? slot * per : steps;
  const int hi = lo + per < steps ? lo + per : steps;

  if (lo < hi) {
    const int KB = p.I >> 7;
    const uint32_t w_bytes = H * row_bytes;
    // loads: row (or token) lane / 8, chunk lane % 8; weight rows c0 + 2 (lane / 8) + a
    const int l8 = lane >> 3, ch = lane & 7;
    const Spread sp = spread_of(slots_of_wave);
    uint32_t w_off[2 * C];
#pragma unroll
    for (int a = 0; a < 2 * C; ++a) w_off[a] = (uint32_t)(c0 + (MG == 1 ? 2 * l8 + a : 8 * a + l8)) * row_bytes + 16u * ch;
    // scales: e4m3 [ceil(H / 128)][KB] fp32, e2m1 words [KB][H]
    const uint32_t s_bytes = FMT == kFp8 ? ((H + 127) >> 7) * (uint32_t)KB * 4u : (uint32_t)KB * H * 4u;
    const uint32_t s_off = FMT == kFp8 ? (uint32_t)(c0 >> 7) * (uint32_t)KB * 4u
                           : MG == 1    ? (half * H + (uint32_t)(c0 + 2 * r8)) * 4u
                                        : (uint32_t)(c0 + (lane & 15)) * 4u;
    const uint32_t s_step = FMT == kFp8 ? 4u : 8u * H;
    const uint32_t h_bytes = (uint32_t)p.T * (uint32_t)p.k * I * 2u;

    // what is loaded next: step ld_k of [k_lo, k_hi) of expert ld_a of the list, group ld_g of its ld_n; the lane's rows of h,
    // weights and tokens.  An expert's groups take its steps one after the other (32 tokens of one group are common, more rare).
    int ld_a = lo / KS;
    int k_lo = lo - ld_a * KS, k_hi = 0, left = hi - lo;  // steps of the run past k_hi
    int ld_k = k_lo, ld_g = 0, ld_n = 1, first = 0, members = 0;
    const uint8_t* wbase = p.w2;
    const uint8_t* sbase = static_cast<const uint8_t*>(p.s2);
    constexpr int N = MG == 1 ? 1 : MG / 2;  // tokens of a lane's columns: one of 8, or one of every 16
    uint32_t h_off[MG];
    float fac[N];
    int token[N];
    auto enter_expert = [&]() {
      const uint32_t r = __builtin_amdgcn_readfirstlane(s.run[ld_a]);
      const int e = expert_of(r);
      wbase = p.w2 + (int64_t)e * w_bytes;
      sbase = static_cast<const uint8_t*>(p.s2) + (int64_t)e * s_bytes;
      first = start_of(r);
      members = count_of(r);
      ld_n = (members + 8 * MG - 1) / (8 * MG);
      k_hi = KS - k_lo < left ? KS : k_lo + left;
      left -= k_hi - k_lo;
    };
    auto enter_group = [&]() {
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        const int r = 8 * (MG * ld_g + g);
        h_off[g] = r + l8 < members ? (s.entry[first + r + l8] & 0xffffu) * I * 2u + 16u * P * ch : kOOB;
      }
#pragma unroll
      for (int g = 0; g < N; ++g) {
        const int r = 8 * MG * ld_g + (MG == 1 ? r8 : 16 * g + (lane & 15));
        fac[g] = r < members ? s.weight[first + r] : 0.f;
        token[g] = r < members ? (int)(s.entry[first + r] >> 16) : -1;
      }
    };
    enter_expert();
    enter_group();
    bool fresh = true;  // the next load begins a group of tokens

    u32x4 w[D][2 * C];
    u32x2 sc[D][C];
    u32x4 hr[D][MG][P];
    float fr[D][N];
    int tr[D][N];
    bool nr[D], vr[D];
    int gr[D];  // groups of 8 that hold a token
    auto load = [&](int d) {
      if (ld_k == k_hi && (ld_g + 1 < ld_n || left > 0)) {
        if (++ld_g == ld_n) {
          ++ld_a;
          ld_g = k_lo = 0;
          enter_expert();
        }
        ld_k = k_lo;
        enter_group();
        fresh = true;
      }
      const bool in = ld_k < k_hi;
      // past the run's last step the ranges are empty: zeros, and no traffic
      const __amdgpu_buffer_rsrc_t rw = make_rsrc(wbase, in ? w_bytes : 0u);
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(sbase, in ? s_bytes : 0u);
      const __amdgpu_buffer_rsrc_t rh = make_rsrc(p.h, in ? h_bytes : 0u);
      const uint32_t k = in ? (uint32_t)ld_k : 0u;
      const bool over = FMT == kFp4 && (k + 1) * 256u > I;  // a last half step has no upper chunks
      const bool cut = over && ch >= 4;
#pragma unroll
      for (int a = 0; a < 2 * C; ++a) w[d][a] = __builtin_amdgcn_raw_buffer_load_b128(rw, cut ? kOOB : w_off[a], k * 128u, NT ? kStream : 0);
      if constexpr (FMT == kFp8) sc[d][0][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, s_off, k * s_step, 0);
      else if constexpr (MG == 1) sc[d][0] = __builtin_amdgcn_raw_buffer_load_b64(rs, over && half ? kOOB : s_off, k * s_step, 0);
      else {
#pragma unroll
        for (int n2 = 0; n2 < C; ++n2) {
          sc[d][n2][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, s_off + 64u * n2, k * s_step, 0);
          sc[d][n2][1] = __builtin_amdgcn_raw_buffer_load_b32(rs, over ? kOOB : s_off + 64u * n2, k * s_step + 4u * H, 0);
        }
      }
#pragma unroll
      for (int g = 0; g < MG; ++g)
#pragma unroll
        for (int t = 0; t < P; ++t)
          hr[d][g][t] = __builtin_amdgcn_raw_buffer_load_b128(rh, cut || h_off[g] == kOOB ? kOOB : h_off[g] + 16u * t, k * 2u * kStepDepth<FMT>, 0);
#pragma unroll
      for (int g = 0; g < N; ++g) {
        fr[d][g] = fac[g];
        tr[d][g] = token[g];
      }
      nr[d] = fresh;
      vr[d] = in;
      gr[d] = (members - 8 * MG * ld_g + 7) >> 3;
      fresh = false;
      if (in) ++ld_k;
    };
    constexpr int Q = MG == 1 ? 2 : N;  // accumulators: of the rows 2 i and 2 i + 1, or of 16 tokens each
    f32x4 acc[C][Q];
    int to[N];
    float by[N];
    auto clear = [&]() {
#pragma unroll
      for (int n2 = 0; n2 < C; ++n2)
#pragma unroll
        for (int a = 0; a < Q; ++a) acc[n2][a] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    // the accumulators into the sums: of 8 tokens lanes (token r8, q < 2) of the lower half have columns 8 q + 2 e + a
    auto flush = [&]() {
      wave_fence();  // a token's sums may be another lane's from the expert before
      if constexpr (MG == 1) {
        const f32x4 x = halves(acc[0][0]), y = halves(acc[0][1]);
        if (to[0] >= 0 && !half && q < 2) {
          f32x4* at = &sums[to[0] * (kDownCols / 4) + 2 * q];
          at[0] += f32x4{x[0], y[0], x[1], y[1]} * by[0];
          at[1] += f32x4{x[2], y[2], x[3], y[3]} * by[0];
        }
      } else {
#pragma unroll
        for (int a = 0; a < Q; ++a)
          if (to[a] >= 0)
#pragma unroll
            for (int n2 = 0; n2 < C; ++n2) sums[to[a] * (C * kDownCols / 4) + 4 * n2 + q] += acc[n2][a] * by[a];
      }
    };
#pragma unroll
    for (int g = 0; g < N; ++g) {
      to[g] = -1;
      by[g] = 0.f;
    }
    clear();
#pragma unroll
    for (int d = 0; d < D; ++d) load(d);
    bool any = false, more = true;
    while (more) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        __builtin_amdgcn_sched_barrier(0);
        if (nr[d] && vr[d]) {  // uniform
          if (any) flush();
          any = true;
#pragma unroll
          for (int g = 0; g < N; ++g) {
            to[g] = tr[d][g];
            by[g] = fr[d][g];
          }
          clear();
        }
        auto add = [&](int n2, int a, f32x4 o) {
          if constexpr (FMT == kFp8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n2][a][e] = __builtin_fmaf(o[e], __uint_as_float(sc[d][0][0]), acc[n2][a][e]);
          } else {
            acc[n2][a] = o;
          }
        };
        if constexpr (MG == 1) {
          u32x4 x[P];
#pragma unroll
          for (int t = 0; t < P; ++t) x[t] = spread(sp, t, hr[d][0][t]);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const float ex = FMT == kFp4 ? exponent_of(sc[d][0][a], q) : 1.f;
            const u32x4 chunk = spread(sp, a, w[d][a]);
            f32x4 o = FMT == kFp8 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[0][a];
#pragma unroll
            for (int t = 0; t < P; ++t) o = mfma(widened<FMT>(chunk, t, ex), x[t], o);
            add(0, a, o);
          }
        } else {
          bf16x8 v[C][2][P];
#pragma unroll
          for (int n2 = 0; n2 < C; ++n2) {
            u32x4 chunk[2];
            spread16(sp, w[d][2 * n2], w[d][2 * n2 + 1], chunk);
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) {
              const float ex = FMT == kFp4 ? exponent_of(sc[d][n2][s2], q) : 1.f;
#pragma unroll
              for (int t = 0; t < P; ++t) v[n2][s2][t] = widened<FMT>(chunk[s2], t, ex);
            }
          }
#pragma unroll
          for (int a = 0; a < Q; ++a) {
            if (a > 0 && 2 * a >= gr[d]) break;  // uniform
            f32x4 o[C];
#pragma unroll
            for (int n2 = 0; n2 < C; ++n2) o[n2] = FMT == kFp8 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[n2][a];
#pragma unroll
            for (int t = 0; t < P; ++t) {
              u32x4 x[2];
              spread16(sp, hr[d][2 * a][t], hr[d][2 * a + 1][t], x);
#pragma unroll
              for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                for (int n2 = 0; n2 < C; ++n2) o[n2] = mfma(v[n2][s2][t], x[s2], o[n2]);
            }
#pragma unroll
            for (int n2 = 0; n2 < C; ++n2) add(n2, a, o[n2]);
          }
        }
        load(d);
      }
      more = vr[0];
    }
    flush();
  }
}

template <int FMT, bool FEW, bool NT>
__global__ void __launch_bounds__(64 * kDownWaves<FEW>, FEW ? 4 : 2) experts_down_kernel(ExpertsParams p) {
  constexpr int W = kDownWaves<FEW>;
  constexpr int THREADS = 64 * W;
  __shared__ ExpertsTable s;
  __shared__ __attribute__((aligned(16))) f32x4 sums[W][(FEW ? 8 : 2 * kExpertsMaxTokens) * (kDownCols / 4)];  // [token][four columns]
  __shared__ __attribute__((aligned(16))) u32x4 spread_s[W][64 * kSpreadSlots];
  __shared__ int last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  {
    const int n = p.T * p.k;
    for (int i = threadIdx.x; i < n; i += THREADS) {
      s.run[i] = p.table->run[i];
      s.entry[i] = p.table->entry[i];
      s.weight[i] = p.table->weight[i];
    }
    if (threadIdx.x == 0) s.n = p.table->n;
  }
  for (int i = lane; i < (FEW ? 1 : 2) * p.T * (kDownCols / 4); i += 64) sums[wave][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  // tokens of an expert on average: an expert of more takes its steps group by group
  const int chosen = __builtin_amdgcn_readfirstlane(s.n), entries = entries_of(s);
  const bool wide = !FEW && entries > kPairTokens * chosen;
  const int cols = wide ? 2 * kDownCols : kDownCols, splits = wide ? 2 * p.splits : p.splits;
  const int tile = (int)blockIdx.x / splits, split = (int)blockIdx.x - tile * splits;
  const int c0 = tile * cols;
  const int slot = split * W + wave, slots = W * splits;
  if (!wide) down_run<FMT, 1, 1, FEW, NT>(p, s, sums[wave], spread_s[wave], c0, slot, slots);
  if constexpr (!FEW) {
    // (16 tokens a pass against 32, e4m3: 8 of an expert 140.1 and 143.6 us, 12: 81.4 and 81.5, 24: 59.3 and 51.0; e2m1 100.7 and
    // 107, 61.1 and 62.1, 49.8 and 45.0)
    if (wide && entries <= 12 * chosen) down_run<FMT, 2, 2, FEW, NT>(p, s, sums[wave], spread_s[wave], c0, slot, slots);
    else if (wide) down_run<FMT, 4, 2, FEW, NT>(p, s, sums[wave], spread_s[wave], c0, slot, slots);
  }
  __syncthreads();
  // the waves' sums in order: a thread takes four columns of a token, of 32 columns two times four
  constexpr int E = FEW ? 1 : 2;
  const int fours = p.T * cols / 4;
  f32x4 y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int u = threadIdx.x + THREADS * e;
    y[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (u < fours)
#pragma unroll
      for (int o = 0; o < W; ++o) y[e] += sums[o][u];
  }
  if (splits > 1) {
    // The workgroups' sums meet in the workspace: sc1 stores and loads are coherent across the XCDs' L2 caches; every wave's
    // stores are acknowledged (vmcnt 0) before the barrier that precedes the relaxed counter increment, and the last
    // workgroup loads only after its own increment has returned.  It adds them in order and leaves the counter at zero.
    const uint32_t one = (uint32_t)fours * 16u;
    const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.partials, (uint32_t)splits * (uint32_t)p.H * (uint32_t)p.T * 4u);
    uint32_t off[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int u = threadIdx.x + THREADS * e;
      off[e] = u < fours ? ((uint32_t)tile * (uint32_t)splits + (uint32_t)split) * one + (uint32_t)u * 16u : kOOB;
      asm volatile("" : "+v"(off[e]));
    }
    // All addresses first, and the stores back to back: a register of a 16-byte store that the next instruction overwrites can
    // reach memory overwritten (the compiler keeps one instruction between them only where the scalar offset is a constant, and
    // the split's place in that register had single words of 2 in 56 calls wrong).
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int e = 0; e < E; ++e) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[e]), rp, off[e], 0, kCoherent);
    wait_vmcnt<0>();
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    if (threadIdx.x == 0)
      last = __hip_atomic_fetch_add(&p.counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned int)(splits - 1);
    __syncthreads();
    if (!last) return;
    if (threadIdx.x == 0) __hip_atomic_store(&p.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    uint32_t from[E];  // of the first split
#pragma unroll
    for (int e = 0; e < E; ++e) {
      from[e] = off[e] == kOOB ? kOOB : off[e] - (uint32_t)split * one;
      y[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (int i0 = 0; i0 < splits; i0 += 4) {  // four in flight; past the last, an empty place
      f32x4 t[E][4];
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[e][i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rp, i0 + i < splits ? from[e] : kOOB, (uint32_t)(i0 + i < splits ? i0 + i : 0) * one, kCoherent));
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[e] += t[e][i];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int u = threadIdx.x + THREADS * e;
    if (u < fours)
      *reinterpret_cast<uint2*>(p.y + (int64_t)(u / (cols / 4)) * p.H + c0 + 4 * (u % (cols / 4))) =
          uint2{pack_bf16x2(y[e][0], y[e][1]), pack_bf16x2(y[e][2], y[e][3])};
  }
}

template <int FMT, bool NT>
hipError_t launch_format(const ExpertsParams& p, int cus, hipStream_t stream) {
  const int64_t most = (int64_t)(p.G < p.T * p.k ? p.G : p.T * p.k) * (p.I / 16);  // units, where every choice names another expert
  // workgroups a CU: what the registers let be there at once, but for e2m1 of up to 16 tokens, whose 191 hold two of the three
  const int64_t room = (int64_t)(p.T <= 16 ? 3 : 2) * cus;
  const dim3 up((unsigned)(most < room ? most : room));
  if (p.T <= 16) hipLaunchKernelGGL((experts_up_kernel<FMT, 2, NT>), up, dim3(kUpThreads), 0, stream, p);
  else hipLaunchKernelGGL((experts_up_kernel<FMT, 4, NT>), up, dim3(kUpThreads), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)(p.H / kDownCols * p.splits));
  if (p.T <= 8) hipLaunchKernelGGL((experts_down_kernel<FMT, true, NT>), grid, dim3(64 * kDownWaves<true>), 0, stream, p);
  else hipLaunchKernelGGL((experts_down_kernel<FMT, false, NT>), grid, dim3(64 * kDownWaves<false>), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

// Workgroups that share 16 columns of the down projection: as many as give the chip eight waves a CU, with two steps a wave
int experts_splits(int64_t T, int64_t choices, int64_t H, int64_t I, int64_t G, int cus) {
  const int64_t tiles = H / kDownCols;
  if (tiles > 1024) return 1;  // counters
  const int waves = T <= 8 ? kDownWaves<true> : kDownWaves<false>;
  const int64_t steps = (G < choices ? G : choices) * (I / 128);
  int64_t s = 8 * (int64_t)cus / waves / tiles;
  if (s > steps / (2 * waves)) s = steps / (2 * waves);
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

size_t experts_h_bytes(int64_t choices, int64_t I) { return ((size_t)choices * (size_t)I * 2 + 255) / 256 * 256; }

hipError_t launch_moe_experts(const ExpertsParams& p, bool fp4, bool stream_weights, int cus, hipStream_t stream) {
  if (fp4) return stream_weights ? launch_format<kFp4, true>(p, cus, stream) : launch_format<kFp4, false>(p, cus, stream);
  return stream_weights ? launch_format<kFp8, true>(p, cus, stream) : launch_format<kFp8, false>(p, cus, stream);
}

}  // namespace dg
