// Root-mean-square norm of a row and its residual for gfx950, with its output
// as it is and / or as e4m3 codes with one scale per 128 (the left operand of
// the FP8 products), and its gradient:
//   h = rnd(x + residual),  r = 1 / sqrt(mean(h^2) + eps),  v = (h r) w
//   y = rnd(v);  q, sf = the 1x128 quantisation of v (quant.hip states it)
//   dx = dh + r (w dy - n mean(w dy n)),  n = h r;   dw = sum over rows of dy n
// The norm is of h as it is stored (rounded to its type): what the backward
// pass reads is then what the forward pass normalised.  Sums and statistics
// are fp32, v is quantised before any rounding.
//
// HBM-bound: a row stays in the registers of its waves between the sum of its
// squares and the outputs, so x and the residual are read once, and nothing is
// written that is not asked for.  16384 x 7168 bf16 with residual and codes
// (826 MB) 145-150 us, 5.5-5.7 TB/s, the vector units busy 0.77 of the cycles
// beside; 8192 x 4096 bf16 with residual (268 MB) 52 us, its gradient (as many)
// 47 us and 4.8 for the weight's.  One row of 7168 is a launch and a chain of
// loads, sum and quotients: 3.6 us.

#include "block_internal.hpp"
#include "e4m3.hpp"
#include "rows8.hpp"

namespace dg {
namespace {

// NW waves take a row, CH runs of 8 values a lane: run i of wave w is the
// 512 columns from (i NW + w) 512 on, so that 16 lanes hold one 128-column
// group and a wave's run one word of power-of-two scales.
template <bool BF16, int KIND, int CH, int NW, bool NT>
__global__ void __launch_bounds__(NW <= 4 ? 256 : 64 * NW) rms_norm_kernel(NormParams p) {
  constexpr int ROWS = NW <= 4 ? 4 / NW : 1;  // of a workgroup
  __shared__ float part[ROWS][NW];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = wave / NW, w = wave % NW;
  // the 64 workgroups of a run take their row blocks so that each XCD's eight
  // are neighbours: the scales of neighbouring rows share cache lines
  int blk = blockIdx.x;
  if ((blk | 63) < (int)gridDim.x) blk = (blk & ~63) | ((blk & 7) << 3) | ((blk >> 3) & 7);
  const int64_t row = (int64_t)blk * ROWS + slot;
  const bool live = row < p.M;
  const int64_t at = (live ? row : 0) * p.K;
  const int K = p.K;
  Raw8<BF16> h[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = ((i * NW + w) * 64 + lane) * 8;
    h[i] = Raw8<BF16>{};
    if (live && c < K) h[i] = load8<BF16, NT>(p.x, at + c);
  }
  if (p.residual) {
    Raw8<BF16> r[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = ((i * NW + w) * 64 + lane) * 8;
      r[i] = Raw8<BF16>{};
      if (live && c < K) r[i] = load8<BF16, NT>(p.residual, at + c);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float a[8], b[8];
      values(h[i], a);
      values(r[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += b[e];
      h[i] = rounded<BF16>(a);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = ((i * NW + w) * 64 + lane) * 8;
    float a[8];
    values(h[i], a);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(a[e], a[e], sum);
    if (p.h && live && c < K) store8<BF16, NT>(p.h, at + c, h[i]);
  }
  sum = wave_sum(sum);
  if constexpr (NW > 1) {
    if (lane == 0) part[slot][w] = sum;
    __syncthreads();
    sum = part[slot][0];
#pragma unroll
    for (int i = 1; i < NW; ++i) sum += part[slot][i];
  }
  if (!live) return;
  const float r = 1.f / sqrtf(sum / (float)K + p.eps);
  if (p.rstd && w == 0 && lane == 0) p.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int run = i * NW + w;
    const int c = (run * 64 + lane) * 8;
    const bool in = c < K;
    float v[8], g[8];
    values(h[i], v);
    // (past K whole groups are outside, and nothing of them is kept)
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 0.f;
    if (in) weights8(p.weight, p.weight_bf16, c, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (v[e] * r) * g[e];
    if (p.y && in) store8<BF16, NT>(p.y, at + c, rounded<BF16>(v));
    if constexpr (KIND != kNoQuant) {
      const float amax = group_amax(v);
      const int kb = run * 4 + (lane >> 4);
      uint2 out;
      if constexpr (KIND == kScaleUe8m0) {
        const int code = ue8m0_code(amax);
        const float inv = __builtin_ldexpf(1.f, 127 - code);
        out.x = pack4_pow2(v[0], v[1], v[2], v[3], inv);
        out.y = pack4_pow2(v[4], v[5], v[6], v[7], inv);
        // a run is one word of four codes, those past K zero
        if ((lane & 15) == 0 && run * 512 < K)
          (static_cast<uint8_t*>(p.sf) + ((int64_t)run * p.M + row) * 4)[lane >> 4] = in ? (uint8_t)code : 0;
      } else {
        const float s = scale_of(amax);
        float y[8];
        quotients_of<8>(v, y, s);
        out.x = e4m3x4(y[0], y[1], y[2], y[3]);
        out.y = e4m3x4(y[4], y[5], y[6], y[7]);
        if ((lane & 15) == 0 && in) static_cast<float*>(p.sf)[(int64_t)kb * p.M + row] = s;
      }
      (void)kb;
      if (in) {
        typedef unsigned int raw2 __attribute__((ext_vector_type(2)));
        if constexpr (NT) __builtin_nontemporal_store(raw2{out.x, out.y}, reinterpret_cast<raw2*>(p.q + at + c));
        else *reinterpret_cast<uint2*>(p.q + at + c) = out;
      }
    }
  }
}

// A workgroup of 8 waves takes 8 / NW rows at a time; the gradient of the
// weight is summed in registers over all its rows, then over its slots, and
// written as one row of partials that launch_column_sum joins.  Two workgroups
// a CU, so the partials are 512 rows at most (8 MB of a row of 4096).
template <bool BF16, int CH, int NW>
__global__ void __launch_bounds__(512) rms_norm_bwd_kernel(NormBwdParams p) {
  constexpr int SLOTS = 8 / NW;
  __shared__ float part[2][SLOTS][NW];
  __shared__ __attribute__((aligned(16))) float acc_s[SLOTS > 1 ? CH * NW * 512 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = wave / NW, w = wave % NW;
  const int K = p.K;
  float acc[CH][8];
  float g[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = ((i * NW + w) * 64 + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = g[i][e] = 0.f;
    if (c < K) weights8(p.weight, p.weight_bf16, c, g[i]);
  }
  const int64_t step = (int64_t)gridDim.x * SLOTS;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * SLOTS; r0 < p.M; r0 += step, turn ^= 1) {  // uniform over the workgroup
    const int64_t row = r0 + slot;
    const bool live = row < p.M;
    const int64_t at = (live ? row : 0) * K;
    Raw8<BF16> d[CH], h[CH], o[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = ((i * NW + w) * 64 + lane) * 8;
      d[i] = h[i] = o[i] = Raw8<BF16>{};
      if (live && c < K) {
        d[i] = load8<BF16>(p.dy, at + c);
        h[i] = load8<BF16>(p.h, at + c);
        if (p.dh) o[i] = load8<BF16>(p.dh, at + c);
      }
    }
    const float r = live ? p.rstd[row] : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float a[8], b[8];
      values(d[i], a);
      values(h[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = b[e] * r;
        acc[i][e] = __builtin_fmaf(a[e], n, acc[i][e]);
        sum = __builtin_fmaf(a[e] * g[i][e], n, sum);
      }
    }
    sum = wave_sum(sum);
    if constexpr (NW > 1) {
      if (lane == 0) part[turn][slot][w] = sum;
      __syncthreads();  // (the other half of `part` is what the next rows write)
      sum = part[turn][slot][0];
#pragma unroll
      for (int i = 1; i < NW; ++i) sum += part[turn][slot][i];
    }
    const float m = sum / (float)K;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = ((i * NW + w) * 64 + lane) * 8;
      float a[8], b[8], t[8];
      values(d[i], a);
      values(h[i], b);
      values(o[i], t);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] += r * (a[e] * g[i][e] - (b[e] * r) * m);
      if (live && c < K) store8<BF16>(p.dx, at + c, rounded<BF16>(t));
    }
  }
  if constexpr (SLOTS > 1) {  // slots in order
    for (int s = 1; s < SLOTS; ++s) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float4* at = reinterpret_cast<float4*>(acc_s + ((i * NW + w) * 64 + lane) * 8);
        if (slot == s) {
          at[0] = float4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
          at[1] = float4{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
        }
      }
      __syncthreads();
      if (slot == 0)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const float* at = acc_s + ((i * NW + w) * 64 + lane) * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[i][e] += at[e];
        }
    }
  }
  if (slot != 0) return;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = ((i * NW + w) * 64 + lane) * 8;
    if (c >= K) continue;
    float4* at = reinterpret_cast<float4*>(p.partials + (int64_t)blockIdx.x * K + c);
    at[0] = float4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    at[1] = float4{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
  }
}

// 64 columns x 16 slices of rows a workgroup; rows are `stride` apart
constexpr int kSumCols = 64;
constexpr int kSumSlices = 16;
constexpr int kSumMostCols = 1 << 27;  // of a launch: 16 threads a column, and thread counts are 32 bits
__global__ void __launch_bounds__(64 * 16) column_sum_kernel(const float* __restrict__ partials, float* __restrict__ out,
                                                                          int64_t rows, int N, int64_t stride) {
  __shared__ float s[kSumSlices][kSumCols];
  const int col = threadIdx.x % kSumCols, sl = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + col;
  const int64_t per = (rows + kSumSlices - 1) / kSumSlices;
  const int64_t hi = (sl + 1) * per < rows ? (sl + 1) * per : rows;
  float a = 0.f;
  if (c < N) {
    for (int64_t r = sl * per; r < hi; r += 8) {  // eight rows in flight
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r + i < hi ? partials[(r + i) * stride + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a += v[i];
    }
  }
  s[sl][col] = a;
  __syncthreads();
  if (sl == 0 && c < N) {
#pragma unroll
    for (int i = 1; i < kSumSlices; ++i) a += s[i][col];
    out[c] = a;
  }
}

// runs of 512 columns that a lane holds of a row
constexpr int kMostRuns = 4;

template <bool BF16, int KIND, int CH, int NW>
void norm_one(const NormParams& p, bool nt, hipStream_t stream) {
  constexpr int ROWS = NW <= 4 ? 4 / NW : 1;
  const dim3 grid((unsigned)((p.M + ROWS - 1) / ROWS)), wg(NW <= 4 ? 256 : 64 * NW);
  if constexpr (NW == 1 || CH == kMostRuns)  // (shapes of many rows: the others are for few)
    if (nt) {
      hipLaunchKernelGGL((rms_norm_kernel<BF16, KIND, CH, NW, true>), grid, wg, 0, stream, p);
      return;
    }
  hipLaunchKernelGGL((rms_norm_kernel<BF16, KIND, CH, NW, false>), grid, wg, 0, stream, p);
}

template <bool BF16, int KIND, int NW>
void norm_runs(const NormParams& p, int ch, bool nt, hipStream_t stream) {
  constexpr int MOST = kNormMaxK / 512 / NW < kMostRuns ? kNormMaxK / 512 / NW : kMostRuns;
  if (ch <= 1) return norm_one<BF16, KIND, 1, NW>(p, nt, stream);
  if (ch <= 2) return norm_one<BF16, KIND, 2, NW>(p, nt, stream);
  if constexpr (MOST >= 4) norm_one<BF16, KIND, 4, NW>(p, nt, stream);
}

template <bool BF16, int KIND>
hipError_t norm_shape(const NormParams& p, int cus, hipStream_t stream) {
  // The fewest waves a row with four runs a lane, more while that leaves the chip's waves idle.  (A row of 14 runs by one wave
  // of 16, two of 8 and four of 4: 16384 x 7168 with codes 202, 167 and 162 us: with fewer registers more rows are in flight.)
  const int runs = (p.K + 511) / 512;
  int nw = 1;
  while (nw < 16 && (nw * kMostRuns < runs || (nw < runs && p.M * nw < 16 * cus))) nw *= 2;
  const int ch = (runs + nw - 1) / nw;
  // Rows that the 256 MB Infinity Cache cannot hold are streamed past it, in and out (16384 x 7168 bf16 173 -> 162 us; 1021 x
  // 2048 fp32, which it holds from one call to the next: 7.6 -> 8.6, so not there; 8192 x 4096 bf16 with its backward pass: no
  // difference)
  const int64_t row = (int64_t)p.K * (BF16 ? 2 : 4);
  const bool nt = p.M * (row * (1 + (p.residual != nullptr) + (p.h != nullptr) + (p.y != nullptr)) + (p.q ? p.K : 0)) >= (int64_t)512 << 20;
  switch (nw) {
    case 1: norm_runs<BF16, KIND, 1>(p, ch, nt, stream); break;
    case 2: norm_runs<BF16, KIND, 2>(p, ch, nt, stream); break;
    case 4: norm_runs<BF16, KIND, 4>(p, ch, nt, stream); break;
    case 8: norm_runs<BF16, KIND, 8>(p, ch, nt, stream); break;
    default: norm_runs<BF16, KIND, 16>(p, ch, nt, stream); break;
  }
  return hipGetLastError();
}

// waves a row and runs a lane of the backward kernel: two runs (four above 8192 columns)
struct BwdShape {
  int nw, ch;
};
BwdShape bwd_shape(int64_t K) {
  const int runs = (int)((K + 511) / 512);
  BwdShape s{1, 1};
  while (s.nw < 8 && s.nw * 2 < runs) s.nw *= 2;
  s.ch = (runs + s.nw - 1) / s.nw;
  return s;
}

template <bool BF16>
hipError_t bwd_launch(const NormBwdParams& p, int cus, hipStream_t stream) {
  const BwdShape s = bwd_shape(p.K);
  const dim3 grid((unsigned)norm_bwd_grid(p.M, p.K, cus)), wg(512);
#define DG_BWD(CH, NW) hipLaunchKernelGGL((rms_norm_bwd_kernel<BF16, CH, NW>), grid, wg, 0, stream, p)
  if (s.nw == 1) {
    if (s.ch == 1) DG_BWD(1, 1);
    else DG_BWD(2, 1);
  } else if (s.nw == 2) {
    DG_BWD(2, 2);
  } else if (s.nw == 4) {
    DG_BWD(2, 4);
  } else if (s.ch <= 2) {
    DG_BWD(2, 8);
  } else {
    DG_BWD(4, 8);
  }
#undef DG_BWD
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormParams& p, bool bf16, int kind, int cus, hipStream_t stream) {
#define DG_KIND(B)                                                       \
  (kind == kScaleF32 ? norm_shape<B, kScaleF32>(p, cus, stream)          \
                     : kind == kScaleUe8m0 ? norm_shape<B, kScaleUe8m0>(p, cus, stream) : norm_shape<B, kNoQuant>(p, cus, stream))
  return bf16 ? DG_KIND(true) : DG_KIND(false);
#undef DG_KIND
}

// workgroups of the backward kernel, each of which leaves a row of partials
int norm_bwd_grid(int64_t M, int64_t K, int cus) {
  const int slots = 8 / bwd_shape(K).nw;
  const int64_t need = (M + slots - 1) / slots;
  return (int)(need < 2 * cus ? need : 2 * cus);
}

hipError_t launch_rms_norm_bwd(const NormBwdParams& p, bool bf16, int cus, hipStream_t stream) {
  if (p.M > 0) {
    const hipError_t e = bf16 ? bwd_launch<true>(p, cus, stream) : bwd_launch<false>(p, cus, stream);
    if (e != hipSuccess) return e;
  }
  return launch_column_sum(p.partials, p.dw, norm_bwd_grid(p.M, p.K, cus), p.K, stream);
}

hipError_t launch_column_sum(const float* partials, float* out, int64_t rows, int N, hipStream_t stream) {
  for (int64_t c = 0; c < N; c += kSumMostCols) {
    const int n = (int)(N - c < kSumMostCols ? N - c : kSumMostCols);
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((n + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumSlices), 0, stream, partials + c,
                       out + c, rows, n, (int64_t)N);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace dg
