// Gradient of a product's epilogue D = act(z) + residual, z = A . B^T + bias,
// for gfx950:
//   dz = dy act'(z)   (bf16, and as e4m3 codes with one fp32 scale per 128)
//   dbias = sum over rows of dz
// (the residual's gradient is dy itself).  dz is quantised and summed before it
// is rounded to bf16.
//
// HBM-bound: dy and z are read once, dz and its codes written once.  A wave
// takes 512 columns of a row, 8 a lane, so 16 lanes hold a scale's group; a
// workgroup a run of consecutive rows, so that it fills whole cache lines of the
// MN-major scales, and sums the bias' gradient in registers over them.  The
// workgroups' sums meet in launch_column_sum, in order.  4096 x 4096 with the
// erf gelu, codes and bias (118 MB) 26.7 us, 4.4 TB/s, and 4.9 for the bias;
// beside the loads the vector units are busy 0.84 of the cycles there (the slope
// of the gelu and the quotients).

#include "activation.hpp"
#include "block_internal.hpp"
#include "e4m3.hpp"
#include "rows8.hpp"

namespace dg {
namespace {

constexpr int kBatch = 2;  // rows in flight of a wave

// one rounded product, not fused with the sum it goes into: the bias' gradient is the same whatever else is asked for
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

template <int ACT, bool QUANT>
__global__ void __launch_bounds__(256) epilogue_bwd_kernel(EpilogueBwdParams p) {
  __shared__ __attribute__((aligned(16))) float sums[3][512];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = blockIdx.x * 512 + lane * 8;
  const bool in = c < p.N;
  const int64_t lo = (int64_t)blockIdx.y * p.rows_per_wg;
  const int64_t hi = lo + p.rows_per_wg < p.M ? lo + p.rows_per_wg : p.M;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t r0 = lo + wave; r0 < hi; r0 += 4 * kBatch) {
    Raw8<true> d[kBatch], z[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t r = r0 + 4 * i;
      d[i] = z[i] = Raw8<true>{};
      if (in && r < hi) {
        d[i] = load8<true>(p.dy, r * p.N + c);
        if constexpr (ACT != kActNone) z[i] = load8<true>(p.pre, r * p.N + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t r = r0 + 4 * i;
      if (r >= hi) break;  // uniform
      float v[8], s[8];
      values(d[i], v);
      if constexpr (ACT != kActNone) {
        values(z[i], s);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = product(v[e], activate_slope<ACT>(s[e]));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[e];
      if (p.dz && in) store8<true>(p.dz, r * p.N + c, rounded<true>(v));
      if constexpr (QUANT) {  // N is a multiple of 128: a group's lanes are all inside or all outside
        const float s_ = scale_of(group_amax(v));
        float y[8];
        quotients_of<8>(v, y, s_);
        if (in) {
          *reinterpret_cast<uint2*>(p.q + r * p.N + c) = uint2{e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7])};
          if ((lane & 15) == 0) p.sf[(int64_t)(c >> 7) * p.M + r] = s_;
        }
      }
    }
  }
  if (!p.partials) return;
  if (wave > 0) {
    float4* at = reinterpret_cast<float4*>(&sums[wave - 1][lane * 8]);
    at[0] = float4{acc[0], acc[1], acc[2], acc[3]};
    at[1] = float4{acc[4], acc[5], acc[6], acc[7]};
  }
  __syncthreads();
  if (wave > 0 || !in) return;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += sums[w][lane * 8 + e];
  float4* at = reinterpret_cast<float4*>(p.partials + (int64_t)blockIdx.y * p.N + c);
  at[0] = float4{acc[0], acc[1], acc[2], acc[3]};
  at[1] = float4{acc[4], acc[5], acc[6], acc[7]};
}

template <int ACT>
void bwd_act(const EpilogueBwdParams& p, dim3 grid, hipStream_t stream) {
  if (p.q) hipLaunchKernelGGL((epilogue_bwd_kernel<ACT, true>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((epilogue_bwd_kernel<ACT, false>), grid, dim3(256), 0, stream, p);
}

}  // namespace

// Rows of a workgroup: a multiple of 8 (four waves, two rows in flight each), as many workgroups as eight to a CU, at most 1024
// of them down the rows (4096 x 4096 with gelu, codes and bias: four rows in flight and four workgroups 31 us, two and four 29,
// two and eight 27)
static int64_t most_down(int64_t N, int cus) {
  const int64_t cols = (N + 511) / 512;
  const int64_t down = (8 * (int64_t)cus + cols - 1) / cols;
  return down < 1024 ? down : 1024;
}
int64_t epilogue_bwd_rows(int64_t M, int64_t N, int cus) {
  const int64_t down = most_down(N, cus);
  const int64_t rows = (M + down - 1) / down;
  return (rows + 7) / 8 * 8;
}
int64_t epilogue_bwd_partials(int64_t M, int64_t N, int cus) {
  const int64_t down = most_down(N, cus);
  return (M + 7) / 8 < down ? (M + 7) / 8 : down;
}

hipError_t launch_epilogue_bwd(const EpilogueBwdParams& p, int act, hipStream_t stream) {
  const int64_t down = (p.M + p.rows_per_wg - 1) / p.rows_per_wg;
  if (down > 0) {  // without rows only the bias' gradient is written: zeros
    const dim3 grid((unsigned)((p.N + 511) / 512), (unsigned)down);
    switch (act) {
      case kActNone: bwd_act<kActNone>(p, grid, stream); break;
      case kActRelu: bwd_act<kActRelu>(p, grid, stream); break;
      case kActSilu: bwd_act<kActSilu>(p, grid, stream); break;
      case kActGelu: bwd_act<kActGelu>(p, grid, stream); break;
      default: bwd_act<kActGeluTanh>(p, grid, stream); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p.partials) return hipSuccess;
  return launch_column_sum(p.partials, p.dbias, down, p.N, stream);
}

}  // namespace dg
