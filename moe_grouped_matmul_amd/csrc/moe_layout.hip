// From the experts chosen for each token to the row order of the grouped
// products, on the device.  idx holds n = T * k choices in (token, choice)
// order; expert g (of the G held here, g = idx - first) owns
//   contiguous: a segment of rows that starts at a multiple of 128, segments
//               in expert order;
//   masked:     rows [g max_m, g max_m + max_m), choices past max_m dropped;
// and its choices take its rows in (token, choice) order, so the layout is a
// function of idx alone.
//
// Three launches: counts per block of choices (and the fill of the row
// arrays), a scan over blocks and experts, and the placement.

#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

constexpr int kLayMaxGroups = 1024;
constexpr int kLayThreads = 256;
constexpr int kLayWaves = kLayThreads / 64;
constexpr int kLayItems = 2048;  // choices per block
constexpr int kLayWaveItems = kLayItems / kLayWaves;

__device__ __forceinline__ int local_expert(int v, int first, int G) {
  const int g = v - first;  // v < 0 (no expert) never lands in range: first >= 0
  return v >= 0 && g >= 0 && g < G ? g : -1;
}

// ws[block][g]: choices of expert g in the block; row arrays filled with -1
__global__ void __launch_bounds__(kLayThreads) layout_count_kernel(LayoutParams p) {
  __shared__ int hist[kLayMaxGroups];
  const int b = (int)blockIdx.x;
  for (int g = threadIdx.x; g < p.G; g += kLayThreads) hist[g] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)b * kLayItems;
  for (int64_t i = i0 + threadIdx.x; i < p.n && i < i0 + kLayItems; i += kLayThreads) {
    const int g = local_expert(p.idx[i], p.first, p.G);
    if (g >= 0) atomicAdd(&hist[g], 1);
  }
  __syncthreads();
  int* out = static_cast<int*>(p.ws) + (int64_t)b * p.G;
  for (int g = threadIdx.x; g < p.G; g += kLayThreads) out[g] = hist[g];
  for (int64_t r = (int64_t)b * kLayThreads + threadIdx.x; r < p.rows; r += (int64_t)gridDim.x * kLayThreads) {
    p.row_token[r] = -1;
    if (p.m_indices) p.m_indices[r] = -1;
  }
}

// in place: ws[block][g] becomes the first row of the block's choices of g (relative to the
// expert's first row when masked: the rank is needed there); counts written
__global__ void __launch_bounds__(kLayMaxGroups) layout_scan_kernel(LayoutParams p, int blocks) {
  __shared__ int wsum[kLayMaxGroups / 64];
  const int g = threadIdx.x;
  int* ws = static_cast<int*>(p.ws);
  int run = 0;
  if (g < p.G) {
    for (int b = 0; b < blocks; ++b) {
      const int c = ws[(int64_t)b * p.G + g];
      ws[(int64_t)b * p.G + g] = run;
      run += c;
    }
    p.counts[g] = p.max_m && run > p.max_m ? (int)p.max_m : run;
  }
  if (p.max_m) return;
  // exclusive prefix of the segment lengths
  int v = g < p.G ? (run + 127) / 128 * 128 : 0;
  const int own = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if ((g & 63) >= o) v += u;
  }
  if ((g & 63) == 63) wsum[g >> 6] = v;
  __syncthreads();
  int start = v - own;
  for (int i = 0; i < (g >> 6); ++i) start += wsum[i];
  if (g < p.G)
    for (int b = 0; b < blocks; ++b) {
      ws[(int64_t)b * p.G + g] += start;  // n + 128 G < 2^31: every row number is an int
    }
}

__global__ void __launch_bounds__(kLayThreads) layout_place_kernel(LayoutParams p) {
  __shared__ int next[kLayWaves][kLayMaxGroups];  // next row (rank when masked) of each expert, per wave
  const int b = (int)blockIdx.x;
  const int wave = threadIdx.x >> 6;
  const int lane = threadIdx.x & 63;
  const int* base = static_cast<const int*>(p.ws) + (int64_t)b * p.G;
  for (int i = threadIdx.x; i < kLayWaves * p.G; i += kLayThreads) next[i / p.G][i % p.G] = 0;
  __syncthreads();
  const int64_t w0 = (int64_t)b * kLayItems + (int64_t)wave * kLayWaveItems;
  const int64_t w1 = w0 + kLayWaveItems < p.n ? w0 + kLayWaveItems : p.n;
  for (int64_t i = w0 + lane; i < w1; i += 64) {
    const int g = local_expert(p.idx[i], p.first, p.G);
    if (g >= 0) atomicAdd(&next[wave][g], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < p.G; g += kLayThreads) {
    int run = base[g];
#pragma unroll
    for (int w = 0; w < kLayWaves; ++w) {
      const int c = next[w][g];
      next[w][g] = run;
      run += c;
    }
  }
  __syncthreads();
  int bits = 1;
  while ((1 << bits) <= p.G) ++bits;  // codes 0 .. G (G: none)
  for (int64_t i = w0; i < w1; i += 64) {  // uniform: the wave's choices in order
    const bool in = i + lane < w1;
    const int g = in ? local_expert(p.idx[i + lane], p.first, p.G) : -1;
    const int code = g < 0 ? p.G : g;
    unsigned long long same = ~0ull;  // lanes with this lane's expert
    for (int k = 0; k < bits; ++k) {
      const unsigned long long m = __ballot((code >> k) & 1);
      same &= (code >> k) & 1 ? m : ~m;
    }
    const int before = __popcll(same & ((1ull << lane) - 1ull));
    int row = -1;
    if (g >= 0) {
      const int first = next[wave][g];
      const int64_t at = (int64_t)first + before;
      if (p.max_m)
        row = at < p.max_m ? (int)((int64_t)g * p.max_m + at) : -1;
      else
        row = at < p.rows ? (int)at : -1;
    }
    __builtin_amdgcn_wave_barrier();
    if (g >= 0 && before == 0) next[wave][g] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      p.row_of[i + lane] = row;
      if (row >= 0) {
        p.row_token[row] = (int)((i + lane) / p.k);
        if (p.m_indices) p.m_indices[row] = g;
      }
    }
  }
}

}  // namespace

size_t layout_workspace_bytes(int64_t n, int64_t G) {
  const int64_t blocks = n > 0 ? (n + kLayItems - 1) / kLayItems : 1;
  return (size_t)(blocks * G * 4);
}

hipError_t launch_layout(const LayoutParams& p, hipStream_t stream) {
  const int blocks = (int)(p.n > 0 ? (p.n + kLayItems - 1) / kLayItems : 1);
  hipLaunchKernelGGL(layout_count_kernel, dim3(blocks), dim3(kLayThreads), 0, stream, p);
  hipLaunchKernelGGL(layout_scan_kernel, dim3(1), dim3(kLayMaxGroups), 0, stream, p, blocks);
  if (p.n > 0) hipLaunchKernelGGL(layout_place_kernel, dim3(blocks), dim3(kLayThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
