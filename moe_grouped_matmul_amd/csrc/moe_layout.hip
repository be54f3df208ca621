// From the experts chosen for each token to the row order of the grouped
// products, on the device.  idx holds n = T * k choices in (token, choice)
// order; expert g (of the G held here, g = idx - first) owns
//   contiguous: a segment of rows that starts at a multiple of 128, segments
//               in expert order;
//   masked:     rows [g max_m, g max_m + max_m), choices past max_m dropped;
// and its choices take its rows in (token, choice) order, so the layout is a
// function of idx alone.
//
// Up to 2048 choices one workgroup and one launch do everything.  Beyond, a
// first launch writes the counts of each block of choices (1024, or what makes
// at most 128 blocks) and every workgroup of the second sums the columns of
// counts before its own block and over all blocks, so no workgroup waits for
// another.  Inside a workgroup every wave counts its own run of choices, the
// waves' counts are summed in order, and a wave ranks 64 choices at a time by
// matching their experts bit by bit.  Rows that hold nothing are known from
// the counts alone, so their -1 needs no order against the placement; the
// workgroups share them.
//
// The traffic is a megabyte or two: what bounds it is launch latency, the
// dependent steps, and the scattered 4-byte stores of row_token and m_indices
// that one CU passes on (one line a cycle); blocks are many for those and few
// for the columns of counts that every workgroup reads.  Measured: 256 tokens x
// 8 in one launch 4.3 us; 16384 x 8 of 64 experts 9.4 us (2.4 the counts);
// 131072 x 8 of 256 experts 28 us with 128 blocks, 29 with 256, 49 with 512;
// a million x 8 222 us, 2.1 ms with blocks of 2048.
#include <type_traits>

#include "dg_internal.hpp"
#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

constexpr int kLayThreads = 1024;  // also the most experts: a thread per expert
constexpr int kLayWaves = kLayThreads / 64;
constexpr int kLaySingle = 2;       // 64-choice chunks of a wave where one workgroup places all
constexpr int kLayMaxBlocks = 128;  // their counts are read by every workgroup
constexpr int kLayBatch = 8;        // counts a thread has in flight
constexpr int kLaySlices = 16;      // threads that share an expert's column of counts

__device__ __forceinline__ int local_expert(int v, int first, int G) {
  const int g = v - first;  // v < 0 (no expert) never lands in range: first >= 0
  return v >= 0 && g >= 0 && g < G ? g : -1;
}

// 64-choice chunks of each wave; one block: kLaySingle
int chunks_of(int64_t n) {
  if (n <= (int64_t)kLaySingle * kLayThreads) return kLaySingle;
  return (int)((n + (int64_t)kLayThreads * kLayMaxBlocks - 1) / ((int64_t)kLayThreads * kLayMaxBlocks));
}
int blocks_of(int64_t n) {
  const int64_t per = (int64_t)chunks_of(n) * kLayThreads;
  return n > 0 ? (int)((n + per - 1) / per) : 1;
}

// Counts of a block in the workspace: a block of up to kLaySingle chunks a wave has at most 2048 choices, which 16 bits hold.
template <int C>
using Count = std::conditional_t<C != 0, uint16_t, int32_t>;
static_assert(kLaySingle * kLayThreads < 65536, "16-bit counts");

// counts[block][g], behind the workspace's counters: choices of expert g in the block
template <int C>
__global__ void __launch_bounds__(kLayThreads) layout_count_kernel(LayoutParams p, int chunks) {
  __shared__ int hist[kLayThreads];
  hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * chunks * kLayThreads + threadIdx.x;
  for (int c = 0; c < chunks; ++c) {
    const int64_t i = i0 + (int64_t)c * kLayThreads;
    const int g = i < p.n ? local_expert(p.idx[i], p.first, p.G) : -1;
    if (g >= 0) atomicAdd(&hist[g], 1);
  }
  __syncthreads();
  Count<C>* counts = reinterpret_cast<Count<C>*>(static_cast<uint8_t*>(p.ws) + kWsCounterBytes);
  if ((int)threadIdx.x < p.G) counts[(int64_t)blockIdx.x * p.G + threadIdx.x] = (Count<C>)hist[threadIdx.x];
}

// workgroups [0, blocks) place their block; all share the rows that hold
// nothing.  C: chunks of a wave, held in registers (0: `chunks`, read twice)
template <int C>
__global__ void __launch_bounds__(kLayThreads) layout_place_kernel(LayoutParams p, int blocks, int chunks, int slots) {
  __shared__ int next[kLayWaves][kLayThreads];  // next row (rank when masked) of each expert, per wave
  __shared__ int start_of[kLayThreads + 1];     // first row of each expert's segment (contiguous)
  __shared__ int count_of[kLayThreads];
  __shared__ int part[2][kLayThreads];          // a slice's sum of a column, before this block and in all
  __shared__ int wsum[kLayWaves];
  const int b = (int)blockIdx.x;
  const int tid = threadIdx.x;
  const int wave = tid >> 6;
  const int lane = tid & 63;
  const int G = p.G;
  const bool placing = b < blocks;
  const bool single = blocks == 1;
  const int nc = C ? C : chunks;
  if (tid < G) {
#pragma unroll
    for (int w = 0; w < kLayWaves; ++w) next[w][tid] = 0;
  }
  // the wave's own choices (one block: every workgroup counts it, for the totals)
  const int64_t w0 = (int64_t)(single ? 0 : b) * nc * kLayThreads + (int64_t)wave * nc * 64;
  const auto choice = [&](int c) {
    const int64_t i = w0 + 64 * c + lane;
    return (placing || single) && i < p.n ? local_expert(p.idx[i], p.first, G) : -1;
  };
  int e[C ? C : 1];
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) e[c] = choice(c);
  }
  // choices of each expert before this block, and in all: `slots` (a power of
  // two) experts side by side, each column cut into slices of blocks
  if (!single) {
    const int g = tid & (slots - 1);
    const int slice = tid / slots;
    const int slices = kLayThreads / slots < kLaySlices ? kLayThreads / slots : kLaySlices;
    int before = 0, total = 0;
    if (g < G && slice < slices) {
      const Count<C>* col = reinterpret_cast<const Count<C>*>(static_cast<const uint8_t*>(p.ws) + kWsCounterBytes) + g;
      for (int c0 = slice; c0 < blocks; c0 += kLayBatch * slices) {
        int v[kLayBatch];
#pragma unroll
        for (int c = 0; c < kLayBatch; ++c) v[c] = c0 + c * slices < blocks ? col[(int64_t)(c0 + c * slices) * G] : 0;
#pragma unroll
        for (int c = 0; c < kLayBatch; ++c) {
          before += c0 + c * slices < b ? v[c] : 0;
          total += v[c];
        }
      }
    }
    part[0][tid] = before;
    part[1][tid] = total;
  }
  __syncthreads();
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (e[c] >= 0) atomicAdd(&next[wave][e[c]], 1);
  } else {
    for (int c = 0; c < nc; ++c) {
      const int g = choice(c);
      if (g >= 0) atomicAdd(&next[wave][g], 1);
    }
  }
  int before = 0, total = 0;
  if (!single && tid < G) {
    for (int i = tid; i < kLayThreads && i < slots * kLaySlices; i += slots) {
      before += part[0][i];
      total += part[1][i];
    }
  }
  __syncthreads();
  if (single && tid < G) {
#pragma unroll
    for (int w = 0; w < kLayWaves; ++w) total += next[w][tid];
  }
  // first rows: exclusive prefix of the padded segment lengths
  int start = 0;
  if (!p.max_m) {
    const int own = (total + 127) & ~127;
    int v = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(v, o);
      if (lane >= o) v += u;
    }
    if (lane == 63) wsum[wave] = v;
    __syncthreads();
    start = v - own;
#pragma unroll
    for (int w = 0; w < kLayWaves; ++w) start += w < wave ? wsum[w] : 0;
    start_of[tid] = start;
    if (tid == kLayThreads - 1) start_of[kLayThreads] = start + own;
  }
  if (tid < G) {
    const int held = p.max_m && total > p.max_m ? (int)p.max_m : total;
    count_of[tid] = held;
    if (b == 0) p.counts[tid] = held;
    int run = start + before;
#pragma unroll
    for (int w = 0; w < kLayWaves; ++w) {
      const int c = next[w][tid];
      next[w][tid] = run;
      run += c;
    }
  }
  __syncthreads();
  if (placing) {
    int bits = 1;
    while ((1 << bits) <= G) ++bits;  // codes 0 .. G (G: none)
    const auto place = [&](int c, int g) __attribute__((always_inline)) {
      const int64_t i = w0 + 64 * c + lane;
      const int code = g < 0 ? G : g;
      unsigned long long same = ~0ull;  // lanes with this lane's expert
      for (int k = 0; k < bits; ++k) {
        const unsigned long long m = __ballot((code >> k) & 1);
        same &= (code >> k) & 1 ? m : ~m;
      }
      const int rank = __popcll(same & ((1ull << lane) - 1ull));
      int row = -1;
      if (g >= 0) {
        const int64_t at = (int64_t)next[wave][g] + rank;
        if (p.max_m) row = at < p.max_m ? (int)((int64_t)g * p.max_m + at) : -1;
        else row = at < p.rows ? (int)at : -1;
      }
      __builtin_amdgcn_wave_barrier();  // LDS accesses of a wave are in order: read above, then advanced
      if (g >= 0 && rank == 0) next[wave][g] += __popcll(same);
      __builtin_amdgcn_wave_barrier();
      if (i < p.n) {
        p.row_of[i] = row;
        if (row >= 0) {
          p.row_token[row] = (int)((uint32_t)i / (uint32_t)p.k);
          if (p.m_indices) p.m_indices[row] = g;
        }
      }
    };
    // the wave's choices in order
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (w0 + 64 * c < p.n) place(c, e[c]);  // uniform
    } else {
      for (int c = 0; c < nc && w0 + 64 * c < p.n; ++c) place(c, choice(c));
    }
  }
  // rows that hold nothing, shared by all workgroups
  const int64_t stride = (int64_t)gridDim.x * kLayThreads;
  if (p.max_m) {
    for (int64_t r = (int64_t)b * kLayThreads + tid; r < p.rows; r += stride) {
      const uint32_t g = (uint32_t)r / (uint32_t)p.max_m;
      if ((int)((uint32_t)r - g * (uint32_t)p.max_m) >= count_of[g]) p.row_token[r] = -1;
    }
    return;
  }
  for (int g = b * kLayWaves + wave; g < G; g += (int)gridDim.x * kLayWaves) {  // a wave behind each expert's choices
    const int64_t lo = (int64_t)start_of[g] + count_of[g];
    int64_t hi = (int64_t)start_of[g] + ((count_of[g] + 127) & ~127);
    if (hi > p.rows) hi = p.rows;
    for (int64_t r = lo + lane; r < hi; r += 64) {
      p.row_token[r] = -1;
      p.m_indices[r] = -1;
    }
  }
  for (int64_t r = start_of[kLayThreads] + (int64_t)b * kLayThreads + tid; r < p.rows; r += stride) {  // behind the last segment
    p.row_token[r] = -1;
    p.m_indices[r] = -1;
  }
}

}  // namespace

// The first kWsCounterBytes are left as they are: other operators keep counters there that have to be zero between calls.
// A single block uses nothing of it.
static size_t workspace_of(size_t counts, int chunks) {
  return kWsCounterBytes + (chunks <= kLaySingle ? sizeof(Count<1>) : sizeof(Count<0>)) * counts;
}
size_t layout_workspace_needed(int64_t n, int64_t G) {
  const size_t counts = (size_t)blocks_of(n) * (size_t)G;
  return blocks_of(n) == 1 ? 4 * counts : workspace_of(counts, chunks_of(n));
}
// What is asked for grows with n, so that a buffer for the most choices serves fewer (131073 choices make 65 blocks, 131072
// make 128), and is no less than 4 bytes a count.
size_t layout_workspace_bytes(int64_t n, int64_t G) {
  if (blocks_of(n) == 1) return layout_workspace_needed(n, G);
  const int64_t most = (n + kLayThreads - 1) / kLayThreads;
  const size_t counts = (size_t)(most < kLayMaxBlocks ? most : kLayMaxBlocks) * (size_t)G;
  const size_t bytes = workspace_of(counts, chunks_of(n));
  return bytes > 4 * counts ? bytes : 4 * counts;
}

hipError_t launch_layout(const LayoutParams& p, hipStream_t stream) {
  const int blocks = blocks_of(p.n);
  const int chunks = chunks_of(p.n);
  int slots = 1;
  while (slots < p.G) slots *= 2;
  auto count = chunks <= kLaySingle ? layout_count_kernel<1> : layout_count_kernel<0>;
  if (blocks > 1) hipLaunchKernelGGL(count, dim3(blocks), dim3(kLayThreads), 0, stream, p, chunks);
  // further workgroups where the rows outnumber the choices
  const int64_t f = (p.rows + 4 * kLayThreads - 1) / (4 * kLayThreads);
  const int fill = (int)(f < 256 ? f : 256);
  auto kernel = chunks == kLaySingle ? layout_place_kernel<kLaySingle> : chunks == 1 ? layout_place_kernel<1> : layout_place_kernel<0>;
  hipLaunchKernelGGL(kernel, dim3(blocks > fill ? blocks : fill), dim3(kLayThreads), 0, stream, p, blocks, chunks, slots);
  return hipGetLastError();
}

}  // namespace dg
