// Expert rows back to tokens, and the gradient, for gfx950:
//   y[t] = sum_j w[t, j] * rows[row_of[t, j]]
//   drows[row_of[t, j]] = w[t, j] * dy[t],   dw[t, j] = <rows[row_of[t, j]], dy[t]>
// over the choices j whose row is in [0, R).  rows and drows are bf16, sums
// are held in fp32 and rounded once; the order of a token's sum is that of its
// choices.
//
// HBM-bound: every chosen row is read once (forward and, for dw, backward) or
// written once (drows); 8 columns of a token are one 16-byte load per choice,
// and all choices' loads are issued before the first is used.  A wave takes a
// run of columns of a token, or a choice of the backward pass: workgroups would
// idle on short rows (2569 tokens x 8 x 320 with the gradient, a workgroup and
// a wave each: 20 and 12 us; 256 x 8 x 7168 20.6 and 18.1).  Rows that the
// Infinity Cache cannot hold from one call to the next are streamed past it,
// and y and drows with them (non-temporal), and then the backward pass takes a
// whole token per workgroup, which reads its dy once (4096 x 8 x 7168 279 us
// against 291, 1024 x 8 x 4096 38 against 46), unless a token's rows are too
// short for that.  Measured, bf16, 4096 tokens x 8 x 7168: forward 90 us (5.9
// TB/s), backward 188 us (5.3 TB/s); 256 tokens x 8 x 7168, held by the
// Infinity Cache, 6.8 us forward.

#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

template <bool NT>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  if constexpr (!NT) return *reinterpret_cast<const uint4*>(p);
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return uint4{v.x, v.y, v.z, v.w};
}

template <bool NT>
__device__ __forceinline__ void store16(void* p, uint4 a) {
  const u32x4 v{a.x, a.y, a.z, a.w};
  if constexpr (NT) __builtin_nontemporal_store(v, static_cast<u32x4*>(p));
  else *static_cast<u32x4*>(p) = v;
}

__device__ __forceinline__ void bf16x8(uint4 w, float* v) {
  v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
  v[4] = __uint_as_float(w.z << 16); v[5] = __uint_as_float(w.z & 0xffff0000u);
  v[6] = __uint_as_float(w.w << 16); v[7] = __uint_as_float(w.w & 0xffff0000u);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

template <bool BF16>
__device__ __forceinline__ void values8(const void* x, int64_t at, float* d) {
  if constexpr (BF16) {
    bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at), d);
  } else {
    const float* s = static_cast<const float*>(x) + at;
    const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
    d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w; d[4] = b.x; d[5] = b.y; d[6] = b.z; d[7] = b.w;
  }
}

// A wave takes 512 columns of one token, a thread 8 of them with the rows of eight
// choices in flight; a choice without a row reads nothing.
constexpr int kCombBatch = 8;
template <bool BF16, bool NT>
__global__ void __launch_bounds__(256) combine_kernel(const uint16_t* __restrict__ rows, const int32_t* __restrict__ row_of,
                                                      const float* __restrict__ w, void* __restrict__ y, int k, int N,
                                                      int64_t R, int64_t T, int parts) {
  const unsigned unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int64_t t = unit / (unsigned)parts;
  const int c = (int)(unit - (unsigned)t * (unsigned)parts) * 512 + (threadIdx.x & 63) * 8;
  if (t >= T || c >= N) return;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < k; j0 += kCombBatch) {
    uint4 raw[kCombBatch];
    float wj[kCombBatch];
#pragma unroll
    for (int j = 0; j < kCombBatch; ++j) {
      raw[j] = uint4{0u, 0u, 0u, 0u};
      wj[j] = 0.f;
      if (j0 + j < k) {  // uniform, and so is the row
        const int64_t r = row_of[t * k + j0 + j];
        if (r >= 0 && r < R) {
          wj[j] = w[t * k + j0 + j];
          raw[j] = load8<NT>(rows + r * N + c);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kCombBatch; ++j) {
      float v[8];
      bf16x8(raw[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(wj[j], v[i], s[i]);
    }
  }
  if constexpr (BF16) {
    store16<NT>(static_cast<uint16_t*>(y) + t * N + c, pack8(s));
  } else {
    float* d = static_cast<float*>(y) + t * N + c;
    store16<NT>(d, uint4{__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]), __float_as_uint(s[3])});
    store16<NT>(d + 4, uint4{__float_as_uint(s[4]), __float_as_uint(s[5]), __float_as_uint(s[6]), __float_as_uint(s[7])});
  }
}

// one wave per (token, choice)
template <bool BF16>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const void* __restrict__ dy, const uint16_t* __restrict__ rows,
                                                          const int32_t* __restrict__ row_of, const float* __restrict__ w,
                                                          uint16_t* __restrict__ drows, float* __restrict__ dw, int k, int N,
                                                          int64_t R, int64_t T) {
  const unsigned i = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int lane = threadIdx.x & 63;
  const int64_t t = i / (unsigned)k;
  if (t >= T) return;
  const int64_t r = row_of[i];
  if (r < 0 || r >= R) {  // uniform
    if (lane == 0) dw[i] = 0.f;
    return;
  }
  const float wj = w[i];
  float dot = 0.f;
  for (int c = lane * 8; c < N; c += 512) {
    float v[8], d[8], o[8];
    bf16x8(load8<false>(rows + r * N + c), v);
    values8<BF16>(dy, t * N + c, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dot = __builtin_fmaf(v[e], d[e], dot);
      o[e] = wj * d[e];
    }
    *reinterpret_cast<uint4*>(drows + r * N + c) = pack8(o);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) dot += __shfl_xor(dot, o);
  if (lane == 0) dw[i] = dot;
}

// one workgroup per token, rows and drows streamed
template <bool BF16>
__global__ void __launch_bounds__(256) combine_bwd_token_kernel(const void* __restrict__ dy, const uint16_t* __restrict__ rows,
                                                                const int32_t* __restrict__ row_of,
                                                                const float* __restrict__ w, uint16_t* __restrict__ drows,
                                                                float* __restrict__ dw, int k, int N, int64_t R) {
  __shared__ float part[kCombBatch][4];
  const int64_t t = blockIdx.x;
  for (int j0 = 0; j0 < k; j0 += kCombBatch) {
    float dot[kCombBatch];
#pragma unroll
    for (int j = 0; j < kCombBatch; ++j) dot[j] = 0.f;
    for (int c = threadIdx.x * 8; c < N; c += 256 * 8) {
      uint4 raw[kCombBatch];
      int64_t r[kCombBatch];  // uniform, -1: no row
#pragma unroll
      for (int j = 0; j < kCombBatch; ++j) {
        r[j] = j0 + j < k ? row_of[t * k + j0 + j] : -1;
        if (r[j] >= R) r[j] = -1;
        raw[j] = r[j] >= 0 ? load8<true>(rows + r[j] * N + c) : uint4{0u, 0u, 0u, 0u};
      }
      float d[8];
      values8<BF16>(dy, t * N + c, d);
#pragma unroll
      for (int j = 0; j < kCombBatch; ++j) {
        if (r[j] < 0) continue;
        const float wj = w[t * k + j0 + j];
        float v[8], o[8];
        bf16x8(raw[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dot[j] = __builtin_fmaf(v[e], d[e], dot[j]);
          o[e] = wj * d[e];
        }
        store16<true>(drows + r[j] * N + c, pack8(o));
      }
    }
#pragma unroll
    for (int j = 0; j < kCombBatch; ++j) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) dot[j] += __shfl_xor(dot[j], o);
      if ((threadIdx.x & 63) == 0) part[j][threadIdx.x >> 6] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kCombBatch && j0 + (int)threadIdx.x < k) {
      const float* s = part[threadIdx.x];
      dw[t * k + j0 + threadIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
    }
    __syncthreads();  // before the next eight choices' sums
  }
}

}  // namespace

// A launch has at most 2^24 - 1 workgroups of 256 threads; longer calls run in chunks of tokens (units of at most 2^23 waves
// or workgroups).
constexpr int64_t kCombMaxGroups = (int64_t)1 << 23;

// Rows that do not stay in the 256 MB Infinity Cache with what else is in use: from 96 MB on, from 48 MB on where drows is
// written too. Streamed against not, forward: 33, 59, 88, 235 million values 13.2 / 12.7, 31 / 36, 39 / 46, 91 / 105 us;
// with the backward pass: 15, 29, 34, 59, 235 million 22.9 / 18.1, 35 / 37, 38 / 46, 81 / 93, 279 / 291 us.
static bool streams(int64_t T, int64_t k, int64_t N, int64_t R, int64_t mb) {
  return (T * k < R ? T * k : R) * N * 2 >= mb << 20;
}

hipError_t launch_combine(const uint16_t* rows, const int32_t* row_of, const float* w, void* y, bool bf16_y, int64_t T,
                          int64_t k, int64_t N, int64_t R, hipStream_t stream) {
  const int parts = (int)((N + 511) / 512);
  const int64_t chunk = kCombMaxGroups / parts;  // parts <= 2^21
  const bool nt = streams(T, k, N, R, 96);
  const auto kernel = bf16_y ? (nt ? combine_kernel<true, true> : combine_kernel<true, false>)
                             : (nt ? combine_kernel<false, true> : combine_kernel<false, false>);
  for (int64_t t = 0; t < T; t += chunk) {
    const int64_t n = T - t < chunk ? T - t : chunk;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((n * parts + 3) / 4)), dim3(256), 0, stream, rows, row_of + t * k, w + t * k,
                       static_cast<void*>(static_cast<uint8_t*>(y) + t * N * (bf16_y ? 2 : 4)), (int)k, (int)N, R, n, parts);
  }
  return hipGetLastError();
}

// A workgroup per token pays where a token's choices have values for all its threads.  84 MB of rows, a wave per choice
// against a workgroup per token, us (six sets of buffers in rotation, so nothing is cached from one call to the next):
//   k N = 2048: k = 1 54 / 66, k = 2 44 / 62, k = 4 42 / 63;  2560, k = 8: 49 / 57
//   k N = 4096: k = 1 55 / 53, k = 2 46 / 42, k = 4 40 / 40, k = 8 41 / 41
//   k N = 8192: k = 2 48 / 41, k = 4 43 / 38, k = 8 39 / 38
// Narrower rows: k = 8, N = 64: 165 / 241; k = 2, N = 64: 169 / 846, N = 16: 628 / 3359.  Rows that stayed in the cache (one
// set of buffers) are faster with a wave per choice, at k = 8, N = 2048: 84 MB 30 / 36, 130 MB 50 / 56.
constexpr int64_t kCombTokenValues = 4096;

hipError_t launch_combine_bwd(const void* dy, bool bf16_y, const uint16_t* rows, const int32_t* row_of, const float* w,
                              uint16_t* drows, float* dw, int64_t T, int64_t k, int64_t N, int64_t R,
                              hipStream_t stream) {
  const bool token = streams(T, k, N, R, 48) && k * N >= kCombTokenValues;
  const int64_t chunk = kCombMaxGroups / k;
  for (int64_t t = 0; t < T; t += chunk) {
    const int64_t n = T - t < chunk ? T - t : chunk;
    const void* from = static_cast<const uint8_t*>(dy) + t * N * (bf16_y ? 2 : 4);
    if (token) {
      const auto kernel = bf16_y ? combine_bwd_token_kernel<true> : combine_bwd_token_kernel<false>;
      hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(256), 0, stream, from, rows, row_of + t * k, w + t * k, drows, dw + t * k,
                         (int)k, (int)N, R);
    } else {
      const auto kernel = bf16_y ? combine_bwd_kernel<true> : combine_bwd_kernel<false>;
      hipLaunchKernelGGL(kernel, dim3((unsigned)((n * k + 3) / 4)), dim3(256), 0, stream, from, rows, row_of + t * k, w + t * k,
                         drows, dw + t * k, (int)k, (int)N, R, n);
    }
  }
  return hipGetLastError();
}

}  // namespace dg
