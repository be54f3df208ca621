// Microscaled 4-bit quantiser and its inverse for gfx950.
//
// A row is cut into blocks of 32 elements.  A block's scale is 2^(c - 127),
// the smallest power of two with 6 * 2^(c - 127) >= amax (6 is the largest
// e2m1 magnitude; c is clamped to [0, 253], a block of zeros has c = 127), and
// its elements are e2m1_RNE(x * 2^(127 - c)): the multiplication is exact, so
// the code is the e2m1 value nearest to x / scale, ties to the even mantissa,
// the sign of zero kept.  A block that holds a NaN or an infinity has the NaN
// code c = 255 and elements 0, so whatever reads it gives NaN.
//
// Codes are packed two to a byte (the lower nibble first), the scale bytes of
// four consecutive blocks to an int32 word, words MN-major ([K/128][rows]).
//
// Both kernels are HBM-bound: a row is read once, a block's largest magnitude is a
// maximum over the 4 lanes (bf16 input, 8 values each) or 8 (fp32, 4 each)
// that hold it.

#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// c of a block with largest magnitude bits u (sign cleared): with amax = 1.f * 2^(E - 127)
// and 6 = 1.5 * 2^2 the least exponent is E - 129 where 1.f <= 1.5, else E - 128
__device__ __forceinline__ int mx_code(uint32_t u) {
  if (u >= 0x7f800000u) return 255;
  if (u == 0) return 127;
  const int c = (int)(u >> 23) - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0);
  return (u >> 23) == 0 || c < 0 ? 0 : c;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A 256-thread workgroup handles 4 PER rows x 512 columns of one group: each
// of its four waves PER rows, every load and store of the wide side a whole
// kilobyte (fp32 input: two, each lane 16 bytes of either), the rows of a wave
// in flight together.  Rows per wave by measurement, 8 x 4096 x 7168, before
// large arrays were streamed: fp32 input 1, 2, 4 rows 190, 204, 209 us; bf16
// input 113-122, 105, 106 us; reading back 146-158, 105, 106 us.
constexpr int kQCols = 512;

// first row and column of this workgroup
template <int ROWS>
__device__ __forceinline__ int64_t q_place(int K, int* col) {
  const int tiles = (K - 1) / kQCols + 1;  // K reaches the last multiple of 128 below 2^31
  const int64_t rb = (int64_t)blockIdx.x / tiles;
  *col = (int)((int64_t)blockIdx.x - rb * tiles) * kQCols;
  return rb * ROWS;
}

// maximum with the lane that DPP control C exchanges with
template <int C>
__device__ __forceinline__ uint32_t dpp_max(uint32_t u) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, C, 0xf, 0xf, true);
  return o > u ? o : u;
}

// row_token: row r takes row row_token[r] of x, rows whose entry is outside
// [0, T) are not written.  NT: x is streamed past the caches
template <bool BF16, int PER, bool NT>
__global__ void __launch_bounds__(256) quant_mxfp4_kernel(const void* __restrict__ x, uint8_t* __restrict__ q,
                                                          int32_t* __restrict__ sf, const int32_t* __restrict__ row_token,
                                                          int64_t T, int64_t R, int K) {
  // 16-byte pieces of a row per lane, their elements, and the lanes of a block
  constexpr int NP = BF16 ? 1 : 2;
  constexpr int NE = BF16 ? 8 : 4;
  constexpr int LPB = 32 / NE;
  constexpr int ROWS = 4 * PER;
  __shared__ uint32_t words[4][ROWS];
  __shared__ int live[ROWS];
  int col0;
  const int64_t r0 = q_place<ROWS>(K, &col0);
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t g = blockIdx.y;
  const int KB = K >> 7;
  bool active[PER];
  uint4 raw[PER][NP];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t r = r0 + wave * PER + i;
    bool row = r < R;
    int64_t src = g * R + r;
    if (row_token) {
      src = row ? row_token[g * R + r] : -1;
      row = src >= 0 && src < T;
    }
    active[i] = row;
    if (lane == 0) live[wave * PER + i] = row;
#pragma unroll
    for (int h = 0; h < NP; ++h) {
      const int col = col0 + h * 256 + lane * NE;
      raw[i][h] = uint4{0u, 0u, 0u, 0u};
      if (row && col < K) {
        const void* from = static_cast<const uint8_t*>(x) + (src * (int64_t)K + col) * (BF16 ? 2 : 4);
        if constexpr (NT) {
          const u32x4 v = __builtin_nontemporal_load(static_cast<const u32x4*>(from));
          raw[i][h] = uint4{v.x, v.y, v.z, v.w};
        } else {
          raw[i][h] = *static_cast<const uint4*>(from);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = wave * PER + i;
#pragma unroll
    for (int h = 0; h < NP; ++h) {
      const uint4 w = raw[i][h];
      float v[NE];
      if constexpr (BF16) {
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
        v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
      } else {
        v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
      }
      // magnitudes compare as integers, NaN above infinity above every number
      uint32_t u = 0;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const uint32_t a = __float_as_uint(v[e]) & 0x7fffffffu;
        u = a > u ? a : u;
      }
      u = dpp_max<0xB1>(u);                       // pairs of lanes
      u = dpp_max<0x4E>(u);                       // pairs of pairs
      if constexpr (LPB == 8) u = dpp_max<0x141>(u);  // the quads of eight
      const int c = mx_code(u);
      uint32_t out = 0;
      if (c != 255) {
        const float inv = __builtin_ldexpf(1.0f, 127 - c);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0] * inv, v[1] * inv, 1.0f, 0);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2] * inv, v[3] * inv, 1.0f, 1);
        if constexpr (BF16) {
          out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4] * inv, v[5] * inv, 1.0f, 2);
          out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6] * inv, v[7] * inv, 1.0f, 3);
        }
      }
      const int col = col0 + h * 256 + lane * NE;
      uint8_t* dst = q + (g * R + r0 + row) * (int64_t)(K >> 1) + (col >> 1);
      if constexpr (BF16) {
        if (active[i] && col < K) *reinterpret_cast<uint32_t*>(dst) = out;
      } else {  // the even lane stores its neighbour's four codes too
        out |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)out, 0xB1, 0xf, 0xf, true) << 16;
        if (active[i] && col < K && (lane & 1) == 0) *reinterpret_cast<uint32_t*>(dst) = out;
      }
      const int blk = (h * 256 + lane * NE) >> 5;  // of the row's 16
      if (lane % LPB == 0) reinterpret_cast<uint8_t*>(&words[blk >> 2][row])[blk & 3] = (uint8_t)c;
    }
  }
  __syncthreads();
  if (threadIdx.x < 4 * ROWS) {  // the rows' words of one 128 are contiguous
    const int row = threadIdx.x & (ROWS - 1);
    const int kb = (col0 >> 7) + threadIdx.x / ROWS;
    if (live[row] && kb < KB) sf[(g * KB + kb) * R + r0 + row] = (int32_t)words[threadIdx.x / ROWS][row];
  }
}

// NT: y is streamed past the caches
template <bool BF16, int PER, bool NT>
__global__ void __launch_bounds__(256) dequant_mxfp4_kernel(const uint8_t* __restrict__ q, const int32_t* __restrict__ sf,
                                                            void* __restrict__ y, int64_t R, int K) {
  int col;
  int64_t r0 = q_place<4 * PER>(K, &col);
  const int lane = threadIdx.x & 63;
  const int64_t g = blockIdx.y;
  r0 += (threadIdx.x >> 6) * PER;
  col += lane * 8;
  uint32_t code[PER], word[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool in = col < K && r0 + i < R;
    code[i] = in ? *reinterpret_cast<const uint32_t*>(q + (g * R + r0 + i) * (int64_t)(K >> 1) + (col >> 1)) : 0u;
    word[i] = in ? (uint32_t)sf[(g * (K >> 7) + (col >> 7)) * R + r0 + i] : 0u;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t w = code[i];
    const uint32_t c = (word[i] >> (8 * ((lane >> 2) & 3))) & 255u;
    const float s = c == 255 ? __uint_as_float(0x7fc00000u) : __builtin_ldexpf(1.0f, (int)c - 127);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // e2m1 magnitude m: m < 2 is m / 2 (subnormal), else 2^(m / 2 - 1) * (1 + (m % 2) / 2)
      const uint32_t n = (w >> (4 * e)) & 15u;
      const uint32_t m = n & 7u;
      const uint32_t a = m < 2 ? m * 0x3f000000u : (126u << 23) + (m << 22);
      v[e] = __uint_as_float(a | ((n & 8u) << 28)) * s;
    }
    if (col >= K || r0 + i >= R) continue;
    const int64_t off = (g * R + r0 + i) * (int64_t)K + col;
    const auto put = [&](void* to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      const u32x4 w{a, b, c, d};
      if constexpr (NT) __builtin_nontemporal_store(w, static_cast<u32x4*>(to));
      else *static_cast<u32x4*>(to) = w;
    };
    if constexpr (BF16) {
      put(static_cast<uint16_t*>(y) + off, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      float* d = static_cast<float*>(y) + off;
      put(d, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      put(d + 4, __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    }
  }
}

template <int PER>
dim3 q_grid(int64_t G, int64_t R, int64_t K) {
  return dim3((unsigned)((R + 4 * PER - 1) / (4 * PER) * ((K + kQCols - 1) / kQCols)), (unsigned)G);
}

// The wide side is streamed from 16 MB on (there and back, streamed against not: 8 x 4096 x 7168 fp32 269 / 310 us, 4096 x
// 7168 fp32 38 / 43, bf16 28 / 31, 2048 x 7168 bf16 15.8 / 16.6, 1024 x 4096 bf16 the same; 8192 rows gathered, back only,
// 46 / 63).
bool streams(int64_t G, int64_t R, int64_t K, bool bf16) { return G * R * K * (bf16 ? 2 : 4) >= (int64_t)16 << 20; }

}  // namespace

hipError_t launch_quant_mxfp4(const void* x, bool bf16, uint8_t* q, int32_t* sf, const int32_t* row_token, int64_t G,
                              int64_t T, int64_t R, int64_t K, hipStream_t stream) {
  const bool nt = !row_token && streams(G, R, K, bf16);  // gathered rows are read again
  const auto kernel = bf16 ? (nt ? quant_mxfp4_kernel<true, 2, true> : quant_mxfp4_kernel<true, 2, false>)
                           : (nt ? quant_mxfp4_kernel<false, 1, true> : quant_mxfp4_kernel<false, 1, false>);
  hipLaunchKernelGGL(kernel, bf16 ? q_grid<2>(G, R, K) : q_grid<1>(G, R, K), dim3(256), 0, stream, x, q, sf, row_token, T, R, (int)K);
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t* q, const int32_t* sf, void* y, bool bf16, int64_t G, int64_t R,
                                int64_t K, hipStream_t stream) {
  const bool nt = streams(G, R, K, bf16);
  const auto kernel = bf16 ? (nt ? dequant_mxfp4_kernel<true, 2, true> : dequant_mxfp4_kernel<true, 2, false>)
                           : (nt ? dequant_mxfp4_kernel<false, 2, true> : dequant_mxfp4_kernel<false, 2, false>);
  hipLaunchKernelGGL(kernel, q_grid<2>(G, R, K), dim3(256), 0, stream, q, sf, y, R, (int)K);
  return hipGetLastError();
}

}  // namespace dg
