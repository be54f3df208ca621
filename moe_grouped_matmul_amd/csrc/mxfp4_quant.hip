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
// Both kernels are HBM-bound.

#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

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

// Grid (ceil(R / 16) * (K / 128), G); a 256-thread workgroup quantises 128
// columns of 16 consecutive rows: 16 lanes per row, 8 elements per lane, four
// lanes per block, so the 16 rows' scale words are 64 contiguous bytes.
// row_token: row r takes row row_token[r] of x, rows whose entry is outside
// [0, T) are not written.
template <bool BF16>
__global__ void __launch_bounds__(256) quant_mxfp4_kernel(const void* __restrict__ x, uint8_t* __restrict__ q,
                                                          int32_t* __restrict__ sf, const int32_t* __restrict__ row_token,
                                                          int64_t T, int64_t R, int K) {
  const int KB = K >> 7;
  const int64_t rb = (int64_t)blockIdx.x / KB;
  const int kb = (int)((int64_t)blockIdx.x - rb * KB);
  const int sub = threadIdx.x & 15;
  const int64_t r = rb * 16 + (threadIdx.x >> 4);
  const int64_t g = blockIdx.y;
  bool active = r < R;
  int64_t src = g * R + r;
  if (row_token) {
    src = active ? row_token[g * R + r] : -1;
    active = src >= 0 && src < T;
  }
  if (!active) src = 0;
  const int64_t off = src * (int64_t)K + ((int64_t)kb << 7) + (sub << 3);
  float v[8];
  if (active) {
    if constexpr (BF16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + off);
      v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
      v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    } else {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + off);
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + off + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  // magnitudes compare as integers, NaN above infinity above every number
  uint32_t u = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
    u = a > u ? a : u;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const uint32_t a = __shfl_xor(u, o);
    u = a > u ? a : u;
  }
  const int c = mx_code(u);
  const float inv = c == 255 ? 0.f : __builtin_ldexpf(1.0f, 127 - c);
  uint32_t out = 0;
  if (c != 255) {
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0] * inv, v[1] * inv, 1.0f, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2] * inv, v[3] * inv, 1.0f, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4] * inv, v[5] * inv, 1.0f, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6] * inv, v[7] * inv, 1.0f, 3);
  }
  // the four blocks' codes (lanes 0, 4, 8, 12 of the row) into one word
  uint32_t word = (uint32_t)c << (8 * (sub >> 2));
  word |= __shfl_xor(word, 4);
  word |= __shfl_xor(word, 8);
  if (!active) return;
  *reinterpret_cast<uint32_t*>(q + (g * R + r) * (int64_t)(K >> 1) + ((int64_t)kb << 6) + (sub << 2)) = out;
  if (sub == 0) sf[(g * KB + kb) * R + r] = (int32_t)word;
}

// the same grid; a lane reads 8 codes and its block's scale byte
template <bool BF16>
__global__ void __launch_bounds__(256) dequant_mxfp4_kernel(const uint8_t* __restrict__ q, const int32_t* __restrict__ sf,
                                                            void* __restrict__ y, int64_t R, int K) {
  const int KB = K >> 7;
  const int64_t rb = (int64_t)blockIdx.x / KB;
  const int kb = (int)((int64_t)blockIdx.x - rb * KB);
  const int sub = threadIdx.x & 15;
  const int64_t r = rb * 16 + (threadIdx.x >> 4);
  const int64_t g = blockIdx.y;
  if (r >= R) return;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(q + (g * R + r) * (int64_t)(K >> 1) + ((int64_t)kb << 6) + (sub << 2));
  const uint32_t c = ((uint32_t)sf[(g * KB + kb) * R + r] >> (8 * (sub >> 2))) & 255u;
  const float s = c == 255 ? __uint_as_float(0x7fc00000u) : __builtin_ldexpf(1.0f, (int)c - 127);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // e2m1 magnitude m: m < 2 is m / 2 (subnormal), else 2^(m / 2 - 1) * (1 + (m % 2) / 2)
    const uint32_t n = (w >> (4 * i)) & 15u;
    const uint32_t m = n & 7u;
    const float a = m < 2 ? 0.5f * (float)m : __uint_as_float((126u << 23) + (m << 22));
    v[i] = (n & 8u ? -a : a) * s;
  }
  const int64_t off = (g * R + r) * (int64_t)K + ((int64_t)kb << 7) + (sub << 3);
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + off) =
        uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else {
    float* d = static_cast<float*>(y) + off;
    *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace

hipError_t launch_quant_mxfp4(const void* x, bool bf16, uint8_t* q, int32_t* sf, const int32_t* row_token, int64_t G,
                              int64_t T, int64_t R, int64_t K, hipStream_t stream) {
  const dim3 grid((unsigned)((R + 15) / 16 * (K / 128)), (unsigned)G);
  if (bf16)
    hipLaunchKernelGGL(quant_mxfp4_kernel<true>, grid, dim3(256), 0, stream, x, q, sf, row_token, T, R, (int)K);
  else
    hipLaunchKernelGGL(quant_mxfp4_kernel<false>, grid, dim3(256), 0, stream, x, q, sf, row_token, T, R, (int)K);
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t* q, const int32_t* sf, void* y, bool bf16, int64_t G, int64_t R,
                                int64_t K, hipStream_t stream) {
  const dim3 grid((unsigned)((R + 15) / 16 * (K / 128)), (unsigned)G);
  if (bf16)
    hipLaunchKernelGGL(dequant_mxfp4_kernel<true>, grid, dim3(256), 0, stream, q, sf, y, R, (int)K);
  else
    hipLaunchKernelGGL(dequant_mxfp4_kernel<false>, grid, dim3(256), 0, stream, q, sf, y, R, (int)K);
  return hipGetLastError();
}

}  // namespace dg
