// Device helpers of the block-scaled e4m3 quantisers: scales, codes and the
// correctly rounded quotients, shared by every kernel that writes e4m3 with a
// scale per group (quant.hip states the rules).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

constexpr float kE4M3Max = 448.0f;

// four fp32 values -> four e4m3 bytes (a in byte 0): clamp to +-448, then the
// hardware's round-to-nearest-even conversion, two values per instruction
__device__ __forceinline__ float clamp448(float v) { return fminf(fmaxf(v, -kE4M3Max), kE4M3Max); }
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(a), clamp448(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(c), clamp448(d), lo, true);
}

__device__ __forceinline__ float scale_from_amax(float amax) {
  const float s = amax / kE4M3Max;  // IEEE-correct division (no fast-math)
  return s == 0.0f ? 1.0f : s;
}

// UE8M0 code of a group: c = 127 + min{e : 448 * 2^e >= amax}, clamped to
// [0, 254]; an all-zero group gets 127.  With amax = 1.f * 2^(E - 127) and
// 448 = 1.75 * 2^8 the minimum is E - 135 when 1.f <= 1.75 (mantissa field
// <= 0x600000) and E - 134 above; subnormal and tiny amax clamp to 0.
__device__ __forceinline__ int ue8m0_code(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 127;
  const int c = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (u >> 23) == 0 ? 0 : (c < 0 ? 0 : (c > 254 ? 254 : c));
}

// x * 2^(127 - c): an exact power-of-two scaling (one rounding only when the
// product is an fp32 subnormal, far below the e4m3 grid)
__device__ __forceinline__ uint32_t pack4_pow2(float a, float b, float c, float d, float inv) {
  return e4m3x4(a * inv, b * inv, c * inv, d * inv);
}

// stores code c of K block kb into its packed word (byte kb % 4); the last
// block of a row also zeroes the word's unused bytes
__device__ __forceinline__ void store_code(uint8_t* word, int kb, int KB, int c) {
  word[kb & 3] = (uint8_t)c;
  if (kb == KB - 1)
    for (int j = (kb & 3) + 1; j < 4; ++j) word[j] = 0;
}

// fl32(x / s) for e4m3 rounding, given r = fl32(1 / s) (IEEE division).  The
// product y = fl32(x * r) carries two roundings of relative size 2^-24 each,
// so it lies within a few fp32 steps of the correctly rounded quotient
// fl32(x / s).  Rounding to the normal e4m3 grid keeps the top 3 mantissa
// bits (the low 20 are dropped): both values give the same byte unless a
// rounding midpoint of the grid (low 20 bits 0x80000) lies within kGuard
// steps of y.  Those rare elements, and everything outside the normal range
// (e4m3 subnormals, non-finite values), take the IEEE division instead.
constexpr uint32_t kGuard = 16;
__device__ __forceinline__ bool product_safe(float y) {
  const uint32_t a = __float_as_uint(y) & 0x7fffffffu;
  const uint32_t low = a & 0xfffffu;
  return a >= 0x3c800000u + kGuard && a < 0x7f000000u && (low + kGuard - 0x80000u) > 2u * kGuard;
}

// q[0..N) = bytes of fl32(x[e] / s): the products, with the division redone
// (rarely) for the elements whose product is not safe
template <int N>
__device__ __forceinline__ void quotients(const float* x, float* y, float s, float r) {
  bool all_safe = true;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    y[e] = x[e] * r;
    all_safe &= product_safe(y[e]);
  }
  if (!all_safe) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!product_safe(y[e])) y[e] = x[e] / s;
  }
}

// The same scale and quotients for kernels whose arithmetic is what bounds them
// (a norm's rows, a gradient): fewer instructions, longer code.  16384 x 7168 rows
// of the norm 162 -> 154 us; in the quantisers alone, short and bound by memory,
// 64 x 7168 takes 3.3 us with them and 3.0 with those above.
//
// fl32(amax / 448), 1 where that is zero.  The product with fl32(1 / 448) and one
// correction by the remainder (exact in an FMA) is the correctly rounded
// quotient where nothing underflows (compared over all mantissas at both ends
// of the range); outside, the IEEE division.
__device__ __forceinline__ float scale_of(float amax) {
  if (amax >= 0x1p-60f && amax < 0x1p+120f) {
    constexpr float r = 1.0f / kE4M3Max;
    const float s = amax * r;
    return __builtin_fmaf(__builtin_fmaf(-kE4M3Max, s, amax), r, s);
  }
  return scale_from_amax(amax);
}

// q[0..N) = bytes of fl32(x[e] / s), |x[e]| <= 448 s up to rounding.  The
// hardware's reciprocal (1 ulp) leaves the products within the guard; the nearest
// to a midpoint and the least of all N that is not zero tell whether one of them
// may not be safe (a reciprocal in the normal range bounds the largest), and then
// those that are not are divided.  A product of zero is the byte of a zero.
// (Zeros are common: a bf16 sum of two like values, the slope of a relu.)
template <int N>
__device__ __forceinline__ void quotients_of(const float* x, float* y, float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  uint32_t near = 0xffffffffu, least = 0xffffffffu;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    y[e] = x[e] * r;
    const uint32_t d = (__float_as_uint(y[e]) + (kGuard - 0x80000u)) & 0xfffffu;  // up to 2 kGuard about a midpoint
    near = d < near ? d : near;
    const uint32_t m = (__float_as_uint(y[e]) << 1) - 1u;  // by magnitude, zero above all
    least = m < least ? m : least;
  }
  const bool normal = __float_as_uint(r) - 0x00800000u < 0x7e000000u;
  if (!(normal && near > 2u * kGuard && least >= ((0x3c800000u + kGuard) << 1) - 1u)) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!normal || !(product_safe(y[e]) || y[e] == 0.f)) y[e] = x[e] / s;
  }
}

}  // namespace dg
