// Activations of the products' epilogue and their derivatives, in fp32.
#pragma once

#include <hip/hip_runtime.h>

namespace dg {

enum Activation { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// 1 / (1 + e^-z): the hardware's 2^x and reciprocal, 1 ulp each
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

// z Phi(z) = max(z, 0) - a Phi(-a), a = |z|.  Phi(-a) = e^(-a^2 / 2) T(1 / (1 + c a)): what is left of the tail beside
// its exponential is smooth in that argument, and a polynomial of degree 6 without a constant was fitted here to it over [0, 13.4]
// with weights that bound both what is off relative to 1 (1.3e-7 with the fp32 roundings) and relative to the result, which
// falls below 2^-126 in that range (5.5e-5 of it, where bf16 rounds by up to 3.9e-3; 1e-6 above -2).  (A polynomial of
// log2 Phi(-a) alone needs degree 11 for 1.9e-3 of the result; one of degree 8 that bounds what is off of 1 alone, 43% wrong at
// -7, took 1.2 us less at the end of 4096 x 4096 x 7168: 121.5 and 122.7 us.)
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 16.f);  // e^(-a^2 / 2) is zero in fp32 there, and infinities stay out of the products
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.295893878f, a, 1.f));
  const float e = __builtin_amdgcn_exp2f(-0.5f * 1.44269504f * a * a);
  float p = __builtin_fmaf(-0.0838792995f, t, 0.248623431f);
  p = __builtin_fmaf(p, t, -0.0515091605f);
  p = __builtin_fmaf(p, t, 0.159625828f);
  p = __builtin_fmaf(p, t, 0.108404532f);
  p = __builtin_fmaf(p, t, 0.118734419f);
  return __builtin_fmaf(-(a * t * p), e, z < 0.f ? 0.f : z);  // NaN stays
}

// Phi(z) of the normal distribution and e^(-z^2 / 2), which its slope needs both.  The complementary error
// function is formula 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical
// Functions (after Hastings), off by at most 1.5e-7: half of that here, where a
// bf16 result near 1 is rounded by up to 2e-3.
__device__ __forceinline__ float normal_cdf(float z, float* density) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.f));
  const float e = __builtin_amdgcn_exp2f(-0.5f * 1.44269504f * z * z);
  float p = __builtin_fmaf(1.061405429f, t, -1.453152027f);
  p = __builtin_fmaf(p, t, 1.421413741f);
  p = __builtin_fmaf(p, t, -0.284496736f);
  p = __builtin_fmaf(p, t, 0.254829592f);
  const float tail = 0.5f * p * t * e;
  *density = e;
  return z < 0.f ? tail : 1.f - tail;
}

constexpr float kGeluTanh = 2.f * 0.79788456f;  // 2 sqrt(2 / pi): (1 + tanh u) / 2 = sigmoid(2 u)

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;  // NaN stays
  if constexpr (ACT == kActSilu) return z * sigmoid(z);
  if constexpr (ACT == kActGelu) return gelu(z);
  if constexpr (ACT == kActGeluTanh) return z * sigmoid(kGeluTanh * __builtin_fmaf(0.044715f * z * z, z, z));
  return z;
}

template <int ACT>
__device__ __forceinline__ float activate_slope(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : z != z ? z : 0.f;
  if constexpr (ACT == kActSilu) {
    const float p = sigmoid(z);
    return p * __builtin_fmaf(z, 1.f - p, 1.f);
  }
  if constexpr (ACT == kActGelu) {
    float e;
    const float p = normal_cdf(z, &e);
    return __builtin_fmaf(z * e, 0.39894228f, p);
  }
  if constexpr (ACT == kActGeluTanh) {
    // the slope is 0 or 1 to fp32 past |z| = 12, where z^2 may leave its range
    const float c = z > 16.f ? 16.f : z < -16.f ? -16.f : z;
    const float s = c * c;
    const float p = sigmoid(kGeluTanh * __builtin_fmaf(0.044715f * s, c, c));
    return __builtin_fmaf(c * p * (1.f - p) * kGeluTanh, __builtin_fmaf(3.f * 0.044715f, s, 1.f), p);
  }
  return 1.f;
}

}  // namespace dg
