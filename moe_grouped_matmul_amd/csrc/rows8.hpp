// Device helpers of the kernels that hold 8 consecutive values of a row in a
// lane, so that 16 lanes hold a group of 128.
#pragma once

#include "gemm_common.hpp"

namespace dg {

typedef unsigned int raw4 __attribute__((ext_vector_type(4)));

// 8 consecutive values of a row as they lie in memory: four registers of bf16 pairs or eight floats
template <bool BF16>
struct Raw8 {
  raw4 v[BF16 ? 1 : 2];
};
// (NT: past the caches)
template <bool BF16, bool NT = false>
__device__ __forceinline__ Raw8<BF16> load8(const void* base, int64_t at) {
  Raw8<BF16> r;
  const raw4* p = reinterpret_cast<const raw4*>(static_cast<const uint8_t*>(base) + at * (BF16 ? 2 : 4));
  r.v[0] = NT ? __builtin_nontemporal_load(p) : p[0];
  if constexpr (!BF16) r.v[1] = NT ? __builtin_nontemporal_load(p + 1) : p[1];
  return r;
}
template <bool BF16, bool NT = false>
__device__ __forceinline__ void store8(void* base, int64_t at, const Raw8<BF16>& r) {
  raw4* p = reinterpret_cast<raw4*>(static_cast<uint8_t*>(base) + at * (BF16 ? 2 : 4));
  if constexpr (NT) __builtin_nontemporal_store(r.v[0], p);
  else p[0] = r.v[0];
  if constexpr (!BF16) {
    if constexpr (NT) __builtin_nontemporal_store(r.v[1], p + 1);
    else p[1] = r.v[1];
  }
}
template <bool BF16>
__device__ __forceinline__ void values(const Raw8<BF16>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f[2 * i] = __uint_as_float(r.v[0][i] << 16);
      f[2 * i + 1] = __uint_as_float(r.v[0][i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(r.v[0][i]);
      f[4 + i] = __uint_as_float(r.v[1][i]);
    }
  }
}
// 8 weights, whose type is the same for the whole launch
__device__ __forceinline__ void weights8(const void* base, bool bf16, int at, float* f) {
  if (bf16) values(load8<true>(base, at), f);
  else values(load8<false>(base, at), f);
}
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> rounded(const float* f) {
  Raw8<BF16> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      r.v[0][i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    } else {
      r.v[0][i] = __float_as_uint(f[i]);
      r.v[1][i] = __float_as_uint(f[4 + i]);
    }
  }
  return r;
}

__device__ __forceinline__ float wave_sum(float s) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

// Largest magnitude of the 128 values of 16 neighbouring lanes, in all of them: NaN is passed over, and is the result where there
// is nothing else (as in the quantisers).  A lane's maximum is taken with zero, so that its bits are ordered as it is and a
// rotation within the 16 is one instruction; a group of zeros and NaN is looked at again.
__device__ __forceinline__ float group_amax(const float* v) {
  const float a = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fabsf(v[2]));
  const float b = fmaxf(fmaxf(fabsf(v[3]), fabsf(v[4])), fabsf(v[5]));
  const float c = fmaxf(fmaxf(fabsf(v[6]), fabsf(v[7])), 0.f);
  uint32_t u = __float_as_uint(fmaxf(fmaxf(a, b), c));
#define DG_ROT(n) (uint32_t) __builtin_amdgcn_update_dpp(0, (int)u, 0x120 + (n), 0xf, 0xf, false)
#define DG_MAX(n)                   \
  do {                              \
    const uint32_t o_ = DG_ROT(n);  \
    u = o_ > u ? o_ : u;            \
  } while (0)
  DG_MAX(8);
  DG_MAX(4);
  DG_MAX(2);
  DG_MAX(1);
#undef DG_MAX
  if (u == 0) {  // all 16 lanes
    bool none = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) none &= v[e] != v[e];
    u = none ? 1u : 0u;
    u &= DG_ROT(8);
    u &= DG_ROT(4);
    u &= DG_ROT(2);
    u &= DG_ROT(1);
    if (u) u = 0x7fc00000u;
  }
#undef DG_ROT
  return __uint_as_float(u);
}

}  // namespace dg
