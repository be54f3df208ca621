// What the dense FP8 kernels do with 16 consecutive columns of a finished row
// before they store them: bias, activation, residual.
#pragma once

#include "activation.hpp"
#include "gemm_common.hpp"

namespace dg {

typedef unsigned int epi4 __attribute__((ext_vector_type(4)));

// 4 fp32 of the bias at columns c..c + 3 (zeros past the range: no bias, or no such column)
__device__ __forceinline__ f32x4 bias4(__amdgpu_buffer_rsrc_t r, uint32_t c) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, c * 4u, 0, 0));
}

// two bf16 of a residual and two sums
__device__ __forceinline__ uint32_t add_pack(uint32_t res, float a, float b) {
  return pack_bf16x2(a + __uint_as_float(res << 16), b + __uint_as_float(res & 0xffff0000u));
}

}  // namespace dg
