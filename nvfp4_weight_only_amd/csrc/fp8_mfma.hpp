// A block of 128 of K of the E4M3 x E4M3 products: one 16x16x128 matrix
// instruction (C = 0), and the two FP32 scales of its sum.
//
// The product of two scales need not be an FP32 number where the block's sum times
// both is one.  Each scale is therefore taken apart into a power of two, which the
// matrix instruction applies (its E8M0 scale operands), and a rest in [1, 2): the
// rests' product multiplies the instruction's result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace nvfp4 {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t mfma_frag(const uint4& a, const uint4& b) {
  return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// The scale's power of two as E8M0: its exponent field, 254 for an infinity or NaN
// (which the rest keeps; 255 would be a NaN).
__device__ __forceinline__ int scale_exp(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 0xFFu);
  return e < 254 ? e : 254;
}
// What is left of it: s / 2^(e - 127), exact.
__device__ __forceinline__ float scale_rest(float s, int e) { return __builtin_amdgcn_ldexpf(s, 127 - e); }

__device__ __forceinline__ bool is_normal(float f) { return __builtin_amdgcn_classf(f, 0x108); }
// Whether the product of two scales, both finite and not 0, is no normal FP32 number.
__device__ __forceinline__ bool is_far(float s, float w) {
  return !is_normal(s * w) && __builtin_amdgcn_classf(s, 0x198) && __builtin_amdgcn_classf(w, 0x198);
}

// 16 x 16 sums over 128 of K.
__device__ __forceinline__ f32x4_t mfma128(const i32x8_t& a, const i32x8_t& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
// 16 x 16 sums times 2^(ea - 127 + eb - 127), ea the lane's row of A, eb
// its row of B.
__device__ __forceinline__ f32x4_t mfma128(const i32x8_t& a, const i32x8_t& b, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, ea, 0, eb);
}

}  // namespace nvfp4
