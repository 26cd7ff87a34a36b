// fp8_device.h -- what the FP8 kernels share: e4m3 codes under power-of-two scales.
#pragma once
#include "ffn_device.h"

namespace fp8 {
namespace {

using namespace ffn;

// The exponent field of a block's scale from the largest magnitude's bits: 448 is
// 1.75 * 2^8, so a mantissa up to 1.75 leaves 2^-8 of its power of two, a larger one
// 2^-7; at least the least normal, and 1 for a block of zeros. Infinities and NaN: 255.
__device__ __forceinline__ uint32_t scale_field(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  if (top == 0) return 127;
  const uint32_t e = (top + 0x1fffffu) >> 23;
  return e > 8 ? e - 8 : 1;
}
__device__ __forceinline__ float scale_value(uint32_t field) {
  return field == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, field << 23);
}
// 1 / scale (field 1 .. 247), exact; 0 for NaN, under which codes are 0
__device__ __forceinline__ float scale_inverse(uint32_t field) {
  return field == 255 ? 0.f : __builtin_bit_cast(float, (254 - field) << 23);
}

#if defined(__HIP_DEVICE_COMPILE__)
// Four values times `inverse` as e4m3. At most 448 in magnitude, so nothing saturates; a value
// that the multiplication rounds is below 2^-126, and its code 0 either way. An infinity or a
// NaN has inverse 0 and gives NaN codes: cleared by the caller.
__device__ __forceinline__ uint32_t pack4(const float* v, float inverse) {
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inverse, v[1] * inverse, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inverse, v[3] * inverse, c, true);
}
#endif

__device__ __forceinline__ uint32_t magnitude(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

}  // namespace
}  // namespace fp8
