// Scales and conversions of the block-scaled FP8 quantiser, for the kernels that
// write its forms.
#pragma once

#include "device_util.h"

namespace muonh {

// The scale byte e + 127 of a block from its largest finite magnitude's bits:
// with amax = (1 + f) 2^(E - 127) and 448 = 1.75 * 2^8, e = E - 135, one more
// where 1 + f > 1.75.  Subnormal amax (E = 0) ends at the least byte.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int b = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u);
  return amax == 0 ? 127u : (uint32_t)max(b, 0);
}

// v * 2^-e as E4M3 where v may be Inf or NaN, which become NaN.
__device__ __forceinline__ float scaled(float v, uint32_t byte) {
  const bool finite = (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u;
  // 2^-e; the byte is at most 247, so it is a normal number
  return finite ? v * __uint_as_float((254u - byte) << 23) : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

typedef int16_t i16x2_t __attribute__((ext_vector_type(2)));

// Four finite values divided by the scale's power of two and rounded to E4M3,
// lowest byte first: two conversions that take the scale's exponent field.
__device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d, float scale) {
  i16x2_t r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t quantize4(uint32_t ab, uint32_t cd, float scale) {
  i16x2_t r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, ab), scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, cd), scale, true);
  return __builtin_bit_cast(uint32_t, r);
}
// The largest value of each row of 16 lanes, in all of them (rotations).
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
  return v;
}

}  // namespace muonh
