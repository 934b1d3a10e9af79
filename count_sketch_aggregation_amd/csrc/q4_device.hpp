// q4_device.hpp -- device code shared by the 4-bit kernels: the scale of 32 elements and the
// rounding to 4 bits (internal to libs2r).
#pragma once

#include "q8_device.hpp"
#include "s2r_q4.h"

namespace s2r {

constexpr int kQ4Block = 32;                       // elements of a row under one scale
constexpr uint32_t kQ4MinScale = 17, kQ4MaxScale = 252, kQ4NanScale = 255;

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`: 6 is 1.5 * 2^2, so the
// least power of two s with amax <= 6 s is amax's own over 2^2, one more where amax's mantissa exceeds
// 1.5; adding 0x3fffff carries into the exponent exactly then.  Infinities and NaN are above all others.
__device__ inline uint32_t q4_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return kQ4NanScale;
  const int b = (int)((amax + 0x3fffffu) >> 23) - 2;
  return b < (int)kQ4MinScale ? kQ4MinScale : b > (int)kQ4MaxScale ? kQ4MaxScale : (uint32_t)b;
}

// Eight values to eight codes under scale byte b (0 under the NaN scale): the conversion divides by
// the scale, a power of two, rounds to nearest even, and keeps what is beyond 6 at 6.
__device__ inline uint32_t q4_encode8(const float* x, uint32_t b) {
  const float s = scale_value(b);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[0], x[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2], x[3], s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4], x[5], s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6], x[7], s, 3);
  return b == kQ4NanScale ? 0 : q;
}

// `left` codes of a word stay, the others become 0
__device__ inline uint32_t q4_keep(uint32_t q, int left) {
  return left <= 0 ? 0 : left < 8 ? q & ((1u << (4 * left)) - 1) : q;
}

}  // namespace s2r
