// Codes of 4 exponent and 3 mantissa bits and the scale byte of their block
// (include/xp_model.h): how a block's scale follows from its largest
// magnitude, and codes from values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace xp {

// The scale byte of a block whose largest magnitude has the bits `top`:
// 448 = 1.75 * 2^8, so E is top's exponent less 8, and one more where its
// mantissa is above 1.75 (0x600000, which the sum carries into the exponent).
// Infinities and NaN have the largest bits of all.
__device__ __forceinline__ unsigned scale_of(unsigned top) {
  const int e = (int)((top + 0x1fffffu) >> 23) - 8;
  return top >= 0x7f800000u ? 255u : (unsigned)max(e, 0);
}
// 2^(127 - E), for which E is 247 at most; a value times it is exact, or far
// below the least code.  NaN for 255, which makes every code NaN.
__device__ __forceinline__ float inverse_of(unsigned e) { return __uint_as_float(e == 255u ? 0x7fffffffu : (254u - e) << 23); }
// 2^(E - 127): E = 0 is a subnormal number.
__device__ __forceinline__ float power_of(unsigned e) { return __uint_as_float(e == 255u ? 0x7fffffffu : e == 0u ? 0x00400000u : e << 23); }

__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Four values' codes, the first in the lowest byte.  Rounded to nearest even;
// a block's scale keeps them within 448, so none saturates but by rounding.
// (A NaN's code is 0x7f, whatever its sign.)
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d, float inverse) {
  unsigned short lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inverse), "f"(a * inverse));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inverse), "f"(c * inverse));
  return (unsigned)hi << 16 | lo;
}
// Two codes' values before the scale: exact in fp16.
__device__ __forceinline__ float2 values2(unsigned short codes) {
  unsigned h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace xp
