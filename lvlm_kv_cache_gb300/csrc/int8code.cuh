// The int8 code of a value: clip(round(x / s)), x / s in correctly rounded
// fp32, half away from zero.
#pragma once

#include <stdint.h>

namespace aircache {

// The larger and the smaller value, or NaN where one of them is (fmaxf and fminf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// clip(round(x / s)) with x / s correctly rounded, s > 0, |x| <= 127 s.
// The quotient is first taken as t = x * (1/s) (both correctly rounded:
// within 1.6e-5 of the exact quotient, and the correctly rounded quotient is
// within 3.9e-6 of that).  Away from half-integers both round to the same
// integer, and round-to-nearest-even (rint) equals round-half-away there; within
// 4e-5 of a half-integer the correctly rounded division and roundf decide.
// |t| < 127.5 there, so no clip is needed.  A subnormal s can overflow 1/s and
// is itself a coarse rounding of max / 127: those quotients (t infinite or NaN,
// which fails the comparison below) are divided and clipped.  What has no quotient
// (a NaN, or an infinity under the infinite scale that it makes) has the code 0,
// which under that scale stands for NaN: clipped, it would be minus the largest value.
__device__ __forceinline__ int code(float x, float s, float rs) {
  const float t = x * rs;
  const float rt = rintf(t);
  if (!(fabsf(t - rt) <= 0.5f - 4e-5f)) {
    return __float2int_rz(min_nan(max_nan(roundf(__fdiv_rn(x, s)), -127.f), 127.f));  // (of NaN: 0)
  }
  return (int)rt;
}

// four codes -> one word, byte i = code i
__device__ __forceinline__ uint32_t pack4(int c0, int c1, int c2, int c3) {
  return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
}

}  // namespace aircache
