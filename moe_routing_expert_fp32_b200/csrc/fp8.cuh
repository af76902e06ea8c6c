// fp8.cuh -- the 8-bit block-scaled format shared by the kernels that write it:
// the scale of a block from its largest magnitude, and the rounding to e4m3.
#pragma once

#include <stdint.h>

namespace moe {
namespace fp8 {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f;

// Scale of a block whose largest magnitude is amax (possibly infinity or NaN),
// and *inv = fl32(1 / scale).  pow2: rounded up to a power of two, so that the
// magnitudes still fit below 448 and every product with inv is exact.
__device__ __forceinline__ float block_scale(float amax, int pow2, float& inv) {
  // a NaN fails the comparison and stays
  float s = __fdiv_rn(amax < kAmaxFloor ? kAmaxFloor : amax, kE4m3Max);
  if (pow2) {
    const uint32_t b = __float_as_uint(s);
    if (b < 0x7f800000u) s = __uint_as_float((b + 0x7fffffu) & 0x7f800000u);
  }
  inv = __fdiv_rn(1.0f, s);
  return s;
}

// Four values to e4m3, nearest even, saturating; a in the lowest byte.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

}  // namespace fp8
}  // namespace moe
