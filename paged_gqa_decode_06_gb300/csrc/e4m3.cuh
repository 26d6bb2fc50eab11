// The 8-bit cache format: e4m3 codes with one fp32 scale per (position, KV
// head) row; a value is code * scale.
//
// The quantiser takes the least power of two with max |x| <= 448 * scale, so
// that dividing by it is exact and the code is the value's nearest e4m3
// number (four significant bits) whatever the row's magnitude; a row below
// 2^-100 becomes zeros with scale 0.  Readers accept any scale.
#pragma once

#include <stdint.h>

namespace pgd {

struct RowScale {
  float scale, inv;  // 2^e and 2^-e, or 0 and 0
};

// From the row's largest magnitude: with amax = m * 2^E (1 <= m < 2) and 448 =
// 1.75 * 2^8, e = E - 8, one more when m > 1.75.
__device__ __forceinline__ RowScale e4m3_scale(float amax) {
  // Inf counts as the largest finite number, so it saturates and stays large
  const uint32_t bits = min(__float_as_uint(amax), 0x7f7fffffu);
  if (bits < ((127u - 100u) << 23)) return RowScale{0.f, 0.f};
  const uint32_t e = (bits >> 23) - 8u + ((bits & 0x7fffffu) > 0x600000u ? 1u : 0u);
  return RowScale{__uint_as_float(e << 23), __uint_as_float((254u - e) << 23)};
}

// Two values to two codes (low byte first), nearest even, Inf to +-448, NaN
// to NaN.
__device__ __forceinline__ uint32_t e4m3_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes to two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}

}  // namespace pgd
