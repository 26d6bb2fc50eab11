// The 4-bit cache format: e2m1 codes, two to a byte (the even dim in the low
// nibble), an e4m3 scale for each block of 16 dims and one fp32 scale for each
// (position, KV head) row; a value is code * block * row.
//
// The quantiser takes for the row the least power of two with max |x| <=
// 6 * 448 * row, so that dividing by it is exact and every block's scale is
// the e4m3 number nearest to max |x| / (6 row) of its block; the code is the
// e2m1 number nearest to x / (block row).  (Against one scale for the row
// alone, a block of 16 costs half a bit a value and keeps a small value's bits
// beside a large one 16 dims away.)  Readers accept any scales.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "e4m3.cuh"
#include "elem.cuh"

namespace pgd {

// The row's scale from its largest finite magnitude: with amax = m * 2^E (1 <= m
// < 2) and 6 * 448 = 1.3125 * 2^11, e = E - 11, one more when m > 1.3125.  A
// row below 2^-100 becomes zeros with scale 0.
__device__ __forceinline__ RowScale e2m1_row_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  if (bits < ((127u - 100u) << 23)) return RowScale{0.f, 0.f};
  const uint32_t e = (bits >> 23) - 11u + ((bits & 0x7fffffu) > 0x280000u ? 1u : 0u);
  return RowScale{__uint_as_float(e << 23), __uint_as_float((254u - e) << 23)};
}

// A block's scale: its e4m3 code, and the reciprocal of its value times the row's in
// two parts (0 for a block of zeros and one that is no number, whose codes are 0).
struct BlockScale {
  float inv, rest;
  uint32_t code;
};
__device__ __forceinline__ BlockScale e2m1_block_scale(float amax, RowScale row, bool finite) {
  BlockScale b;
  // (a sixth rounded is enough: 16-bit magnitudes stay 2^-12 from where two codes
  // meet, but for those half way between, five bits times 6, whose product is exact)
  b.code = finite ? e4m3_pack2(amax * row.inv * (1.f / 6.f), 0.f) & 0xffu : 0x7fu;
  const float v = finite ? ElemOps<__half>::unpack2(e4m3_to_half2(b.code)).x : 0.f;
  const float inv = v > 0.f ? __frcp_rn(v) : 0.f;
  b.inv = inv * row.inv;  // (powers of two: exact)
  b.rest = v > 0.f ? fmaf(-inv, v, 1.f) * inv * row.inv : 0.f;
  return b;
}

// x over the block's and the row's scales, rounded once: the reciprocal's parts hold
// 2^-47 of it.  So a value half way between two codes is seen as that; the others
// stay 2^-12 away.
__device__ __forceinline__ float block_div(float x, const BlockScale& b) {
  return fmaf(x, b.inv, fmaf(x, b.rest, 0.f));  // (a zero loses its sign)
}

// Eight values to eight codes, the first in the lowest nibble: nearest even,
// saturating at +-6.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Two values to 16 bits, what is beyond the type's range as its largest number (a NaN
// stays).
template <class E>
__device__ __forceinline__ uint32_t pack2_sat(float lo, float hi) {
  uint32_t r;
  if constexpr (std::is_same<E, __half>::value)
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight codes to four pairs of fp16 values (exact): byte i of the word to r[i],
// its low nibble to the low half.
__device__ __forceinline__ void e2m1_to_half8(uint32_t codes, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(codes));
}

}  // namespace pgd
