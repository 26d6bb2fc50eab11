// Rotary positions: a pair (x1, x2) of a head's first `rot` dims at position p
// becomes (x1 c - x2 s, x2 c + x1 s) with c = cos(p f), s = sin(p f) of the
// pair's frequency, read from a table of fp32 rows [rot / 2 cosines, rot / 2
// sines], one per position.  Pair i is the dims (i, i + rot / 2), or (2 i,
// 2 i + 1) interleaved; the dims from `rot` on stay.
//
// A thread turns units of 16 values: two items of 8 that hold the table's
// pairs 8 u .. 8 u + 7, both members of each.  So nothing is exchanged
// between threads, and rows may be turned where they lie.
#pragma once

#include "elem.cuh"

namespace pgd {

struct RopeArgs {
  const float* table;  // [rows][rot]
  int32_t rows;        // positions that have a row
  int32_t rot;         // rotated dims, a multiple of 16; 0: none
  int32_t interleaved;
  int32_t backward;    // 1: by the negative angle (the gradient)
};

// The unit's two items of 8 values, as item indices of the head.
__device__ __forceinline__ int2 rope_items(const RopeArgs& r, int unit) {
  if (!r.interleaved && 16 * unit < r.rot) return make_int2(unit, unit + r.rot / 16);
  return make_int2(2 * unit, 2 * unit + 1);
}

// Cosines and sines of a unit's eight pairs (unit < rot / 16).
struct RopePairs {
  float c[8], s[8];
};
__device__ __forceinline__ void rope_load(RopePairs& p, const RopeArgs& r, int pos, int unit) {
  const float4* c = reinterpret_cast<const float4*>(r.table + (size_t)pos * r.rot + 8 * unit);
  const float4* s = reinterpret_cast<const float4*>(r.table + (size_t)pos * r.rot + r.rot / 2 +
                                                    8 * unit);
  // (not the read-only path: what wrote the table may still run when this kernel starts)
  const float4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
  // (the sign as bits: a negation of each sine)
  const uint32_t flip = r.backward ? 0x80000000u : 0u;
  auto turn = [&](float x) { return __uint_as_float(__float_as_uint(x) ^ flip); };
  p.c[0] = c0.x, p.c[1] = c0.y, p.c[2] = c0.z, p.c[3] = c0.w;
  p.c[4] = c1.x, p.c[5] = c1.y, p.c[6] = c1.z, p.c[7] = c1.w;
  p.s[0] = turn(s0.x), p.s[1] = turn(s0.y), p.s[2] = turn(s0.z), p.s[3] = turn(s0.w);
  p.s[4] = turn(s1.x), p.s[5] = turn(s1.y), p.s[6] = turn(s1.z), p.s[7] = turn(s1.w);
}

// One pair, each product and the sum rounded by itself (as a composition of
// elementary operations gives it).
__device__ __forceinline__ float2 rope_pair(float x1, float x2, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s)),
                     __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s)));
}

// Turns a unit's items a and b, rounding each value once.
template <class E>
__device__ __forceinline__ void rope_unit(uint4& a, uint4& b, const RopePairs& p,
                                          bool interleaved) {
  using O = ElemOps<E>;
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = O::unpack2(x[i]);
      const float2 y = rope_pair(v.x, v.y, p.c[i], p.s[i]);
      x[i] = O::pack2(y.x, y.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = O::unpack2(x[i]), w = O::unpack2(x[4 + i]);
      const float2 y = rope_pair(v.x, w.x, p.c[2 * i], p.s[2 * i]);
      const float2 z = rope_pair(v.y, w.y, p.c[2 * i + 1], p.s[2 * i + 1]);
      x[i] = O::pack2(y.x, z.x);
      x[4 + i] = O::pack2(y.y, z.y);
    }
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(x[4], x[5], x[6], x[7]);
}

}  // namespace pgd
