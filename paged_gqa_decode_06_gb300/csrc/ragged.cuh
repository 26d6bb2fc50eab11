// Ragged rows: which sequence a row (or a tile of rows) belongs to, found on
// the device from the offsets, so that a call needs no list made on the host.
#pragma once

#include <stdint.h>

#include "device_common.cuh"

namespace pgd {

// Division by a number the host knows: n / d for n below 2^31, in a multiply
// and a shift (a division by a variable costs a CTA's start about 150 cycles).
struct FastDiv {
  uint32_t d, mul, shift;
  __host__ static FastDiv of(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.shift) < d) ++f.shift;  // d <= 2^shift
    // mul = ceil(2^(31 + shift) / d) < 2^32
    f.mul = (uint32_t)(((1ull << (31 + f.shift)) + d - 1) / d);
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * mul) >> 31) >> shift;
  }
};

// The largest b in [0, n) with f(b) <= x, or -1 when there is none; f does
// not decrease.  One whole warp searches 32 candidates at a time, so up to 32
// sequences cost one load and up to 1024 two.  Whatever f holds, the result
// is in range.
template <class F>
__device__ __forceinline__ int warp_search(int n, int64_t x, int lane, F f) {
  int lo = 0, hi = n;
  bool found = false;
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int64_t cand = (int64_t)lo + (int64_t)lane * step;
    const bool le = cand < hi && f((int)cand) <= x;
    const int count = __popc(__ballot_sync(0xffffffffu, le));
    if (count == 0) break;
    found = true;
    lo += (count - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
    if (hi - lo <= 1) break;
  }
  return found ? lo : -1;
}

// Offsets of sequence b's rows: [first, first + count) of `total` rows.  ok
// is false where the offsets do not ascend inside [0, total].
struct RowRange {
  int32_t first, count;
  bool ok;
};
__device__ __forceinline__ RowRange row_range(const int32_t* offsets, int b, int32_t total) {
  const int32_t a = ld_global_s32(offsets + b), z = ld_global_s32(offsets + b + 1);
  RowRange r{a, 0, a >= 0 && a <= z && z <= total};
  if (r.ok) r.count = z - a;
  return r;
}

}  // namespace pgd
