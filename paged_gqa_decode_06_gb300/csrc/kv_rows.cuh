// Rows of a ragged batch in the paged cache: where each of them sits, shared
// by the kernels that write and read such rows.
#pragma once

#include <type_traits>

#include "combine.cuh"  // grid_dependency_wait
#include "ragged.cuh"

namespace pgd {

struct RowMap {
  const int32_t* page_table;
  const int32_t* offsets;   // [B + 1]
  const int32_t* base;      // append: seq_lens [B]; read: first positions [B] or null (0)
  int32_t* err;
  int32_t total, B, page_size, max_pages, num_pages;
};

// Where a row of the chunk, found in sequence b, sits in the cache: (page, slot),
// page -1 when it has no place there; *pos is its position, -1 where it has none
// inside the table.  report: raises what is wrong.
template <bool kAppend>
__device__ __forceinline__ int2 place_in(const RowMap& a, int b, int row, bool report, bool* owned,
                                         int* pos_out) {
  *owned = false;
  *pos_out = -1;
  if (b < 0) return make_int2(-1, 0);
  const RowRange r = row_range(a.offsets, b, a.total);
  // (with offsets that do not ascend the search may end past the row)
  if (!r.ok || row < r.first || row >= r.first + r.count) return make_int2(-1, 0);
  *owned = true;
  const int64_t base = a.base ? a.base[b] : 0;
  const int64_t pos = base + (row - r.first) - (kAppend ? r.count : 0);
  const int64_t capacity = (int64_t)a.max_pages * a.page_size;
  if (pos < 0 || pos >= capacity || (kAppend && base > capacity)) {
    // an append before position 0 is no row; all else is out of the table
    if (report && (pos >= 0 || !kAppend || base < 0))
      raise_error(a.err, DECODE_ATTN_DEV_BAD_LEN);
    return make_int2(-1, 0);
  }
  *pos_out = (int)pos;
  const size_t pi = (size_t)b * a.max_pages + (size_t)(pos / a.page_size);
  const int page = PGD_IN(pi, (size_t)a.B * a.max_pages, a.err) ? a.page_table[pi] : -1;
  if (page < 0 || page >= a.num_pages) {
    if (report) raise_error(a.err, DECODE_ATTN_DEV_BAD_PAGE);
    return make_int2(-1, 0);
  }
  return make_int2(page, (int)(pos % a.page_size));
}

// The same for a row that one whole warp looks for.
template <bool kAppend>
__device__ __forceinline__ int2 place_row(const RowMap& a, int row, int lane, bool* owned,
                                          int* pos_out) {
  const int b = warp_search(a.B, row, lane, [&](int i) { return (int64_t)a.offsets[i]; });
  return place_in<kAppend>(a, b, row, lane == 0, owned, pos_out);
}

// The same for a row that a thread looks for by itself (the rows of a block side by
// side in one warp).
template <bool kAppend>
__device__ __forceinline__ int2 place_row_alone(const RowMap& a, int row, bool* owned,
                                                int* pos_out) {
  int lo = -1, hi = a.B;  // the largest b with offsets[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ld_global_s32(a.offsets + mid) <= row)
      lo = mid;
    else
      hi = mid;
  }
  return place_in<kAppend>(a, lo, row, true, owned, pos_out);
}

// Offsets that do not ascend inside [0, total], checked once per call.
__device__ __forceinline__ void check_offsets(const RowMap& a, int threads) {
  if (blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < a.B; b += threads)
    if (!row_range(a.offsets, b, a.total).ok) raise_error(a.err, DECODE_ATTN_DEV_BAD_LEN);
}

// Of two pairs of 16-bit values the larger magnitudes, with any sign; a NaN
// only where both are.
template <class E>
__device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same<E, __nv_bfloat16>::value)
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace pgd
