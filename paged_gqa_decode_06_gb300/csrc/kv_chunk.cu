// Rows in and out of the paged cache by the chunk: decode_kv_append_chunk
// scatters a ragged batch's new K/V rows into their pages, as they are or
// quantised (e4m3.cuh), and decode_kv_read gathers rows back to contiguous
// 16-bit rows.
//
// Both move memory: each value is read once and written once.  A block takes
// a few consecutive rows with all their heads; one warp per row finds the
// row's sequence and page while every thread's first values are already on
// their way.  A thread handles 8 values of a row's head, so the D / 8 threads
// of a head are neighbours in a warp and the row's maximum is a few shuffles.
#include <algorithm>

#include "chunk_launch.h"
#include "e4m3.cuh"
#include "host_common.h"

namespace pgd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;  // rows of a block, one warp each to place them

struct KvRows {
  const void* src[2];   // append: new rows K, V [total][Hkv][D]; read: pools
  void* dst[2];         // append: pools [P][PS][Hkv][D]; read: rows
  float* scales[2];     // [P][Hkv][PS] (written by append, read by read)
  const int32_t* page_table;
  const int32_t* offsets;   // [B + 1]
  const int32_t* base;      // append: seq_lens [B]; read: first positions [B] or null (0)
  int32_t* err;
  int32_t total, B, Hkv, D, page_size, max_pages, num_pages, rows_per_block;
};

// Where a row of the chunk sits in the cache: (page, slot), page -1 when it
// has no place there.  Run by one whole warp.
template <bool kAppend>
__device__ __forceinline__ int2 place_row(const KvRows& a, int row, int lane, bool* owned) {
  *owned = false;
  const int b = warp_search(a.B, row, lane, [&](int i) { return (int64_t)a.offsets[i]; });
  if (b < 0) return make_int2(-1, 0);
  const RowRange r = row_range(a.offsets, b, a.total);
  if (!r.ok || row >= r.first + r.count) return make_int2(-1, 0);
  *owned = true;
  const int64_t base = a.base ? a.base[b] : 0;
  const int64_t pos = base + (row - r.first) - (kAppend ? r.count : 0);
  const int64_t capacity = (int64_t)a.max_pages * a.page_size;
  if (pos < 0 || pos >= capacity || (kAppend && base > capacity)) {
    // an append before position 0 is no row; all else is out of the table
    if (lane == 0 && (pos >= 0 || !kAppend || base < 0))
      raise_error(a.err, DECODE_ATTN_DEV_BAD_LEN);
    return make_int2(-1, 0);
  }
  const size_t pi = (size_t)b * a.max_pages + (size_t)(pos / a.page_size);
  const int page = PGD_IN(pi, (size_t)a.B * a.max_pages, a.err) ? a.page_table[pi] : -1;
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) raise_error(a.err, DECODE_ATTN_DEV_BAD_PAGE);
    return make_int2(-1, 0);
  }
  return make_int2(page, (int)(pos % a.page_size));
}

// Offsets that do not ascend inside [0, total], checked once per call.
__device__ __forceinline__ void check_offsets(const KvRows& a) {
  if (blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < a.B; b += kThreads)
    if (!row_range(a.offsets, b, a.total).ok) raise_error(a.err, DECODE_ATTN_DEV_BAD_LEN);
}

template <class E, bool kQuant>
__global__ void __launch_bounds__(kThreads) kv_append_rows_kernel(const KvRows a) {
  __shared__ int2 place_s[kMaxRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.total - row0);
  const int per_head = a.D / 8, per_row = a.Hkv * per_head, items = rows * per_row;
  const uint4* src[2] = {static_cast<const uint4*>(a.src[0]) + (size_t)row0 * per_row,
                         static_cast<const uint4*>(a.src[1]) + (size_t)row0 * per_row};
  grid_dependency_wait();
  grid_launch_dependents();
  uint4 x[2] = {};
  if ((int)threadIdx.x < items) {
    x[0] = __ldg(src[0] + threadIdx.x);
    x[1] = __ldg(src[1] + threadIdx.x);
  }
  if (warp < rows) {
    bool owned;
    const int2 at = place_row<true>(a, row0 + warp, lane, &owned);
    if (lane == 0) place_s[warp] = at;
  }
  check_offsets(a);
  __syncthreads();
  // whole warps walk the items together (the row maximum is a shuffle)
  for (int e0 = warp * 32; e0 < items; e0 += kThreads) {
    const int e = e0 + lane;
    const bool in = e < items;
    if (e0 != warp * 32) {
      x[0] = in ? __ldg(src[0] + e) : make_uint4(0, 0, 0, 0);
      x[1] = in ? __ldg(src[1] + e) : make_uint4(0, 0, 0, 0);
    }
    const int r = in ? e / per_row : 0, c = in ? e % per_row : 0;
    const int2 at = place_s[r];
    const bool go = in && at.x >= 0;
    const int h = c / per_head;
    const size_t cell = ((size_t)at.x * a.page_size + at.y) * per_row + c;
    if constexpr (!kQuant) {
      if (go && PGD_IN(cell, (size_t)a.num_pages * a.page_size * per_row, a.err))
        for (int i = 0; i < 2; ++i) static_cast<uint4*>(a.dst[i])[cell] = x[i];
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float2 f[4];
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[k] = ElemOps<E>::unpack2(w[k]);
          amax = fmaxf(amax, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
        }
        for (int k = 1; k < per_head; k <<= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
        const RowScale s = e4m3_scale(amax);
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = e4m3_pack2(f[k].x * s.inv, f[k].y * s.inv);
        if (!go || !PGD_IN(cell, (size_t)a.num_pages * a.page_size * per_row, a.err)) continue;
        static_cast<uint2*>(a.dst[i])[cell] =
            make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        if (c % per_head == 0)
          a.scales[i][((size_t)at.x * a.Hkv + h) * a.page_size + at.y] = s.scale;
      }
    }
  }
}

template <class E, bool kQuant>
__global__ void __launch_bounds__(kThreads) kv_read_rows_kernel(const KvRows a) {
  __shared__ int2 place_s[kMaxRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.total - row0);
  const int per_head = a.D / 8, per_row = a.Hkv * per_head, items = rows * per_row;
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp < rows) {
    bool owned;
    const int2 at = place_row<false>(a, row0 + warp, lane, &owned);
    if (lane == 0) place_s[warp] = make_int2(owned ? at.x : -2, at.y);
  }
  check_offsets(a);
  __syncthreads();
#pragma unroll 2
  for (int e = threadIdx.x; e < items; e += kThreads) {
    const int r = e / per_row, c = e % per_row;
    const int2 at = place_s[r];
    if (at.x == -2) continue;  // no sequence owns the row
    const size_t cell = ((size_t)at.x * a.page_size + at.y) * per_row + c;
    const bool ok = at.x >= 0 && PGD_IN(cell, (size_t)a.num_pages * a.page_size * per_row, a.err);
    const size_t out = (size_t)row0 * per_row + e;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 y = make_uint4(0, 0, 0, 0);
      if constexpr (!kQuant) {
        if (ok) y = __ldcs(static_cast<const uint4*>(a.src[i]) + cell);
      } else if (ok) {
        const uint2 q = __ldcs(static_cast<const uint2*>(a.src[i]) + cell);
        const float s =
            __ldg(a.scales[i] + ((size_t)at.x * a.Hkv + c / per_head) * a.page_size + at.y);
        const uint32_t pairs[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = ElemOps<__half>::unpack2(e4m3_to_half2(pairs[k]));
          w[k] = ElemOps<E>::pack2(f.x * s, f.y * s);
        }
        y = make_uint4(w[0], w[1], w[2], w[3]);
      }
      static_cast<uint4*>(a.dst[i])[out] = y;
    }
  }
}

template <class Kernel>
int launch_rows(Kernel kern, KvRows& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  int dev = 0, sms = 0, st;
  if (cudaGetDevice(&dev) != cudaSuccess) return DECODE_ATTN_ERR_CUDA;
  if ((st = device_sms(dev, &sms))) return st;
  // a row per block while that leaves SMs idle, then more rows per block
  a.rows_per_block = 1;
  while (a.rows_per_block < kMaxRows && a.total > (int64_t)4 * sms * a.rows_per_block)
    a.rows_per_block *= 2;
  const unsigned blocks = (unsigned)ceil_div(a.total, a.rows_per_block);
  return cuda_status(launch_pdl(kern, done, blocks, kThreads, 0, stream, a));
}

int rows_args(const decode_attn_params* p, int32_t kv_format, int32_t total_rows, KvRows* a) {
  int st = validate_params(p);
  if (st) return st;
  if (total_rows < 0 ||
      (kv_format != DECODE_ATTN_KV_16BIT && kv_format != DECODE_ATTN_KV_E4M3))
    return DECODE_ATTN_ERR_SHAPE;
  a->total = total_rows;
  a->B = p->batch;
  a->Hkv = p->num_kv_heads;
  a->D = p->head_dim;
  a->page_size = p->page_size;
  a->max_pages = p->max_pages_per_seq;
  a->num_pages = p->num_pages;
  return DECODE_ATTN_OK;
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" int decode_kv_append_chunk(const decode_attn_params* p, int32_t kv_format,
                                      int32_t total_rows, const void* k_new, const void* v_new,
                                      const int32_t* row_offsets, const int32_t* seq_lens,
                                      void* k_pages, void* v_pages, float* k_scales,
                                      float* v_scales, const int32_t* page_table,
                                      int32_t* err_flag, void* stream) {
  KvRows a{};
  int st = rows_args(p, kv_format, total_rows, &a);
  if (st || p->batch == 0 || total_rows == 0) return st;
  const bool quant = kv_format == DECODE_ATTN_KV_E4M3;
  if (!k_new || !v_new || !row_offsets || !seq_lens || !k_pages || !v_pages || !page_table ||
      (quant && (!k_scales || !v_scales)))
    return DECODE_ATTN_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages) ||
      (quant && (!aligned16(k_scales) || !aligned16(v_scales))))
    return DECODE_ATTN_ERR_ALIGN;
  a.src[0] = k_new;
  a.src[1] = v_new;
  a.dst[0] = k_pages;
  a.dst[1] = v_pages;
  a.scales[0] = k_scales;
  a.scales[1] = v_scales;
  a.page_table = page_table;
  a.offsets = row_offsets;
  a.base = seq_lens;
  a.err = err_flag;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!quant) return launch_rows(kv_append_rows_kernel<__half, false>, a, s);  // a copy
  return p->dtype == DECODE_ATTN_DTYPE_BF16
             ? launch_rows(kv_append_rows_kernel<__nv_bfloat16, true>, a, s)
             : launch_rows(kv_append_rows_kernel<__half, true>, a, s);
}

extern "C" int decode_kv_read(const decode_attn_params* p, int32_t kv_format, int32_t total_rows,
                              const void* k_pages, const void* v_pages, const float* k_scales,
                              const float* v_scales, const int32_t* page_table,
                              const int32_t* row_offsets, const int32_t* starts, void* k_out,
                              void* v_out, int32_t* err_flag, void* stream) {
  KvRows a{};
  int st = rows_args(p, kv_format, total_rows, &a);
  if (st || p->batch == 0 || total_rows == 0) return st;
  const bool quant = kv_format == DECODE_ATTN_KV_E4M3;
  if (!k_pages || !v_pages || !page_table || !row_offsets || !k_out || !v_out ||
      (quant && (!k_scales || !v_scales)))
    return DECODE_ATTN_ERR_NULL;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_out) || !aligned16(v_out) ||
      (quant && (!aligned16(k_scales) || !aligned16(v_scales))))
    return DECODE_ATTN_ERR_ALIGN;
  a.src[0] = k_pages;
  a.src[1] = v_pages;
  a.dst[0] = k_out;
  a.dst[1] = v_out;
  a.scales[0] = const_cast<float*>(k_scales);
  a.scales[1] = const_cast<float*>(v_scales);
  a.page_table = page_table;
  a.offsets = row_offsets;
  a.base = starts;
  a.err = err_flag;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!quant) return launch_rows(kv_read_rows_kernel<__half, false>, a, s);  // a copy
  return p->dtype == DECODE_ATTN_DTYPE_BF16
             ? launch_rows(kv_read_rows_kernel<__nv_bfloat16, true>, a, s)
             : launch_rows(kv_read_rows_kernel<__half, true>, a, s);
}
