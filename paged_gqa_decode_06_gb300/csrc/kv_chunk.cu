// Rows in and out of the paged cache by the chunk: decode_kv_append_chunk
// scatters a ragged batch's new K/V rows into their pages, as they are or
// quantised (e4m3.cuh), and decode_kv_read gathers rows back to contiguous
// 16-bit rows.
//
// Both move memory: each value is read once and written once.  A block takes
// a few consecutive rows with all their heads; one warp per row finds the
// row's sequence and page while (in an append) every thread's first values are
// already on their way.  A thread handles 8 values of a row's head, so the D /
// 8 threads of a head are neighbours in a warp and the row's maximum is a few
// shuffles.
//
// Memory bounds the read, and what reaches its rate is the number of loads in
// flight: all loads of kBatch items before the first store.  131072 rows of 8
// heads of 128 read from e4m3: 124 us, 6.5 TB/s (with 1 item 151, with 4
// items, and fewer blocks per SM for their registers, 127; 4 rows per block
// 160, 16 rows 128).  A quantising append issues as much as it moves (80 % of
// the issue slots with each tensor's maximum shuffled by itself): K's and V's
// row maxima share one shuffle as the halves of a word, and the count of
// shuffles is fixed at compile time.  32,354 fp16 rows: 36.6 us, 5.5 TB/s
// (with separate shuffles in a loop 40.5), of which about 5 are the launch and
// the placing of the first rows.
#include <algorithm>
#include <type_traits>

#include "chunk_launch.h"
#include "e4m3.cuh"
#include "host_common.h"

namespace pgd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;  // rows of a block, one warp each to place them
constexpr int kBatch = 2;    // items of 8 values whose loads a thread has in flight

struct KvRows {
  const void* src[2];   // append: new rows K, V [total][Hkv][D]; read: pools
  void* dst[2];         // append: pools [P][PS][Hkv][D]; read: rows
  float* scales[2];     // [P][Hkv][PS] (written by append, read by read)
  const int32_t* page_table;
  const int32_t* offsets;   // [B + 1]
  const int32_t* base;      // append: seq_lens [B]; read: first positions [B] or null (0)
  int32_t* err;
  int32_t total, B, Hkv, D, page_size, max_pages, num_pages, rows_per_block;
  int32_t head_shift;  // 8-value items of a head, log2
  FastDiv by_row;      // items of a row
};

// Where a row of the chunk sits in the cache: (page, slot), page -1 when it
// has no place there.  Run by one whole warp.
template <bool kAppend>
__device__ __forceinline__ int2 place_row(const KvRows& a, int row, int lane, bool* owned) {
  *owned = false;
  const int b = warp_search(a.B, row, lane, [&](int i) { return (int64_t)a.offsets[i]; });
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

// kLanes threads hold a head's row (D / 8); 0: 16-bit rows, copied.
template <class E, int kLanes>
__global__ void __launch_bounds__(kThreads) kv_append_rows_kernel(const KvRows a) {
  constexpr bool kQuant = kLanes > 0;
  __shared__ int64_t cell_s[kMaxRows];   // a row's first 8 values in the pool, or -1
  __shared__ int64_t scale_s[kMaxRows];  // its first head's scale
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.total - row0);
  const int per_row = a.Hkv << a.head_shift, items = rows * per_row;
  const size_t cells = (size_t)a.num_pages * a.page_size * per_row;
  const uint4* src[2] = {static_cast<const uint4*>(a.src[0]) + (size_t)row0 * per_row,
                         static_cast<const uint4*>(a.src[1]) + (size_t)row0 * per_row};
  uint4 x[kBatch][2];
  auto load = [&](int e0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = e0 + u * kThreads;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[u][i] = e < items ? __ldcs(src[i] + e) : make_uint4(0, 0, 0, 0);
    }
  };
  grid_dependency_wait();
  grid_launch_dependents();
  load(threadIdx.x);
  if (warp < rows) {
    bool owned;
    const int2 at = place_row<true>(a, row0 + warp, lane, &owned);
    if (lane == 0) {
      cell_s[warp] = at.x < 0 ? -1 : ((int64_t)at.x * a.page_size + at.y) * per_row;
      scale_s[warp] = (int64_t)at.x * a.Hkv * a.page_size + at.y;
    }
  }
  check_offsets(a);
  __syncthreads();
  // whole warps walk the items together (the row maximum is a shuffle)
  for (int e0 = threadIdx.x; e0 - lane < items; e0 += kThreads * kBatch) {
    if (e0 != (int)threadIdx.x) load(e0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = e0 + u * kThreads;
      if (e - lane >= items) break;
      const int r = e < items ? (int)a.by_row.div(e) : 0;
      const int c = e < items ? e - r * per_row : 0;
      const int64_t first = cell_s[r];
      const size_t cell = first + c;
      const bool go = e < items && first >= 0 && PGD_IN(cell, cells, a.err);
      if constexpr (!kQuant) {
        if (go)
          for (int i = 0; i < 2; ++i) static_cast<uint4*>(a.dst[i])[cell] = x[u][i];
      } else {
        // the largest magnitudes of K's values (low half) and V's
        uint32_t top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          top[i] = top2<E>(top2<E>(x[u][i].x, x[u][i].y), top2<E>(x[u][i].z, x[u][i].w));
        uint32_t both = top2<E>(__byte_perm(top[0], top[1], 0x5410),
                                __byte_perm(top[0], top[1], 0x7632));
#pragma unroll
        for (int k = 1; k < kLanes; k <<= 1)
          both = top2<E>(both, __shfl_xor_sync(0xffffffffu, both, k));
        const float2 amax = ElemOps<E>::unpack2(both & 0x7fff7fffu);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // (a row of NaN alone counts as zeros)
          const RowScale s = e4m3_scale(fmaxf(0.f, i ? amax.y : amax.x));
          const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
          uint32_t q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = ElemOps<E>::unpack2(w[k]);
            q[k] = e4m3_pack2(f.x * s.inv, f.y * s.inv);
          }
          if (!go) continue;
          static_cast<uint2*>(a.dst[i])[cell] =
              make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
          if ((c & (kLanes - 1)) == 0)
            a.scales[i][scale_s[r] + (c >> a.head_shift) * a.page_size] = s.scale;
        }
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
  const int per_row = a.Hkv << a.head_shift, items = rows * per_row;
  const size_t cells = (size_t)a.num_pages * a.page_size * per_row;
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp < rows) {
    bool owned;
    const int2 at = place_row<false>(a, row0 + warp, lane, &owned);
    if (lane == 0) place_s[warp] = make_int2(owned ? at.x : -2, at.y);
  }
  check_offsets(a);
  __syncthreads();
  for (int e0 = threadIdx.x; e0 < items; e0 += kThreads * kBatch) {
    using Raw = std::conditional_t<kQuant, uint2, uint4>;
    Raw x[kBatch][2];
    float s[kBatch][2];
    int page[kBatch];
    // every load of the batch before its first store
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = e0 + u * kThreads;
      page[u] = -2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[u][i] = Raw{};
        s[u][i] = 0.f;
      }
      if (e >= items) continue;
      const int r = a.by_row.div(e), c = e - r * per_row;
      const int2 at = place_s[r];
      page[u] = at.x;
      const size_t cell = ((size_t)at.x * a.page_size + at.y) * per_row + c;
      if (at.x < 0 || !PGD_IN(cell, cells, a.err)) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[u][i] = __ldcs(static_cast<const Raw*>(a.src[i]) + cell);
        if constexpr (kQuant)
          s[u][i] = __ldg(a.scales[i] +
                          ((size_t)at.x * a.Hkv + (c >> a.head_shift)) * a.page_size + at.y);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = e0 + u * kThreads;
      if (page[u] == -2) continue;  // no row, or one of no sequence
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 y;
        if constexpr (!kQuant) {
          y = x[u][i];
        } else {
          const uint2 q = x[u][i];
          const uint32_t pairs[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = ElemOps<__half>::unpack2(e4m3_to_half2(pairs[k]));
            w[k] = ElemOps<E>::pack2(f.x * s[u][i], f.y * s[u][i]);
          }
          y = make_uint4(w[0], w[1], w[2], w[3]);
        }
        static_cast<uint4*>(a.dst[i])[(size_t)row0 * per_row + e] = y;
      }
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
  for (a->head_shift = 3; (8 << a->head_shift) < p->head_dim;) ++a->head_shift;
  a->by_row = FastDiv::of(p->num_kv_heads << a->head_shift);
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
  if (!quant) return launch_rows(kv_append_rows_kernel<__half, 0>, a, s);  // a copy
  const bool bf16 = p->dtype == DECODE_ATTN_DTYPE_BF16;
  switch (a.D) {
    case 64:
      return bf16 ? launch_rows(kv_append_rows_kernel<__nv_bfloat16, 8>, a, s)
                  : launch_rows(kv_append_rows_kernel<__half, 8>, a, s);
    case 128:
      return bf16 ? launch_rows(kv_append_rows_kernel<__nv_bfloat16, 16>, a, s)
                  : launch_rows(kv_append_rows_kernel<__half, 16>, a, s);
    default:
      return bf16 ? launch_rows(kv_append_rows_kernel<__nv_bfloat16, 32>, a, s)
                  : launch_rows(kv_append_rows_kernel<__half, 32>, a, s);
  }
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
