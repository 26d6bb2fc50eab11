// Rows into the paged cache with their rotation, and rows of 4 bits in and out:
// decode_kv_append_rope turns a ragged batch's new keys (and queries) by their
// positions on the way into a cache of 16, 8 or 4 bits, decode_kv_append_fp4
// quantises rows into 4 bits as they are, decode_kv_read_fp4 gathers rows of 4
// bits back to 16.
//
// All move memory: each value is read once and written once.  An append's block
// takes consecutive rows, K and V of every KV head and, two by two, the query heads;
// a thread per row finds the row's sequence and page while every thread's first
// values are already on their way.  A thread handles units of 16 values (rope.cuh) of
// K and of V, or of two query heads, so the D / 16 threads of a head are neighbours in
// a warp and the row's maximum is a few shuffles, K's and V's as the halves of one
// word.  Its unit of the heads it meets is always the same, and so is where the unit's
// blocks of 16 find the rest of their values.
//
// The keys are rounded to the rows' type after the turn, so the cells are
// those of decode_rope followed by an append of its result.
//
// Measured (GB300): called run after run, 32,354 rows of 8 heads of 128, rotated, with 32
// query heads, into 8 bits 120.4 us (6.1 TB/s); 30011 rows of 8 heads of 64 as 16 bits 25
// us (5.2 TB/s: K and V are a fifth of the rows they are sliced from).  Replayed in one
// graph, 32,354 rows into 4 bits 48.6 us (3.5 TB/s: 20 instructions a value, first of them
// the divisions, two operations each; 68 % of the issue slots, the ALU 57 % busy, so neither
// is at its limit, nor is DRAM); 71,533 rows back from 4 bits 64 us (5.9 TB/s; with 16-byte
// stores and 16 values a thread a fourth more); one row each of 64 sequences 3.5 us, the
// launch and two round trips.
#include <algorithm>

#include "chunk_launch.h"
#include "e2m1.cuh"
#include "host_common.h"
#include "kv_rows.cuh"
#include "rope.cuh"

namespace pgd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 64;   // rows of a block, a thread each to place them
constexpr int kBlocksPerSm = 8;  // that a call is cut into, where it has the rows

struct AppendRows : RowMap {
  RopeArgs rope;
  const void* src[3];    // new rows K, V [total][Hkv][D], q [total][Hq][D] or null
  int64_t stride[3];     // between their rows, in 8-value items
  void* dst[2];          // pools
  void* q_out;
  int64_t q_out_stride;
  float* scales[2];      // [P][Hkv][PS]
  uint8_t* blocks[2];    // [P][Hkv][PS][D / 16]
  int32_t Hkv, Hq, rows_per_block;
  FastDiv by_row;        // units of a row: (Hkv + ceil(Hq / 2)) * D / 16
};

// A thread's unit of the block: row r, head (of K and V, or with query set the
// first of two query heads).
struct Place {
  int r, head;
  bool query;
};

// The 16-bit magnitudes of an item's eight values, largest first found: as
// whole numbers, so that an Inf and a NaN stand above all finite values.
__device__ __forceinline__ uint32_t top_bits(uint4 x) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t t = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  return max(t & 0xffffu, t >> 16);
}

// The block maxima of a unit's two items, as 16-bit magnitudes (item a's block
// in the low half): an item's block is its own values and its mate's, item ^ 1.
// Where rope_items puts the two in one unit that is the other item; in half
// pairs the mate is in a neighbour's unit.
template <int kUnits>
struct BlockMates {
  int lane[2];   // lane that holds the mate of item a, b (within the warp)
  int shift[2];  // 0 or 16: as its item a or b
  bool own;
  __device__ __forceinline__ BlockMates(const RopeArgs& r, int unit, int lane_id) {
    const int first = lane_id - unit, half = r.rot / 16;
    own = r.interleaved || unit >= half;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int mate = (own ? 2 * unit + i : unit + i * half) ^ 1;
      const int u = own ? unit : mate < half ? mate : mate - half;
      lane[i] = first + u;
      shift[i] = own ? (i ? 0 : 16) : mate < half ? 0 : 16;
    }
  }
};

// One tensor's item of eight 16-bit values as 4-bit codes.
template <class E>
__device__ __forceinline__ uint32_t pack_codes(uint4 x, const BlockScale& b) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = ElemOps<E>::unpack2(w[i]);
    y[2 * i] = block_div(f.x, b);
    y[2 * i + 1] = block_div(f.y, b);
  }
  const uint32_t r = e2m1_pack8(y);
  return b.inv > 0.f ? r : 0u;
}

template <class E>
__device__ __forceinline__ uint2 pack_e4m3(uint4 x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = ElemOps<E>::unpack2(w[k]);
    q[k] = e4m3_pack2(f.x * inv, f.y * inv);
  }
  return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}

// kFormat: DECODE_ATTN_KV_*; kUnits = D / 16 threads hold a head's row.
template <class E, int kFormat, int kUnits>
__global__ void __launch_bounds__(kThreads) kv_append_turned_kernel(const AppendRows a) {
  constexpr int kItems = 2 * kUnits;  // items of 8 values in a head
  __shared__ int2 place_s[kMaxRows];  // a row's page and slot; page -1: not written
  __shared__ int pos_s[kMaxRows];     // its position; -1: zeros for q, -2: no row
  const int lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.total - row0);
  const int per_row = a.by_row.d, units = rows * per_row;
  const size_t cells = (size_t)a.num_pages * a.page_size * a.Hkv;
  uint4 x[2][2];  // K and V, or two query heads; items a and b
  // a thread's unit of the heads it meets is always the same (a row's units and the
  // block's threads are multiples of a head's)
  const int u = threadIdx.x % kUnits;
  const int2 turned = rope_items(a.rope, u);
  const BlockMates<kUnits> mates(a.rope, u, lane);
  auto place_of = [&](int e) {
    Place p;
    p.r = a.by_row.div(e);
    p.head = (e - p.r * per_row) / kUnits;
    p.query = p.head >= a.Hkv;
    if (p.query) p.head = 2 * (p.head - a.Hkv);
    return p;
  };
  // V is not turned: its unit is 16 neighbouring values
  auto items_of = [&](const Place& p, int i) {
    return i == 1 && !p.query ? make_int2(2 * u, 2 * u + 1) : turned;
  };
  auto load = [&](int e) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (e >= units) continue;
      const Place p = place_of(e);
      const int head = p.head + (p.query ? i : 0);
      if (p.query && head >= a.Hq) continue;
      const int t = p.query ? 2 : i;
      const int2 item = items_of(p, i);
      const uint4* src =
          static_cast<const uint4*>(a.src[t]) + (row0 + p.r) * a.stride[t] + head * kItems;
      x[i][0] = __ldcs(src + item.x);
      x[i][1] = __ldcs(src + item.y);
    }
  };
  grid_dependency_wait();
  grid_launch_dependents();
  load(threadIdx.x);
  if ((int)threadIdx.x < rows) {
    bool owned;
    int pos;
    int2 at = place_row_alone<true>(a, row0 + threadIdx.x, &owned, &pos);
    if (a.rope.rot > 0 && pos >= a.rope.rows) {
      raise_error(a.err, DECODE_ATTN_DEV_BAD_LEN);
      pos = at.x = -1;
    }
    place_s[threadIdx.x] = at;
    pos_s[threadIdx.x] = owned ? pos : -2;
  }
  check_offsets(a, kThreads);
  __syncthreads();
  // whole warps walk the units together (the row maximum is a shuffle)
  for (int e = threadIdx.x; e - lane < units; e += kThreads) {
    if (e != (int)threadIdx.x) load(e);
    const Place p = place_of(min(e, units - 1));
    const int pos = e < units ? pos_s[p.r] : -2;
    const int2 at = place_s[p.r];
    if (pos >= 0 && 16 * u < a.rope.rot) {
      RopePairs turn;
      rope_load(turn, a.rope, pos, u);
      rope_unit<E>(x[0][0], x[0][1], turn, a.rope.interleaved);
      if (p.query) rope_unit<E>(x[1][0], x[1][1], turn, a.rope.interleaved);
    }
    float row_inv[2] = {0.f, 0.f}, row_scale[2] = {0.f, 0.f};
    BlockScale block[2][2];
    if constexpr (kFormat == DECODE_ATTN_KV_E4M3) {
      uint32_t top[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = x[i][0], w = x[i][1];
        top[i] = top2<E>(top2<E>(top2<E>(v.x, v.y), top2<E>(v.z, v.w)),
                         top2<E>(top2<E>(w.x, w.y), top2<E>(w.z, w.w)));
      }
      uint32_t both = top2<E>(__byte_perm(top[0], top[1], 0x5410),
                              __byte_perm(top[0], top[1], 0x7632));
#pragma unroll
      for (int k = 1; k < kUnits; k <<= 1)
        both = top2<E>(both, __shfl_xor_sync(0xffffffffu, both, k));
      const float2 amax = ElemOps<E>::unpack2(both & 0x7fff7fffu);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (a row of NaN alone counts as zeros)
        const RowScale s = e4m3_scale(fmaxf(0.f, i ? amax.y : amax.x));
        row_scale[i] = s.scale;
        row_inv[i] = s.inv;
      }
    }
    if constexpr (kFormat == DECODE_ATTN_KV_E2M1) {
      uint32_t top[2][2];  // block maxima of K's and V's items
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) top[i][k] = top_bits(x[i][k]);
      const uint32_t mine = top[0][0] | top[0][1] << 16;
      top[1][0] = top[1][1] = max(top[1][0], top[1][1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t got = __shfl_sync(0xffffffffu, mine, mates.lane[k]);
        top[0][k] = max(top[0][k], got >> mates.shift[k] & 0xffffu);
      }
      // the row's largest finite magnitude: blocks with an Inf or a NaN aside
      constexpr uint32_t inf = std::is_same<E, __half>::value ? 0x7c00u : 0x7f80u;
      auto finite = [&](uint32_t t) { return t < inf ? t : 0u; };
      uint32_t both = max(finite(top[0][0]), finite(top[0][1])) | finite(top[1][0]) << 16;
#pragma unroll
      for (int k = 1; k < kUnits; k <<= 1)
        both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, k));
      const float2 amax = ElemOps<E>::unpack2(both);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const RowScale s = e2m1_row_scale(i ? amax.y : amax.x);
        row_scale[i] = s.scale;
        row_inv[i] = s.inv;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (i == 1 && k == 1) {
            block[1][1] = block[1][0];
            continue;
          }
          const float m = ElemOps<E>::unpack2(top[i][k]).x;
          block[i][k] = e2m1_block_scale(m, s, top[i][k] < inf);
        }
      }
    }
    if (p.query) {
      if (pos == -2) continue;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (p.head + i >= a.Hq) continue;
        const int2 item = items_of(p, i);
        uint4* dst = static_cast<uint4*>(a.q_out) + (row0 + p.r) * a.q_out_stride +
                     (p.head + i) * kItems;
        dst[item.x] = pos < 0 ? zero : x[i][0];
        dst[item.y] = pos < 0 ? zero : x[i][1];
      }
      continue;
    }
    const size_t cell = ((size_t)at.x * a.page_size + at.y) * a.Hkv + p.head;
    if (pos < 0 || at.x < 0 || !PGD_IN(cell, cells, a.err)) continue;
    const size_t scale_at = ((size_t)at.x * a.Hkv + p.head) * a.page_size + at.y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int2 item = items_of(p, i);
      // (V's two items are neighbours)
      if constexpr (kFormat == DECODE_ATTN_KV_16BIT) {
        uint4* dst = static_cast<uint4*>(a.dst[i]) + cell * kItems;
        dst[item.x] = x[i][0];
        dst[item.y] = x[i][1];
      } else if constexpr (kFormat == DECODE_ATTN_KV_E4M3) {
        const uint2 lo = pack_e4m3<E>(x[i][0], row_inv[i]), hi = pack_e4m3<E>(x[i][1], row_inv[i]);
        uint2* dst = static_cast<uint2*>(a.dst[i]) + cell * kItems;
        if (i == 1) {
          *reinterpret_cast<uint4*>(dst + item.x) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          dst[item.x] = lo;
          dst[item.y] = hi;
        }
      } else {
        const uint32_t lo = pack_codes<E>(x[i][0], block[i][0]);
        const uint32_t hi = pack_codes<E>(x[i][1], block[i][1]);
        uint32_t* dst = static_cast<uint32_t*>(a.dst[i]) + cell * kItems;
        if (i == 1) {
          *reinterpret_cast<uint2*>(dst + item.x) = make_uint2(lo, hi);
        } else {
          dst[item.x] = lo;
          dst[item.y] = hi;
        }
        // a block's scale by the thread of its first item
        uint8_t* at_block = a.blocks[i] + scale_at * kUnits;
        if (!(item.x & 1)) at_block[item.x >> 1] = (uint8_t)block[i][0].code;
        if (!(item.y & 1)) at_block[item.y >> 1] = (uint8_t)block[i][1].code;
      }
      if constexpr (kFormat != DECODE_ATTN_KV_16BIT)
        if (u == 0) a.scales[i][scale_at] = row_scale[i];
    }
  }
}

struct ReadRows : RowMap {
  const uint4* codes[2];      // pools [P][PS][Hkv][D / 32] of 16 bytes
  const float* scales[2];     // [P][Hkv][PS]
  const uint16_t* blocks[2];  // [P][Hkv][PS][D / 32] pairs of blocks
  uint4* out[2];              // [total][Hkv][D]
  int32_t Hkv, rows_per_block;
  int32_t unit_shift;         // units of 32 values in a head, log2
  int32_t wide;               // the outputs lie on 32 bytes
  FastDiv by_row;             // units of a row
};

// 32 bytes in one store (or two): whole sectors.
__device__ __forceinline__ void store_32(uint4* to, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A thread reads units of 32 values of K and of V: 16 bytes of codes, two blocks.
template <class E>
__global__ void __launch_bounds__(kThreads) kv_read_fp4_kernel(const ReadRows a) {
  __shared__ int2 place_s[kMaxRows];  // page -1: zeros, -2: no row
  const int row0 = blockIdx.x * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.total - row0);
  const int per_row = a.Hkv << a.unit_shift, units = rows * per_row;
  grid_dependency_wait();
  grid_launch_dependents();
  if ((int)threadIdx.x < rows) {
    bool owned;
    int pos;
    const int2 at = place_row_alone<false>(a, row0 + threadIdx.x, &owned, &pos);
    place_s[threadIdx.x] = make_int2(owned ? at.x : -2, at.y);
  }
  check_offsets(a, kThreads);
  __syncthreads();
  for (int e = threadIdx.x; e < units; e += kThreads) {
    const int r = a.by_row.div(e), c = e - r * per_row;
    const int2 at = place_s[r];
    if (at.x == -2) continue;  // a row of no sequence
    uint4 q[2] = {};
    uint32_t block[2] = {0u, 0u};
    float s[2] = {0.f, 0.f};
    const size_t cell = ((size_t)at.x * a.page_size + at.y) * per_row + c;
    if (at.x >= 0 && PGD_IN(cell, (size_t)a.num_pages * a.page_size * per_row, a.err)) {
      const int head = c >> a.unit_shift, u = c - (head << a.unit_shift);
      const size_t row = ((size_t)at.x * a.Hkv + head) * a.page_size + at.y;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q[i] = __ldcs(a.codes[i] + cell);
        // (not the read-only path: the kernel before, which an append may be, can still
        // run when this one starts)
        block[i] = a.blocks[i][(row << a.unit_shift) + u];
        s[i] = a.scales[i][row];
      }
    }
    // kSat: a cell beyond the type's range is its largest number (a block's code 6 can
    // stand for more than the value it came from: 65504 becomes 67584); not so under a
    // row scale that is no finite number
    auto put = [&](int i, auto sat) {
      constexpr bool kSat = decltype(sat)::value;
      const uint32_t words[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      const uint32_t two = e4m3_to_half2(block[i]);
      const __half2 pair = *reinterpret_cast<const __half2*>(&two);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const __half2 scale = b ? __high2half2(pair) : __low2half2(pair);
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[4];
          e2m1_to_half8(words[2 * b + k], h);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // code * block is exact in fp16
            const float2 f =
                __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&h[j]), scale));
            w[4 * k + j] = kSat ? pack2_sat<E>(f.x * s[i], f.y * s[i])
                            : ElemOps<E>::pack2(f.x * s[i], f.y * s[i]);
          }
        }
        store_32(a.out[i] + ((size_t)row0 * per_row + e) * 4 + 2 * b, w, a.wide);
      }
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (fabsf(s[i]) < INFINITY)
        put(i, std::true_type{});
      else
        put(i, std::false_type{});
    }
  }
}

// Rows per block: finding the rows' places is most of a small block's time, so a call
// is cut into about 8 blocks an SM of up to 64 rows each, and into more blocks only
// beyond that (30011 rows of 8 heads of 64, 25 rows a block: 25 us, in blocks of 8 rows
// 30; 32,354 rows into 8 bits, with queries, 120.4 and 118.6; 5000 of those without
// queries 13.2 and 14.2).  Four blocks of the append are on an SM at once, six of the
// read.
template <class Kernel, class Args>
int launch_rows(Kernel kern, Args& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  int dev = 0, sms = 0, st;
  if (cudaGetDevice(&dev) != cudaSuccess) return DECODE_ATTN_ERR_CUDA;
  if ((st = device_sms(dev, &sms))) return st;
  a.rows_per_block =
      (int)std::min<int64_t>(kMaxRows, ceil_div(a.total, (int64_t)kBlocksPerSm * sms));
  const unsigned blocks = (unsigned)ceil_div(a.total, a.rows_per_block);
  return cuda_status(launch_pdl(kern, done, blocks, kThreads, 0, stream, a));
}

template <class E, int kFormat>
int launch_append(AppendRows& a, int head_dim, cudaStream_t s) {
  switch (head_dim) {
    case 64: return launch_rows(kv_append_turned_kernel<E, kFormat, 4>, a, s);
    case 128: return launch_rows(kv_append_turned_kernel<E, kFormat, 8>, a, s);
    default: return launch_rows(kv_append_turned_kernel<E, kFormat, 16>, a, s);
  }
}

template <class E>
int launch_append_format(AppendRows& a, int format, int head_dim, cudaStream_t s) {
  switch (format) {
    case DECODE_ATTN_KV_16BIT: return launch_append<E, DECODE_ATTN_KV_16BIT>(a, head_dim, s);
    case DECODE_ATTN_KV_E4M3: return launch_append<E, DECODE_ATTN_KV_E4M3>(a, head_dim, s);
    default: return launch_append<E, DECODE_ATTN_KV_E2M1>(a, head_dim, s);
  }
}

void fill_map(RowMap& a, const decode_attn_params* p, int32_t total) {
  a.total = total;
  a.B = p->batch;
  a.page_size = p->page_size;
  a.max_pages = p->max_pages_per_seq;
  a.num_pages = p->num_pages;
}

// Both appends; rope null: no rotation.
int append(const decode_attn_params* p, const decode_kv_cache* cache, const decode_rope_rows* rope,
           int32_t total_rows, const void* k_new, int64_t k_stride, const void* v_new,
           int64_t v_stride, const int32_t* row_offsets, const int32_t* seq_lens,
           const int32_t* page_table, int32_t* err_flag, void* stream) {
  int st = validate_params(p);
  if (st) return st;
  if (!cache) return DECODE_ATTN_ERR_NULL;
  const int fmt = cache->kv_format;
  if (total_rows < 0 || fmt < DECODE_ATTN_KV_16BIT || fmt > DECODE_ATTN_KV_E2M1)
    return DECODE_ATTN_ERR_SHAPE;
  AppendRows a{};
  fill_map(a, p, total_rows);
  const int D = p->head_dim;
  const int64_t width[3] = {(int64_t)p->num_kv_heads * D, (int64_t)p->num_kv_heads * D,
                            (int64_t)p->num_q_heads * D};
  a.src[0] = k_new;
  a.src[1] = v_new;
  int64_t stride[4] = {k_stride, v_stride, 0, 0};
  if (rope) {
    if (rope->rot_dim < 16 || rope->rot_dim % 16 || rope->rot_dim > D || rope->table_rows <= 0)
      return DECODE_ATTN_ERR_SHAPE;
    a.rope = RopeArgs{rope->table, rope->table_rows, rope->rot_dim, rope->interleaved != 0, 0};
    a.src[2] = rope->q;
    a.q_out = rope->q_out;
    stride[2] = rope->q_stride;
    stride[3] = rope->q_out_stride;
  }
  for (int i = 0; i < 4; ++i) {
    const int64_t w = width[std::min(i, 2)];
    if (stride[i] == 0) stride[i] = w;
    if (stride[i] < w) return DECODE_ATTN_ERR_SHAPE;
    if (stride[i] % 8) return DECODE_ATTN_ERR_ALIGN;
    (i < 3 ? a.stride[i] : a.q_out_stride) = stride[i] / 8;
  }
  if (p->batch == 0 || total_rows == 0) return DECODE_ATTN_OK;
  const bool quant = fmt != DECODE_ATTN_KV_16BIT, fp4 = fmt == DECODE_ATTN_KV_E2M1;
  const void* need[] = {k_new, v_new, row_offsets, seq_lens, cache->k_pages, cache->v_pages,
                        page_table};
  for (const void* ptr : need)
    if (!ptr) return DECODE_ATTN_ERR_NULL;
  if ((quant && (!cache->k_scales || !cache->v_scales)) ||
      (fp4 && (!cache->k_blocks || !cache->v_blocks)) ||
      (rope && (!rope->table || !rope->q != !rope->q_out)))
    return DECODE_ATTN_ERR_NULL;
  const void* aligned[] = {k_new, v_new, cache->k_pages, cache->v_pages,
                           quant ? cache->k_scales : nullptr, quant ? cache->v_scales : nullptr,
                           fp4 ? cache->k_blocks : nullptr, fp4 ? cache->v_blocks : nullptr,
                           a.rope.table, a.src[2], a.q_out};
  for (const void* ptr : aligned)
    if (!aligned16(ptr)) return DECODE_ATTN_ERR_ALIGN;
  a.page_table = page_table;
  a.offsets = row_offsets;
  a.base = seq_lens;
  a.err = err_flag;
  a.dst[0] = cache->k_pages;
  a.dst[1] = cache->v_pages;
  a.scales[0] = cache->k_scales;
  a.scales[1] = cache->v_scales;
  a.blocks[0] = cache->k_blocks;
  a.blocks[1] = cache->v_blocks;
  a.Hkv = p->num_kv_heads;
  a.Hq = a.src[2] ? p->num_q_heads : 0;
  a.by_row = FastDiv::of((a.Hkv + (a.Hq + 1) / 2) * (D / 16));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p->dtype == DECODE_ATTN_DTYPE_BF16 ? launch_append_format<__nv_bfloat16>(a, fmt, D, s)
                                            : launch_append_format<__half>(a, fmt, D, s);
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" int decode_kv_append_rope(const decode_attn_params* p, const decode_kv_cache* cache,
                                     const decode_rope_rows* rope, int32_t total_rows,
                                     const void* k_new, int64_t k_stride, const void* v_new,
                                     int64_t v_stride, const int32_t* row_offsets,
                                     const int32_t* seq_lens, const int32_t* page_table,
                                     int32_t* err_flag, void* stream) {
  if (!rope) return DECODE_ATTN_ERR_NULL;
  return append(p, cache, rope, total_rows, k_new, k_stride, v_new, v_stride, row_offsets,
                seq_lens, page_table, err_flag, stream);
}

extern "C" int decode_kv_append_fp4(const decode_attn_params* p, const decode_kv_cache* cache,
                                    int32_t total_rows, const void* k_new, int64_t k_stride,
                                    const void* v_new, int64_t v_stride,
                                    const int32_t* row_offsets, const int32_t* seq_lens,
                                    const int32_t* page_table, int32_t* err_flag, void* stream) {
  if (cache && cache->kv_format != DECODE_ATTN_KV_E2M1) return DECODE_ATTN_ERR_SHAPE;
  return append(p, cache, nullptr, total_rows, k_new, k_stride, v_new, v_stride, row_offsets,
                seq_lens, page_table, err_flag, stream);
}

extern "C" int decode_kv_read_fp4(const decode_attn_params* p, const decode_kv_cache* cache,
                                  int32_t total_rows, const int32_t* page_table,
                                  const int32_t* row_offsets, const int32_t* starts, void* k_out,
                                  void* v_out, int32_t* err_flag, void* stream) {
  int st = validate_params(p);
  if (st) return st;
  if (!cache) return DECODE_ATTN_ERR_NULL;
  if (total_rows < 0 || cache->kv_format != DECODE_ATTN_KV_E2M1) return DECODE_ATTN_ERR_SHAPE;
  if (p->batch == 0 || total_rows == 0) return DECODE_ATTN_OK;
  const void* need[] = {cache->k_pages, cache->v_pages, cache->k_scales, cache->v_scales,
                        cache->k_blocks, cache->v_blocks, k_out, v_out, page_table, row_offsets};
  for (const void* ptr : need)
    if (!ptr) return DECODE_ATTN_ERR_NULL;
  for (int i = 0; i < 8; ++i)
    if (!aligned16(need[i])) return DECODE_ATTN_ERR_ALIGN;
  ReadRows a{};
  fill_map(a, p, total_rows);
  a.codes[0] = static_cast<const uint4*>(cache->k_pages);
  a.codes[1] = static_cast<const uint4*>(cache->v_pages);
  a.scales[0] = cache->k_scales;
  a.scales[1] = cache->v_scales;
  a.blocks[0] = reinterpret_cast<const uint16_t*>(cache->k_blocks);
  a.blocks[1] = reinterpret_cast<const uint16_t*>(cache->v_blocks);
  a.wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  a.out[0] = static_cast<uint4*>(k_out);
  a.out[1] = static_cast<uint4*>(v_out);
  a.page_table = page_table;
  a.offsets = row_offsets;
  a.base = starts;
  a.err = err_flag;
  a.Hkv = p->num_kv_heads;
  a.unit_shift = ilog2(p->head_dim / 32);
  a.by_row = FastDiv::of(p->num_kv_heads << a.unit_shift);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p->dtype == DECODE_ATTN_DTYPE_BF16 ? launch_rows(kv_read_fp4_kernel<__nv_bfloat16>, a, s)
                                            : launch_rows(kv_read_fp4_kernel<__half>, a, s);
}
