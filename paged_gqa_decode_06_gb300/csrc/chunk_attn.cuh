// Attention of a chunk of new tokens over the paged cache: a ragged batch of
// query tokens (sequence b brings n_b of them, the last n_b of its L_b
// positions), causal, grouped-query, with an optional sliding window:
//   out[t] = sum_k softmax_k(scale * q_t . k) v_k,  k in (p_t - window, p_t].
//
// One CTA owns (tiles of query rows, KV head h, shard of the key range).  The
// G query heads of the group are packed with the tokens into the 128 rows of
// a matrix-instruction tile (row = token * G + g, floor(128 / G) tokens), so
// a K/V row read serves every head of the group and a short chunk still fills
// the tile.  Two such tiles (streams) share every K/V tile at head_dim <= 128;
// at 256 the accumulator of one fills half of the tensor memory.
//
// Both products run on tcgen05: S = Q . K^T from shared memory into tensor
// memory, and O += P . V with P read from tensor memory, where the softmax
// threads write it over S.  Roles: a producer warp (TMA through the page
// table), a warp that issues the matrix instructions, and 128 threads per
// stream that keep one row each (running maximum, sum).  The issue order is
//   S(0) S(1) | O(0) S(2) | O(1) S(3) | ...
// over units u = (key tile, stream): while the softmax of one unit runs, the
// products of the other stream do, so each hides the other.
//
// Both K and V tiles lie in shared memory as [group of 8 tokens][D / 64][8
// tokens][64 dims] with the 128-byte swizzle: one TMA box brings a page's
// piece with all its dims (a 5-D view of the pool), and the groups are evenly
// spaced whatever the page size, which is what an operand descriptor wants:
// K as K-major with D * 16 bytes between groups of 8 tokens, V as MN-major
// with 1024 bytes between chunks of 64 dims.
//
// Keys that only some rows of the CTA attend (the diagonal, a window's start,
// a page's unused positions) lie in the edge tiles.  There the mask is
// applied score by score, and two more warps look V over before its product:
// what no row attends becomes zero, and a NaN or Inf is set to zero and added
// in the epilogue to the rows that attend it, since a product with a weight of
// zero would carry it to the others.
//
// P is rounded once to the element type for the second product, half a step of
// that type each.  An fp16 weight ends at 2^-24, so the reference that a row's
// weights are taken against follows its tiles' maxima down as well as up: the
// largest weight of a tile is 2^2 where it is taken (2^12 in a row's first tile
// with one key far above the others, as a first token that draws all attention
// is), at most 2^15.9 later, and one tile's maximum alone does not hold it up.  So
// the weights that are no normal numbers, off by 2^-25, lose at most 2^-8 of
// what the row has beside its largest tile, and of that tile what is below
// 2^-27 (2^-37) of its largest.  (With a first weight of 1 that is never lowered,
// a context 2^-25 below its first token is lost: all of the output, if that token
// has no value of its own.)  bf16 weights have exponents to spare: they start at
// 2^-16 and stay at or below 1, so that large values do not overflow before they
// are divided by the sum (2^-40 where scores have risen beyond that: values
// below 2^-86 lose bits there).  Sums, maxima and accumulators are fp32.
//
// Measured (GB300): a prompt of 8192 tokens, 32 heads over 8, 348 us, 1.58
// PFLOP/s; 1024 tokens at 131072, 64 heads over 8, 2.7 ms, 1.6 PFLOP/s (3.1 ms
// run after run, where the power limit lowers the clock); at head_dim 256 with a
// window of 1024, three times 1001 tokens, 73 us, 0.69 PFLOP/s.  What bounds it:
// a pair of 128 x 128 tiles takes about 2670 cycles of the tensor cores' 2140
// (8 products of 128 x 128 x 16 take 520 to 550), the chain of barriers between
// product, softmax and product being the rest, and a CTA adds 8 us before its
// first and after its last product.  With loads that cost nothing the prompt
// takes 340 us.  At head_dim 256 that chain is the whole bound: two S buffers
// of 64 keys fit, a tile takes 1800 cycles of the products' 1260, with the row
// threads doubled as well.
#pragma once

#include <type_traits>

#include "combine.cuh"  // grid_dependency_wait, grid_launch_dependents
#include "elem.cuh"
#include "ragged.cuh"
#include "tcgen05.cuh"

namespace pgd {

struct ChunkArgs {
  const int32_t* page_table;  // [B][max_pages]
  const int32_t* offsets;     // [B + 1] rows of each sequence
  const int32_t* seq_lens;    // [B]
  const void* v_pages;
  void* out;                  // [total][Hq][D]
  float* ws_acc;              // [total * Hq][max_shards][D]   (split plans)
  float2* ws_ml;              // [total * Hq][max_shards]; l = -1 marks a bad row
  int32_t* err;               // nullable
  int32_t B, total, Hq, Hkv, G;
  int32_t max_pages, num_pages, page_size, page_shift, box_t;
  int32_t window;
  int32_t tile_tok;           // tokens of one stream's 128 rows
  int32_t item_tok;           // tokens of one CTA (all streams)
  int32_t slots;              // tiles of item_tok tokens over all sequences, at most
  int32_t max_shards, shard_tiles;
  FastDiv by_item, by_heads, by_shards, by_shard_tiles, by_group;
  int32_t stall_tx;           // 0; a test sets extra bytes on the first K tile's barrier
  float scale_log2;
};

// The barriers of a CTA's pipeline: kRing tiles of K and V, kStreams streams.
template <int kRing, int kStreams, int kParts>
struct __align__(8) ChunkBars {
  uint64_t q_full;            // Q has landed
  uint64_t full[kRing];       // a K or V tile has landed
  uint64_t empty[kRing];      // the products are done with it
  uint64_t s_full[2];         // scores of a unit are in tensor memory
  uint64_t p_full[2][kParts]; // so are its weights, 64 keys each
  uint64_t o_full[kStreams];  // a unit's product is in O
  uint64_t done[kStreams];    // so is the last one's
  uint64_t v_edge, v_clean;   // an edge tile's V has landed; is looked over
};

// One CTA's share of the work, found from its slot.
struct ChunkItem {
  int32_t b, t0, t1;     // sequence, its query tokens [t0, t1)
  int32_t row0;          // row of t0 among all tokens
  int32_t p0;            // position of t0
  int32_t lo, hi;        // keys that some query of the item attends
  int32_t base, tiles;   // first key of the first tile, number of key tiles
  int32_t shards;        // CTAs that share the tiles (0: nothing to attend)
  int32_t status;
  bool any;              // the slot holds query tokens
};

// What the CTA shares beside Q and the ring.
template <int kRing, int kStreams, int kKeys, int kMaxEdges>
struct ChunkShared {
  ChunkBars<kRing, kStreams, kKeys / 64> bar;
  ChunkItem item;
  __align__(16) int32_t coord[16];  // row groups of a tile's pieces
  uint32_t tmem;
  int32_t abort;
  int32_t bad_lo, bad_hi;  // positions in pages outside the pool
  // keys of the edge tiles whose V row is not finite
  uint32_t wild[kMaxEdges][kKeys / 32];
  int32_t edge_key[kMaxEdges], wild_any;
};

template <int D>
struct ChunkCfg {
  static constexpr int kStreams = D <= 128 ? 2 : 1;
  static constexpr int kKeys = D <= 128 ? 128 : 64;  // keys of one tile
  static constexpr int kThreads = kStreams * 128 + 128;
  static constexpr int kParts = kKeys / 64;  // P is handed over 64 keys at a time
  static constexpr int kTileBytes = kKeys * D * 2;
  static constexpr int kQBytes = 128 * D * 2;  // one stream
  // the ring holds K and V tiles in turn
  static constexpr int kRing = D == 64 ? 8 : 5;
  static constexpr uint32_t kTmemCols = 512;
  // edge tiles of one CTA: the diagonal and a window's start each cross at
  // most 3 tiles (256 tokens, 128 at D = 256)
  static constexpr int kMaxEdges = 8;
  using Bars = ChunkBars<kRing, kStreams, kParts>;
  using Shared = ChunkShared<kRing, kStreams, kKeys, kMaxEdges>;
  static constexpr int kSmemBytes = kStreams * kQBytes + kRing * kTileBytes + sizeof(Shared);
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
};

// Sequence b owns the slots [offsets[b] / item_tok + b, offsets[b+1] /
// item_tok + b + 1): at least the tiles it needs, and an ascending function
// of b, so a slot finds its sequence by search.
template <int KT>
__device__ __forceinline__ ChunkItem chunk_item(const ChunkArgs& a, int slot, int lane) {
  ChunkItem it{};
  int b;
  RowRange r;
  int32_t L = 0;
  if (a.B < 32) {  // one round trip: every offset and length at once
    const int32_t off = lane <= a.B ? ld_global_s32(a.offsets + lane) : 0;
    const int32_t len = lane < a.B ? ld_global_s32(a.seq_lens + lane) : 0;
    const bool le = lane < a.B && (int)a.by_item.div(max(off, 0)) + lane <= slot;
    b = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    if (b < 0) return it;
    const int32_t z = __shfl_sync(0xffffffffu, off, b + 1);
    r.first = __shfl_sync(0xffffffffu, off, b);
    r.ok = r.first >= 0 && r.first <= z && z <= a.total;
    r.count = r.ok ? z - r.first : 0;
    L = __shfl_sync(0xffffffffu, len, b);
  } else {
    b = warp_search(a.B, slot, lane,
                    [&](int i) { return (int64_t)a.by_item.div(max(a.offsets[i], 0)) + i; });
    if (b < 0) return it;
    r = row_range(a.offsets, b, a.total);
    L = ld_global_s32(a.seq_lens + b);
  }
  it.b = b;
  if (!r.ok) {
    it.status = DECODE_ATTN_DEV_BAD_LEN;
    return it;
  }
  const int64_t t0 = ((int64_t)slot - (a.by_item.div(r.first) + b)) * a.item_tok;
  if (t0 < 0 || t0 >= r.count) return it;
  it.any = true;
  it.t0 = (int32_t)t0;
  it.t1 = min(r.count, it.t0 + a.item_tok);
  it.row0 = r.first + it.t0;
  if (L < 0 || L > a.max_pages * a.page_size) {
    it.status = DECODE_ATTN_DEV_BAD_LEN;
    return it;
  }
  it.p0 = L - r.count + it.t0;
  it.hi = max(0, it.p0 + (it.t1 - it.t0));
  it.lo = a.window > 0 ? max(0, it.p0 - a.window + 1) : 0;
  it.base = it.lo & ~(KT - 1);
  it.tiles = it.hi > it.lo ? (it.hi - it.base + KT - 1) / KT : 0;
  it.shards = min(a.max_shards, (int)a.by_shard_tiles.div(it.tiles + a.shard_tiles - 1));
  return it;
}

// A bit per 16-bit value of w that is not finite (all of its bits set).
template <class E>
__device__ __forceinline__ uint32_t wild2(uint32_t w) {
  constexpr uint32_t kExp = std::is_same<E, __nv_bfloat16>::value ? 0x7f807f80u : 0x7c007c00u;
  return __vcmpeq2(w & kExp, kExp);
}

// Larger magnitude of each of two 16-bit values; NaN if either is.
template <class E>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<E, __nv_bfloat16>::value) {
    const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<__nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<__nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
  } else {
    const __half2 m = __hmax2_nan(__habs2(*reinterpret_cast<__half2*>(&a)),
                                  __habs2(*reinterpret_cast<__half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
}

// The lowest n bits, for any n.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : 0xffffffffu >> (32 - min(n, 32));
}

template <int D>
__device__ __forceinline__ uint64_t k_desc(uint32_t tile) {
  return tc_desc(tile, 16, D * 16);
}
template <int D>
__device__ __forceinline__ uint64_t v_desc(uint32_t tile) {
  return tc_desc(tile, 1024, D * 16);
}

// A tile's place in the ring: K and V tiles alternate, so the next one of
// either is two places on.
template <int NR>
struct RingPos {
  int slot, phase;
  __device__ void next() {
    slot += 2;
    if (slot >= NR) {
      slot -= NR;
      phase ^= 1;
    }
  }
};

// Waits for and issues every product of the CTA, in one thread: the pace of
// this loop is the pace of the tensor cores.  NA streams are active; unit u
// is (tile u / NA, stream u % NA) and uses S buffer u % 2.
template <int D, class E, int NA, class Edge>
__device__ __forceinline__ void chunk_issue(typename ChunkCfg<D>::Bars& bar, uint8_t* smem,
                                            uint32_t tmem, int ntiles, Edge edge,
                                            volatile int32_t* abort, const ChunkArgs& a) {
  using C = ChunkCfg<D>;
  constexpr int KT = C::kKeys, NR = C::kRing;
  constexpr bool kBf16 = std::is_same<E, __nv_bfloat16>::value;
  // a negative scale turns the scores' sign here, so that the softmax only
  // sees its magnitude
  const uint32_t idesc_s = tc_idesc(128, KT, kBf16, false) | (a.scale_log2 < 0.f ? kIdescNegA : 0u);
  constexpr uint32_t kIdescO = tc_idesc(128, D, kBf16, true);
  constexpr uint32_t kTile16 = C::kTileBytes / 16;
  const uint64_t qd = tc_desc(smem_u32(smem), 16, 1024);
  const uint64_t kd = k_desc<D>(smem_u32(smem + C::kStreams * C::kQBytes));
  const uint64_t vd = v_desc<D>(smem_u32(smem + C::kStreams * C::kQBytes));
  const uint32_t tmem_o = tmem + 2 * KT;
  bool ok = true;
  auto wait = [&](uint64_t* b, int parity) {
    if (ok && !mbar_wait_hot(smem_u32(b), parity)) {
      *abort = 1;
      raise_error(a.err, DECODE_ATTN_DEV_TIMEOUT);
      ok = false;
    }
  };
  RingPos<NR> kp{0, 0}, vp{1, 0};
  // S = Q . K^T of stream s and the tile at kp, into buffer buf
  auto issue_s = [&](int s, int buf) {
    if (s == 0) wait(&bar.full[kp.slot], kp.phase);
    if (!ok) return;
    tc_fence_after();
    const uint64_t q0 = qd + s * (C::kQBytes / 16), k0 = kd + kp.slot * kTile16;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const int c = ks >> 2, in = (ks & 3) * 2;  // 32 bytes inside a 64-dim chunk
      tc_mma_ss(tmem + buf * KT, q0 + c * (128 * 128 / 16) + in, k0 + c * (1024 / 16) + in,
                idesc_s, ks > 0);
    }
    tc_commit(smem_u32(&bar.s_full[buf]));
    if (s == NA - 1) {
      tc_commit(smem_u32(&bar.empty[kp.slot]));
      kp.next();
    }
  };
  wait(&bar.q_full, 0);
  issue_s(0, 0);
  if (NA == 2)
    issue_s(1, 1);
  else if (ntiles > 1)
    issue_s(0, 1);
  int cleaned = 0;        // edge tiles looked over so far
  bool told = false;      // V of this tile has landed and, an edge tile's, been handed over
  bool is_edge = edge(0);
  for (int j = 0; j < ntiles && ok; ++j) {
    if (!told) {
      wait(&bar.full[vp.slot], vp.phase);
      if (is_edge) mbar_arrive(smem_u32(&bar.v_edge));
    }
    const bool look = is_edge;
#pragma unroll
    for (int s = 0; s < NA; ++s) {
      const int buf = NA == 2 ? s : (j & 1), phase = NA == 2 ? (j & 1) : ((j >> 1) & 1);
#pragma unroll
      for (int part = 0; part < C::kParts; ++part) {
        wait(&bar.p_full[buf][part], phase);
        if (part == 0 && s == 0 && look) wait(&bar.v_clean, cleaned++ & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t v0 = vd + vp.slot * kTile16 + part * (64 * D * 2 / 16);
        const uint32_t p0 = tmem + buf * KT + part * 32;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)  // O += P . V, 64 keys
          tc_mma_ts(tmem_o + s * D, p0 + ks * 8, v0 + ks * (D * 32 / 16), kIdescO,
                    j > 0 || part > 0 || ks > 0);
      }
      tc_commit(smem_u32(&bar.o_full[s]));
      if (j == ntiles - 1) tc_commit(smem_u32(&bar.done[s]));
      if (s == NA - 1) {
        tc_commit(smem_u32(&bar.empty[vp.slot]));
        vp.next();
        // What the next tile needs is seen to here, where the products queued
        // above still run: V, if it has come already, and an edge tile's is
        // handed over to be looked at while the weights are made.
        is_edge = edge(j + 1);
        told = j + 1 < ntiles && mbar_try_wait(smem_u32(&bar.full[vp.slot]), vp.phase);
        if (told && is_edge) mbar_arrive(smem_u32(&bar.v_edge));
      }
      if (j + (NA == 2 ? 1 : 2) < ntiles) issue_s(s, buf);
    }
  }
}

template <int D, class E>
__global__ void __launch_bounds__(ChunkCfg<D>::kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const ChunkArgs a) {
  using C = ChunkCfg<D>;
  constexpr int NS = C::kStreams, KT = C::kKeys, NR = C::kRing;
  constexpr int kProducer = NS * 4, kMma = NS * 4 + 1;  // warps

  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + NS * C::kQBytes;
  typename C::Shared& sh = *reinterpret_cast<typename C::Shared*>(ring + NR * C::kTileBytes);
  typename C::Bars& bar = sh.bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == kProducer * 32) {
    prefetch_tensormap(&tmap_q);
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    mbar_init(smem_u32(&bar.q_full), 1);
    for (int i = 0; i < NR; ++i) {
      mbar_init(smem_u32(&bar.full[i]), 1);
      mbar_init(smem_u32(&bar.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar.s_full[i]), 1);
      for (int k = 0; k < C::kParts; ++k) mbar_init(smem_u32(&bar.p_full[i][k]), 4);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&bar.o_full[i]), 1);
      mbar_init(smem_u32(&bar.done[i]), 1);
    }
    mbar_init(smem_u32(&bar.v_edge), 1);
    mbar_init(smem_u32(&bar.v_clean), 2);
    fence_mbar_init();
    sh.abort = 0;
    sh.bad_lo = INT32_MAX;
    sh.bad_hi = -1;
    sh.wild_any = 0;
  }
  for (int i = threadIdx.x; i < C::kMaxEdges * KT / 32; i += C::kThreads)
    sh.wild[i / (KT / 32)][i % (KT / 32)] = 0u;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  const int rest = a.by_heads.div(blockIdx.x), h = blockIdx.x - rest * a.Hkv;
  const int place = a.by_shards.div(rest), shard = rest - place * a.max_shards;
  // the last tiles of a sequence see the most keys: they start first
  const int slot = a.slots - 1 - place;
  // The issuing warp allocates the tensor memory while the others look for
  // their item, and takes it from them.
  constexpr int kOthers = NS * 128 + 32;  // the row threads and the issuing warp
  ChunkItem it{};
  if (warp == kMma) {
    tmem_alloc(smem_u32(&sh.tmem), C::kTmemCols);
    tc_fence_before();
  } else {
    it = chunk_item<KT>(a, slot, lane);
  }
  if (threadIdx.x == 0) sh.item = it;
  if (warp < kProducer || warp == kMma) {
    named_barrier_sync(1, kOthers);
    tc_fence_after();
  }
  if (warp == kMma) {
    it = sh.item;
    if (!it.any || shard >= it.shards) tmem_free(sh.tmem, C::kTmemCols);
  }
  if (blockIdx.x == 0)  // offsets that no slot may lead to are checked once
    for (int b = threadIdx.x; b < a.B; b += C::kThreads)
      if (!row_range(a.offsets, b, a.total).ok) raise_error(a.err, DECODE_ATTN_DEV_BAD_LEN);
  if (it.status != 0 && threadIdx.x == 0) raise_error(a.err, it.status);
  if (!it.any) return;
  if (it.shards == 0) {  // no key: zero rows
    if (shard == 0) {
      uint4* out = reinterpret_cast<uint4*>(a.out);
      const int chunks = a.G * D / 8;
      for (int e = threadIdx.x; e < (it.t1 - it.t0) * chunks; e += C::kThreads) {
        const size_t at = ((size_t)(it.row0 + e / chunks) * a.Hq + (size_t)h * a.G) * (D / 8) +
                          e % chunks;
        if (PGD_IN(at, (size_t)a.total * a.Hq * (D / 8), a.err)) out[at] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  if (shard >= it.shards) return;
  // (at most 2^24 tiles and 128 shards)
  int tile0 = 0, ntiles = it.tiles;
  if (it.shards > 1) {
    tile0 = (uint32_t)it.tiles * shard / (uint32_t)it.shards;
    ntiles = (uint32_t)it.tiles * (shard + 1) / (uint32_t)it.shards - tile0;
  }
  const int key0 = it.base + tile0 * KT;  // first key of this CTA's first tile
  const int ns = (it.t1 - it.t0) > a.tile_tok ? NS : 1;  // streams with tokens
  // whether some row of the CTA does not attend all of tile j: its last key
  // is after the first row's position, or its first before the last's window
  const int edge_from = max(0, it.p0 - key0 + 1) / KT;
  const int edge_to =
      a.window > 0 ? it.p0 + (it.t1 - it.t0) - 1 - a.window - key0 : -1;
  auto edge = [&](int j) { return j >= edge_from || j * KT <= edge_to; };

  // two streams: 384 threads launched with 168 registers each; the row threads
  // (128 scores apiece) take 200, the last warpgroup 104
  if (warp >= kProducer) {
    if constexpr (NS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kProducer) {
      const int pieces = KT / a.box_t;
      const int pool_groups = a.num_pages * (a.page_size / 8);
      // The page of this lane's piece of tile j, read a tile ahead (clamped to
      // the table: the address is always good, and nothing waits for it here).
      auto page_of = [&](int j) {
        const int page = (key0 + j * KT + lane * a.box_t) >> a.page_shift;
        const size_t pi = (size_t)it.b * a.max_pages + min(page, a.max_pages - 1);
        return PGD_IN(pi, (size_t)a.B * a.max_pages, a.err) ? ld_global_s32(a.page_table + pi) : -1;
      };
      int phys = page_of(0);
      if (elect_one()) {
        const uint32_t qb = smem_u32(&bar.q_full);
        mbar_arrive_expect_tx(qb, (uint32_t)(ns * (D / 64) * a.tile_tok * a.G * 128));
        for (int s = 0; s < ns; ++s)
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(smem_u32(smem + s * C::kQBytes + c * (128 * 128)), &tmap_q, 0, h * a.G,
                        it.row0 + s * a.tile_tok, c, qb);
      }
      __syncwarp();
      int issued = 0;
      for (int r = 0; r < 2 * ntiles; ++r) {
        const int slot_r = r % NR;
        if ((r & 1) == 0) {
          // where the pieces of the tile are: a row group of the pool, or one
          // past it (zeros) where no query attends
          const int ptok = key0 + (r >> 1) * KT + lane * a.box_t;
          int coord = pool_groups;
          if (lane < pieces && ptok < it.hi && ptok + a.box_t > it.lo) {
            if (phys < 0 || phys >= a.num_pages) {
              raise_error(a.err, DECODE_ATTN_DEV_BAD_PAGE);
              atomicMin(&sh.bad_lo, ptok);
              atomicMax(&sh.bad_hi, ptok + a.box_t);
            } else {
              coord = (phys << (a.page_shift - 3)) + ((ptok & (a.page_size - 1)) >> 3);
            }
          }
          __syncwarp();
          if (lane < 16) sh.coord[lane] = coord;
          phys = page_of((r >> 1) + 1);
        }
        if (r >= NR) {
          int go = 1;
          if (lane == 0) {
            if (!mbar_wait_hot(smem_u32(&bar.empty[slot_r]), ((r / NR) & 1) ^ 1)) {
              sh.abort = 1;
              raise_error(a.err, DECODE_ATTN_DEV_TIMEOUT);
            }
            go = *(volatile int32_t*)&sh.abort ? 0 : 1;
          }
          if (!__shfl_sync(0xffffffffu, go, 0)) break;
        }
        __syncwarp();
        if (elect_one()) {
          // one lane issues every box: lanes in turn cost four times as much
          const uint32_t fb = smem_u32(&bar.full[slot_r]);
          mbar_arrive_expect_tx(fb, C::kTileBytes + (r == 0 ? a.stall_tx : 0));
          const CUtensorMap* map = (r & 1) ? &tmap_v : &tmap_k;
          uint32_t dst = smem_u32(ring + slot_r * C::kTileBytes);
          const uint32_t step = a.box_t * D * 2;
          for (int p = 0; p < pieces; p += 4) {
            const int4 c = *reinterpret_cast<const int4*>(&sh.coord[p]);
            tma_load_5d(dst, map, 0, 0, 0, c.x, h, fb);
            if (pieces > 1) tma_load_5d(dst + step, map, 0, 0, 0, c.y, h, fb);
            if (pieces > 2) {
              tma_load_5d(dst + 2 * step, map, 0, 0, 0, c.z, h, fb);
              tma_load_5d(dst + 3 * step, map, 0, 0, 0, c.w, h, fb);
            }
            dst += 4 * step;
          }
        }
        __syncwarp();
        issued = r + 1;
      }
      // this CTA's copies in flight have landed before the warp exits
      if (lane == 0) {
        mbar_wait_hot(smem_u32(&bar.q_full), 0);
        for (int r = max(0, issued - NR); r < issued; ++r)
          mbar_wait_hot(smem_u32(&bar.full[r % NR]), (r / NR) & 1);
      }
      return;
    }

    if (warp == kMma) {
      // One thread waits for and issues everything: the pace of this loop is
      // the pace of the tensor cores (with warp-wide waits and votes a unit
      // took 2000 cycles, of which the products need 1100).
      if (elect_one()) {
        if (NS == 2 && ns == 2)
          chunk_issue<D, E, NS>(bar, smem, sh.tmem, ntiles, edge, &sh.abort, a);
        else
          chunk_issue<D, E, 1>(bar, smem, sh.tmem, ntiles, edge, &sh.abort, a);
      }
      __syncwarp();
      named_barrier_sync(1, kOthers);  // every row has been read out
      tc_fence_after();
      tmem_free(sh.tmem, C::kTmemCols);
      return;
    }
    // the two warps that look over V's edge tiles
    int edges = 0;
    for (int j = 0; j < ntiles; ++j) {
      if (!edge(j)) continue;
      // (65536 tiles take a tenth of a second, a 2^30-position range all of 8
      // million: the first edge tile may be the last of them)
      if (!mbar_wait_long(smem_u32(&bar.v_edge), edges & 1, 1 + (ntiles >> 16))) sh.abort = 1;
      if (!__all_sync(0xffffffffu, !*(volatile int32_t*)&sh.abort)) break;
      const int k0 = key0 + j * KT;
      uint8_t* vt = ring + ((2 * j + 1) % NR) * C::kTileBytes;
      if (warp == kMma + 1 && lane == 0 && edges < C::kMaxEdges) sh.edge_key[edges] = k0;
      const int first = (warp - kMma - 1) * 32 + lane;
      uint4* tile = reinterpret_cast<uint4*>(vt);
      auto key_of = [&](int e) {  // groups of 8 keys, 1 KB per 64 dims
        return k0 + e / D * 8 + (e % 64) / 8;
      };
      // keys outside the range become zeros: in a pass of their own, or at
      // head_dim 256 in the next one (window of 1024 there 74.1 -> 72.4 us; the
      // prompt at 128, where few tiles have such keys, 350 -> 360)
      if (NS == 2 && (k0 < it.lo || k0 + KT > it.hi))
        for (int e = first; e < C::kTileBytes / 16; e += 64) {
          const int key = key_of(e);
          if (key < it.lo || key >= it.hi) tile[e] = make_uint4(0u, 0u, 0u, 0u);
        }
      // the largest magnitude of this thread's values, NaN if there is one
      uint32_t top = 0;
#pragma unroll 8
      for (int e = first; e < C::kTileBytes / 16; e += 64) {
        const uint4 v = tile[e];
        if (NS == 1 && (key_of(e) < it.lo || key_of(e) >= it.hi)) {
          tile[e] = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        top = max2_nan<E>(max2_nan<E>(top, v.x), max2_nan<E>(v.y, max2_nan<E>(v.z, v.w)));
      }
      if (wild2<E>(top) != 0u)
        for (int e = first; e < C::kTileBytes / 16; e += 64) {
          const uint4 v = tile[e];
          const uint4 m = make_uint4(wild2<E>(v.x), wild2<E>(v.y), wild2<E>(v.z), wild2<E>(v.w));
          if ((m.x | m.y | m.z | m.w) == 0u) continue;
          tile[e] = make_uint4(v.x & ~m.x, v.y & ~m.y, v.z & ~m.z, v.w & ~m.w);
          const int t = key_of(e) - k0;
          if (edges < C::kMaxEdges) atomicOr(&sh.wild[edges][t / 32], 1u << (t & 31));
          sh.wild_any = 1;
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar.v_clean));
      ++edges;
    }
    return;
  }

  // ---------------------------------------------------------- softmax rows
  if constexpr (NS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  const uint32_t tmem = sh.tmem, tmem_o = tmem + 2 * KT;  // O after the two S buffers
  const int s = warp >> 2;
  if (s < ns) {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int tok = a.by_group.div(row);
    const int te = min(it.t1, it.t0 + (s + 1) * a.tile_tok);  // one past the stream's tokens
    const int first_pos = it.p0 + s * a.tile_tok, last_pos = it.p0 + (te - it.t0) - 1;
    const int pos = first_pos + tok;  // this row's position
    const float scale = fabsf(a.scale_log2);
    float m = -INFINITY;
    uint64_t l2 = 0;  // two partial sums
    // log2 of the weight at which the reference is taken: in a row's first tile
    // (kLone: with one key far above its others), when it is taken again, and
    // what a tile may rise over that before
    constexpr bool kHalf = !std::is_same<E, __nv_bfloat16>::value;
    constexpr float kNext = kHalf ? 2.f : -40.f, kFirst = kHalf ? kNext : -16.f;
    constexpr float kLone = 12.f, kGrow = (kHalf ? 15.9f : 0.f) - kNext;
    // fp16: the largest tile maximum of the row beside the one that the reference
    // was taken at, less kNext.  The reference is taken down to it once it has a
    // weight below ntiles * 2^-10: the 2^-25 that each of ntiles * 128 weights
    // may lose are at most 2^-8 of what it brings otherwise.  (Rows of no token
    // never do.)
    [[maybe_unused]] float second =
        tok < a.tile_tok && it.t0 + s * a.tile_tok + tok < te ? -INFINITY : INFINITY;
    [[maybe_unused]] const float low = (float)min(21 - __clz(ntiles), 1) - kNext;
    bool ok = true;
    auto wait = [&](uint64_t* b, int parity) {
      if (ok && !mbar_wait_hot(smem_u32(b), parity)) {
        sh.abort = 1;
        raise_error(a.err, DECODE_ATTN_DEV_TIMEOUT);
        ok = false;
      }
    };
    for (int j = 0; j < ntiles; ++j) {
      const int u = j * ns + s, buf = u & 1;
      const uint32_t tm_s = tmem + buf * KT + lanes;
      wait(&bar.s_full[buf], (u >> 1) & 1);
      __syncwarp();
      tc_fence_after();
      float x[KT];
#pragma unroll
      for (int c = 0; c < KT; c += 32) tmem_ld32(x + c, tm_s + c);
      tmem_wait_ld();
      const int k0 = key0 + j * KT;
      float mult = scale;
      if (k0 + KT - 1 > first_pos || (a.window > 0 && k0 <= last_pos - a.window)) {
        // the edge of some row's range crosses the tile: a bit per key that
        // the row attends; scaled before the mask, so that a scale of 0
        // leaves the mask standing
        const int end = pos - k0 + 1;
        const int begin = a.window > 0 ? end - a.window : 0;
#pragma unroll
        for (int c = 0; c < KT; c += 32) {
          const uint32_t bits = low_bits(end - c) & ~low_bits(begin - c);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[c + i] = (bits & (1u << i)) ? x[c + i] * mult : -INFINITY;
        }
        mult = 1.f;
      }
      auto row_max = [&] {
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < KT; i += 4) {
          top[(i >> 2) & 1] = max3(top[(i >> 2) & 1], x[i], x[i + 1]);
          top[2 + ((i >> 2) & 1)] = max3(top[2 + ((i >> 2) & 1)], x[i + 2], x[i + 3]);
        }
        return fmaxf(max3(top[0], top[1], top[2]), top[3]) * mult;
      };
      // 64 keys' weights against the reference maximum, and their sum
      uint32_t w[32];
      auto weigh = [&](int part) {
        const float mu = m == -INFINITY ? 0.f : m;  // a row without a key so far
        const uint64_t mult2 = pair(mult, mult), nm2 = pair(-mu, -mu);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int k = part * 64 + 2 * i;
          const float2 e = unpair(fma2(pair(x[k], x[k + 1]), mult2, nm2));
          const float p0 = fast_exp2(e.x), p1 = fast_exp2(e.y);
          sum = add2(sum, pair(p0, p1));
          w[i] = ElemOps<E>::pack2(p0, p1);
        }
        return sum;
      };
      // The reference is moved only when a row's weights would leave their
      // range, and then of every row of the warp that has risen: the
      // accumulator is seldom rescaled.  So the first weights are made against
      // it while the tile's maximum is still being taken, and made again in the
      // tiles that move it.  (fp16, against weights of 1 first and 2^15 at most
      // that only move up, which lose small ones: prompt of 8192 351 us, as
      // before, with scores twice as sharp 360 -> 390, four times 418 -> 460, where
      // following every tile down takes 464 and 469; window of 1024 at head_dim
      // 256 71.7 -> 72.6.  Every row's first weight at 2^12: prompt 363.)
      if (j == 0) {
        m = row_max() - kFirst;
        if constexpr (kHalf) {
          // one key so far above the others that the sum is its weight, or next
          // to nothing: their weights get the range they need
          const float2 s2 = unpair(weigh(0));
          const float of = (s2.x + s2.y) * 0x1p-2f;  // in weights of the largest, 2^kNext
          if ((of < 0x1p-10f && m != -INFINITY) || (of > 0.999f && of < 1.f + 0x1p-10f))
            m -= kLone - kNext;
        }
      }
      uint64_t sum = weigh(0);
      const float mx = row_max() - kNext;
      bool grow = mx > m + kGrow, fall = false;
      if constexpr (kHalf) {
        if (j > 0) second = fmaxf(second, fminf(m, mx));
        fall = second < m + low && mx < second + kGrow;
      }
      if (__any_sync(0xffffffffu, grow || fall)) {
        if (fall) {  // past sums stay below 2^80: tiles 2^-64 of others may vanish
          const float2 lh = unpair(l2);
          if ((lh.x + lh.y) * fast_exp2(m - second) > 0x1p80f) {
            fall = false;
            second = m;
          }
        }
        // (a row without a key so far takes its first reference, which in bf16
        // moves no other row)
        const bool begins = m == -INFINITY;
        const bool all = kHalf || __any_sync(0xffffffffu, grow && !begins);
        const float ref = fall ? second : begins ? mx + (kNext - kFirst) : mx;
        grow = fall || (ref > m && (all || begins));
        const float alpha = grow ? fast_exp2(m - ref) : 1.f;
        if (grow) m = ref;
        if (j > 0) {  // (always so: the first tile's maximum is the reference)
          // O holds the products up to the unit before: rescale it in place
          wait(&bar.o_full[s], (j - 1) & 1);
          __syncwarp();
          tc_fence_after();
          l2 = mul2(l2, pair(alpha, alpha));
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            float o[16];
            const uint32_t at = tmem_o + s * D + lanes + c;
            tmem_ld16(o, at);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(at, reinterpret_cast<const uint32_t*>(o));
          }
        }
        sum = weigh(0);
      }
#pragma unroll
      for (int part = 0; part < C::kParts; ++part) {
        if (part > 0) sum = weigh(part);
        tmem_st32(tm_s + part * 32, w);
        l2 = add2(l2, sum);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar.p_full[buf][part]));
      }
    }
    wait(&bar.done[s], 0);
    const float2 lh = unpair(l2);
    const float l = lh.x + lh.y;
    ok = !*(volatile int32_t*)&sh.abort;
    tc_fence_after();
    // rows that attend a page outside the pool are zeroed
    const bool dead =
        !ok || (pos >= sh.bad_lo && (a.window <= 0 || pos - a.window + 1 < sh.bad_hi));
    // this row among the CTA's output rows, or -1
    const size_t row_base = (size_t)it.row0 * a.Hq + (size_t)h * a.G;
    int rel = (s * a.tile_tok + tok) * a.Hq + row - tok * a.G;
    if (tok >= a.tile_tok || it.t0 + s * a.tile_tok + tok >= te ||
        !PGD_IN(row_base + rel, (size_t)a.total * a.Hq, a.err))
      rel = -1;
    // V rows with a NaN or Inf reach the rows that attend them
    auto patch = [&](int c, float (&o)[32]) {
      for (int e = 0; e < C::kMaxEdges; ++e)
        for (int t = 0; t < KT; ++t) {
          const int key = sh.edge_key[e] + t;
          if (!(sh.wild[e][t / 32] >> (t & 31) & 1u) || key > pos ||
              (a.window > 0 && key <= pos - a.window))
            continue;
          const size_t pi = (size_t)it.b * a.max_pages + (key >> a.page_shift);
          const int phys = PGD_IN(pi, (size_t)a.B * a.max_pages, a.err) ? a.page_table[pi] : -1;
          if (phys < 0 || phys >= a.num_pages) continue;
          const uint32_t* v = static_cast<const uint32_t*>(a.v_pages) +
                              ((((size_t)phys << a.page_shift) + (key & (a.page_size - 1))) *
                                   a.Hkv + h) * (D / 2) + c / 2;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t w = __ldg(v + i);
            const float2 f = ElemOps<E>::unpack2(w & wild2<E>(w));
            o[2 * i] += f.x;
            o[2 * i + 1] += f.y;
          }
        }
    };
    // A thread holds a row, so its stores would touch 32 rows at a time; 32
    // columns of the warp's rows go through shared memory instead (this
    // stream's Q, which no product needs any more; 16-byte chunk c of row r at
    // c ^ (r & 7)) and out 4 lanes a row, 8 for a partial.
    const bool whole = it.shards == 1;
    const float inv = dead || l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    if (!whole && rel >= 0)
      a.ws_ml[(row_base + rel) * a.max_shards + shard] = make_float2(m, dead ? -1.f : l);
    uint4* stage = reinterpret_cast<uint4*>(smem + s * C::kQBytes) + (warp & 3) * 256;
    // bytes of 32 columns of a row: 64 of the output, 128 of a partial
    uint8_t* dst = whole ? static_cast<uint8_t*>(a.out) + row_base * D * 2
                         : reinterpret_cast<uint8_t*>(
                               a.ws_acc + (row_base * a.max_shards + shard) * D);
    const int row_bytes = whole ? D * 2 : a.max_shards * D * 4;
    const int per_row = whole ? 4 : 8;  // lanes of 16 bytes
    const int chunk = lane & (per_row - 1), first = whole ? lane >> 2 : lane >> 3;
    int rows4[4];  // the output rows that this lane stores to
#pragma unroll
    for (int i = 0; i < 4; ++i) rows4[i] = __shfl_sync(0xffffffffu, rel, (lane >> 2) + 8 * i);
    // (a small loop: a CTA runs it once, and most of its time would be the
    // fetching of unrolled code)
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tmem_ld32(o, tmem_o + s * D + lanes + c);
      tmem_wait_ld();
      if (sh.wild_any && rel >= 0) patch(c, o);
      if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x = o[8 * i + 2 * k] * inv, y = o[8 * i + 2 * k + 1] * inv;
            w[k] = inv == 0.f ? 0u : ElemOps<E>::pack2(x, y);
          }
          stage[lane * 8 + (i ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          stage[lane * 8 + (i ^ (lane & 7))] =
              make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                         __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
      }
      __syncwarp();
      uint8_t* at = dst + (whole ? c * 2 : c * 4) + chunk * 16;
      if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = stage[(first + 8 * i) * 8 + (chunk ^ first)];
          if (rows4[i] >= 0) *reinterpret_cast<uint4*>(at + (size_t)rows4[i] * row_bytes) = v;
        }
      } else {
#pragma unroll 4
        for (int r = first; r < 32; r += 4) {
          const uint4 v = stage[r * 8 + (chunk ^ (r & 7))];
          const int to = __shfl_sync(0xffffffffu, rel, r);
          if (to >= 0) *reinterpret_cast<uint4*>(at + (size_t)to * row_bytes) = v;
        }
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  named_barrier_sync(1, kOthers);
}

// Merges the shards' partials of every row of a split plan, in ascending
// shard order (same bits every run): one warp per row, launched as a
// programmatic dependent of the attention kernel.
constexpr int kChunkCombineRows = 8;

template <int D, class E>
__global__ void __launch_bounds__(kChunkCombineRows * 32)
    chunk_combine_kernel(const ChunkArgs a) {
  constexpr int KT = ChunkCfg<D>::kKeys;
  constexpr int V = D / 32;  // dims per lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = a.item_tok * a.G;
  const int blocks = (rows + kChunkCombineRows - 1) / kChunkCombineRows;
  const int h = (blockIdx.x / blocks) % a.Hkv;
  const int slot = blockIdx.x / (blocks * a.Hkv);
  const int r = (blockIdx.x % blocks) * kChunkCombineRows + warp;
  // (the lengths and offsets were complete before the attention kernel began)
  const ChunkItem it = chunk_item<KT>(a, slot, lane);
  const int tok = r / a.G, g = r % a.G;
  grid_dependency_wait();
  grid_launch_dependents();
  if (!it.any || it.shards < 2 || r >= rows || it.t0 + tok >= it.t1) return;
  const size_t row = (size_t)(it.row0 + tok) * a.Hq + (size_t)h * a.G + g;
  if (!PGD_IN(row, (size_t)a.total * a.Hq, a.err)) return;
  const float2* ml = a.ws_ml + row * a.max_shards;
  const float* acc = a.ws_acc + row * a.max_shards * D + lane * V;
  float M = -INFINITY;
  bool dead = false;
  for (int s0 = 0; s0 < it.shards; s0 += 32) {
    const float2 v = s0 + lane < it.shards ? __ldcg(ml + s0 + lane) : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, v.x);
    dead |= v.y < 0.f;
  }
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
  dead = __any_sync(0xffffffffu, dead);
  float o[V], L = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  if (!dead && M != -INFINITY) {
#pragma unroll 8
    for (int s = 0; s < it.shards; ++s) {
      const float2 v = __ldcg(ml + s);
      const float c = fast_exp2(v.x - M);
      float x[V];
      if constexpr (V == 2) {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(acc + (size_t)s * D));
        x[0] = f.x;
        x[1] = f.y;
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(acc + (size_t)s * D + i));
          x[i] = f.x;
          x[i + 1] = f.y;
          x[i + 2] = f.z;
          x[i + 3] = f.w;
        }
      }
      L = __fmaf_rn(c, v.y, L);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = __fmaf_rn(c, x[i], o[i]);
    }
  }
  const float inv = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i)
    w[i] = inv == 0.f ? 0u : ElemOps<E>::pack2(o[2 * i] * inv, o[2 * i + 1] * inv);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D + lane * V);
  if constexpr (V == 2) {
    dst[0] = w[0];
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace pgd
