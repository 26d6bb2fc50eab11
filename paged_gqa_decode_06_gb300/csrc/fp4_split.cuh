// Decode attention over a 4-bit cache (e2m1.cuh: e2m1 codes, an e4m3 scale per
// 16 dims, an fp32 scale per (position, KV head) row of K and of V): out =
// sum_t p_t vs_t vb_t vc_t with scores scale * ks_t * (q . kb_t kc_t).
//
// One CTA per (shard, KV head or several, sequence); the products are mma.sync
// with the tokens on M and the group's query rows on N, the row scales enter in
// fp32 with the scores and the weights, and the merges are those of the 8-bit
// kernel (quant_split.cuh).  What differs:
//  * Every warp is its own pipeline: 32 positions of one head at a time, whose
//    codes and scales it copies itself (cp.async, 16 bytes a lane) two units
//    ahead, K as soon as K is used up and V after V.  No warp waits for another
//    until the end, and no wait can hang.  (A producer warp with TMA boxes, as for 8
//    bits, brought a stage in about 0.9 us whatever it held, and a page's piece of one
//    head is 1 KB: four sequences of 131072 positions took 199 us.)
//  * Turning codes into fragments bounds the kernel, and of that the ALU's
//    half-rate instructions (conversions, permutations).  A byte holds two
//    neighbouring dims of one token and is converted as it is, one instruction for
//    two values: for K they are neighbours of the contraction (four dims of a
//    lane in the place of two and two; q is loaded in the same order).  For V the
//    contraction runs over (token, dim parity): a row of the product's 16 is a
//    pair of dims, a token's weight w takes the places (w, 0) for the even dims
//    and (0, w) for the odd ones, so that no nibble has to move to its
//    neighbour token's.  Up to four query rows leave half of the eight columns
//    free, which then take the odd dims at no cost; with more rows the odd dims
//    are products of their own.
//  * A code times its block's scale is exact in fp16 (two significant bits times
//    four, between 2^-10 and 2688).  The scales of a unit are made ready once, a
//    position a lane, and read back by the lanes that meet them.  Up to four
//    query rows K's codes go into the products as they are: of the eight columns
//    four take the first block of each 32 dims and four the second, and their
//    sums are scaled in fp32 (a quarter of the multiplications).  The two halves
//    of a score lie two lanes apart; of the lanes that add them up one half takes
//    the unit's first 16 positions on and the other the last 16.
//  * The weights are rounded to fp16 once, the largest 2^14: 11 bits down to 2^-28
//    of it, nothing below 2^-39; the sum keeps them unrounded.  Against 64 bits an
//    fp16 result is off by 2.1e-4 to 2.5e-4 (rel. L2), by its own rounding alone 2.1e-4,
//    a bf16 one by its rounding.  (The 8-bit kernel's second product for the remainder
//    takes the products that the parities need here.)
//  * A block without a number among its scales (NaN) is the only way that codes
//    reach a product as no number, so a position outside a row's range is
//    cleared by its V blocks' scales alone.
//
// Measured (GB300): four sequences of 131072 positions, 64 heads over 8, 132.5 us (4.8
// TB/s; the 8-bit cache 187), 64 of U[1, 8192] with 32 heads 84 us (3.9 TB/s; 111),
// 64 of 8192 128.5 us, one of 3060 8.7 us; 16 of 8192 with 16 rows a head 69 us (2.3 TB/s).
// No unit is at its limit in the long step: 340 instructions for 16 positions of a head (64
// conversions, 64 scalings, 24 products, 60 for the copies, 70 for the softmax) take 60 %
// of the slots that 16 warps an SM have; the ALU is busy 44 % of the time, the tensor
// cores 34 %, DRAM 60 %.  With the copies left out it takes 113 us, without the softmax
// 116, without either product 111.  Uneven lengths are short of balance beside that: 64
// of 8192 reach 4960 GB/s, of U[1, 8192] 3860.
#pragma once

#include "e2m1.cuh"
#include "quant_split.cuh"

namespace pgd {

struct Fp4Args {
  SplitArgs s;               // as for the 16-bit split kernel; G and Hkv of HC heads as one
  const uint8_t* codes[2];   // K, V [P][PS][Hkv][D / 2]
  const float* scales[2];    // [P][Hkv][PS]
  const uint8_t* blocks[2];  // [P][Hkv][PS][D / 16]
  int32_t G1, heads;         // query heads per KV head, KV heads
};

constexpr int kUnit = 32;  // positions that a warp takes at a time

// NQ: query rows of a head that the kernel has room for, 4, 8 or 16; HC: heads
// of a CTA, each with its share of the warps.
template <int D, int NQ, int HC>
struct Fp4Cfg {
  // Small CTAs: while one finds its pages or folds, the SM's others go on (64
  // sequences of 8192: 127 us with four of 4 warps, 137 with two of 8).  What 16
  // warps leave is 128 registers; 16 rows and head_dim 256 need more.
  static constexpr int kWarps = 4;
  static constexpr int kCtas = D == 256 ? 2 : NQ == 16 ? 3 : 4;  // of an SM
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kWidth = D / 2;                 // bytes of a position's codes
  static constexpr int kBlocks = D / 16;               // block scales of a position
  static constexpr int kCodeBytes = kUnit * kWidth;    // K or V codes of a unit
  static constexpr int kSlotBytes = 2 * (kCodeBytes + kUnit * kBlocks + kUnit * 4);
  // a unit's scales as the lanes read them: block scales of K (fp16, or with up to
  // four rows fp32 times the row's) and of V (fp16), and (K scale, V scale, its
  // log2) per position
  static constexpr int kReadyK = kUnit * kBlocks * (NQ == 4 ? 4 : 2);
  static constexpr int kReadyV = kUnit * kBlocks * 2;
  // (V's take K's place: they are made after the scores)
  static constexpr int kReadyBytes = kReadyK + kUnit * 16;
  static_assert(kReadyV <= kReadyK, "");
  static constexpr int kWarpBytes = 2 * kSlotBytes + kReadyBytes;
  static constexpr int kRingBytes = kWarps * kWarpBytes;
  // the ring, which also holds the warps' states for the fold and what the merge
  // stages of a group's rows
  static constexpr int kMergeBytes = merge_smem_bytes(NQ * HC < 16 ? NQ * HC : 16);
  static constexpr int kSmemBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  // static shared memory and what is left of a CTA's share of the SM's 228 KB
  // for a cluster's receive buffer
  static constexpr int kTableBytes = kMaxPieces * 4 + 3 * 1024;
  static constexpr int kRecvRoom = 228 * 1024 / kCtas - 1024 - kSmemBytes - kTableBytes;
  static_assert(kWarps % HC == 0 && kWarpBytes % 128 == 0, "");
};

// Byte offset of (token t, 16-byte chunk c) in a tile of codes, rows of W bytes
// with 16-byte chunks permuted so that eight rows' chunk c meet distinct banks.
template <int W>
__device__ __forceinline__ uint32_t fp4_offset(int t, int c) {
  static_assert(W == 32 || W == 64 || W == 128, "");
  const int key = W == 128 ? (t & 7) : W == 64 ? ((t >> 1) & 3) : ((t >> 2) & 1);
  return (uint32_t)(t * W + ((c ^ key) << 4));
}

// Blocks of a row's dims that a NaN reaches by a position that only some rows
// attend, kept beside the accumulators: the products would carry it to all.
template <int ROWS>
struct Fp4Wild {
  uint32_t bits[ROWS];
  int32_t any;
};

__device__ __forceinline__ __half2 as_half2(uint32_t a) {
  return *reinterpret_cast<const __half2*>(&a);
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(as_half2(a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int OFF>
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0 + %2], [%1], 16;" ::"r"(dst), "l"(src),
               "n"(OFF)
               : "memory");
}
// The same where `in`, without a branch.
template <int OFF>
__device__ __forceinline__ void cp_async_16_if(bool in, uint32_t dst, const void* src) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\t"
      "@p cp.async.cg.shared.global.L2::256B [%0 + %2], [%1], 16;\n\t}" ::"r"(dst),
      "l"(src), "n"(OFF), "r"((int)in)
      : "memory");
}
template <int OFF>
__device__ __forceinline__ void ldmatrix_x4_at(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}
template <int OFF>
__device__ __forceinline__ void ldmatrix_x4_trans_at(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}
// A value that the compiler keeps in its register and does not work out again.
__device__ __forceinline__ void keep(uint32_t& x) { asm volatile("" : "+r"(x)); }

// Calls f(std::integral_constant<int, i>) for i in [0, N).
template <int N, class F>
__device__ __forceinline__ void static_for(F f) {
  if constexpr (N > 0) {
    static_for<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's copies of its units.  What a lane copies is the same in every unit but
// for where the unit's pages lie, so a unit costs a lane one look-up in the table
// of pieces, whose results the lanes exchange, and one multiply-add per copy
// (worked out anew the addresses took 126 of 414 instructions for 16 positions, and the
// long step 182 us, not 157).  Pieces that no row attends point at the pool's first rows: what
// they bring is masked with the rest.
template <int D>
struct Fp4Loader {
  using C = Fp4Cfg<D, 4, 1>;
  // a slot: K codes, V codes, K blocks, V blocks, K rows, V rows
  static constexpr int kV = C::kCodeBytes, kKb = 2 * C::kCodeBytes,
                       kVb = kKb + kUnit * C::kBlocks, kKr = kVb + kUnit * C::kBlocks,
                       kVr = kKr + kUnit * 4;
  // codes: a copy brings 32 chunks of 16 bytes, kRows positions (16, 8 or 4)
  static constexpr int kChunks = C::kWidth / 16, kRows = 32 / kChunks, kCopies = kUnit / kRows;
  // scales: the first kBlockLanes lanes a block's copy of kPer positions each, and
  // (of the rest, or at head_dim 256 in a copy of its own) 16 lanes the row scales
  // of 4, K's and then V's
  static constexpr int kBlockLanes = 2 * C::kBlocks, kPer = 16 / C::kBlocks;
  static constexpr bool kOne = kBlockLanes + 16 <= 32;

  const Fp4Args& a;
  const int32_t* coord;         // first pool row of each piece of 2^box_shift positions
  const uint8_t* codes_at[2];   // this lane's chunk and row of a copy, in the pools' first rows
  const uint8_t* scale_at;      // this lane's scales there (kOne: of K's blocks, or of rows)
  const uint8_t* row_at;        // its row scales there
  int64_t block_step;           // from K's to V's
  uint32_t code_to, scale_to;   // the lane's places in a slot
  uint32_t row_bytes, page_bytes, scale_size, row_page_bytes;
  int box_shift, page_shift, lane, lane_row;
  int t_scale, t_row;  // positions of this lane's scale copies
  bool has_block, has_scale, has_row;
  // of the unit whose K is on its way: pool rows of the code copies (of two, where
  // each brings 4 positions), the block scales
  static constexpr int kHeld = kCopies < 4 ? kCopies : 4;
  int32_t rows[kHeld];
  const uint8_t* from;

  __device__ __forceinline__ Fp4Loader(const Fp4Args& args, const int32_t* coord_s, int lane_id,
                                       int head, int shift)
      : a(args), coord(coord_s), box_shift(shift), page_shift(args.s.page_shift), lane(lane_id) {
    const int chunk = lane % kChunks;
    lane_row = lane / kChunks;
    row_bytes = (uint32_t)a.heads * C::kWidth;
    code_to = fp4_offset<C::kWidth>(lane_row, chunk);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      codes_at[kv] =
          a.codes[kv] + (size_t)lane_row * row_bytes + (size_t)head * C::kWidth + chunk * 16;
    block_step = a.blocks[1] - a.blocks[0];
    const size_t head_at = (size_t)head << page_shift;
    const int r = kOne ? lane - kBlockLanes : lane;
    has_block = lane < kBlockLanes;
    has_row = r >= 0 && r < 16;
    has_scale = has_block || (kOne && has_row);
    t_row = 4 * (r & 7);
    row_at = reinterpret_cast<const uint8_t*>(a.scales[(r >> 3) & 1] + head_at);
    const bool rows_here = kOne && !has_block;
    t_scale = rows_here ? t_row : lane * kPer & (kUnit - 1);
    scale_size = rows_here ? 4 : C::kBlocks;
    scale_to = rows_here ? kKr + 16 * r : kKb + 16 * lane;
    scale_at = rows_here ? row_at : a.blocks[0] + head_at * C::kBlocks;
    // a page's scales lie heads apart, so its index is its pool row's and as much
    // for the pages before it
    const uint32_t page_step = (uint32_t)(a.heads - 1) << page_shift;
    page_bytes = page_step * scale_size;
    row_page_bytes = page_step * 4;
  }

  __device__ __forceinline__ bool ok(int row, int count) const {
    return PGD_IN(row + count - 1, (uint64_t)a.s.num_pages * a.s.page_size, a.s.err);
  }
  __device__ __forceinline__ void codes(uint32_t to, const uint8_t* at) const {
    static_for<kCopies>([&](auto copy) {
      constexpr int k = decltype(copy)::value;
      // (rows of 128 bytes: a copy is half the period of their chunks' order)
      const uint32_t place = C::kWidth == 128 && (k & 1) ? code_to ^ 64u : code_to;
      const int row = kRows == 4 ? rows[k / 2] + 4 * (k & 1) : rows[k];
      if (ok(row + lane_row, 1))
        cp_async_16<k * kRows * C::kWidth>(to + place, at + (int64_t)row * (int32_t)row_bytes);
    });
  }
  // K of unit u into the slot at `to`
  __device__ __forceinline__ void k(uint32_t to, int u) {
    // the pool row of positions 8 (lane % 4) .. of the unit (pieces have 8 or more)
    const int p = u * kUnit + 8 * (lane & 3);
    const int mine = coord[p >> box_shift] + (p & ((1 << box_shift) - 1));
    auto row_of = [&](int t) { return __shfl_sync(0xffffffffu, mine, t >> 3) + (t & 7); };
    // (at head_dim 64 a copy spans 16 positions, whose upper 8 have a row of their own)
    const int upper = kRows == 16 ? lane_row & 8 : 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) rows[i] = row_of(i * (kUnit / kHeld) + upper) - upper;
    codes(to, codes_at[0]);
    const int row = row_of(t_scale);
    from = scale_at + (uint64_t)(uint32_t)(row >> page_shift) * page_bytes +
           (uint64_t)(uint32_t)row * scale_size;
    cp_async_16_if<0>(has_scale && ok(row, kPer), to + scale_to, from);
    if constexpr (!kOne) {
      const int r = row_of(t_row);
      const uint8_t* at = row_at + (uint64_t)(uint32_t)(r >> page_shift) * row_page_bytes +
                          (uint64_t)(uint32_t)r * 4;
      cp_async_16_if<kKr>(has_row && ok(r, 4), to + 16 * lane, at);
    }
    cp_async_commit();
  }
  // V of the unit that k() brought last, into the same slot
  __device__ __forceinline__ void v(uint32_t to) const {
    codes(to + kV, codes_at[1]);
    cp_async_16_if<kVb - kKb>(has_block, to + scale_to, from + block_step);
    cp_async_commit();
  }
};

// One position's block scales as fp16, the chunks' (of 32 dims) first blocks and
// then their second ones.
template <int NB>
__device__ __forceinline__ void ready_scales(const uint32_t (&w)[NB / 4], uint8_t* to) {
  uint32_t h[NB / 2];
  if constexpr (NB == 4) {
    const uint32_t x = __byte_perm(w[0], 0u, 0x3120);
    h[0] = e4m3_to_half2(x & 0xffffu);
    h[1] = e4m3_to_half2(x >> 16);
    *reinterpret_cast<uint2*>(to) = make_uint2(h[0], h[1]);
  } else {
#pragma unroll
    for (int k = 0; k < NB / 8; ++k) {
      const uint32_t first = __byte_perm(w[2 * k], w[2 * k + 1], 0x6420);
      const uint32_t second = __byte_perm(w[2 * k], w[2 * k + 1], 0x7531);
      h[2 * k] = e4m3_to_half2(first & 0xffffu);
      h[2 * k + 1] = e4m3_to_half2(first >> 16);
      h[NB / 4 + 2 * k] = e4m3_to_half2(second & 0xffffu);
      h[NB / 4 + 2 * k + 1] = e4m3_to_half2(second >> 16);
    }
#pragma unroll
    for (int k = 0; k < NB / 8; ++k)
      reinterpret_cast<uint4*>(to)[k] =
          make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
  }
}
// Of those the chunks' first or second ones (NB bytes on), two chunks to a register.
template <int NB>
__device__ __forceinline__ void read_scales(const uint8_t* at, __half2 (&s)[NB / 4]) {
  if constexpr (NB == 4) {
    s[0] = as_half2(*reinterpret_cast<const uint32_t*>(at));
  } else if constexpr (NB == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    s[0] = as_half2(v.x), s[1] = as_half2(v.y);
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    s[0] = as_half2(v.x), s[1] = as_half2(v.y), s[2] = as_half2(v.z), s[3] = as_half2(v.w);
  }
}
template <int NB>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[NB / 4]) {
  if constexpr (NB == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  } else if constexpr (NB == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// Up to four rows: one position's block scales as fp32, times f, in the same order.
template <int NB>
__device__ __forceinline__ void ready_scales_f32(const uint32_t (&w)[NB / 4], float f,
                                                 uint8_t* to) {
  float4* out = reinterpret_cast<float4*>(to);
  auto pair = [&](uint32_t two) {
    const float2 x = ElemOps<__half>::unpack2(e4m3_to_half2(two));
    return make_float2(x.x * f, x.y * f);
  };
  if constexpr (NB == 4) {
    const uint32_t x = __byte_perm(w[0], 0u, 0x3120);
    const float2 first = pair(x & 0xffffu), second = pair(x >> 16);
    out[0] = make_float4(first.x, first.y, second.x, second.y);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < NB / 8; ++k) {
        const uint32_t x = __byte_perm(w[2 * k], w[2 * k + 1], h ? 0x7531 : 0x6420);
        const float2 lo = pair(x & 0xffffu), hi = pair(x >> 16);
        out[h * (NB / 8) + k] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
  }
}

// The scores of a unit with up to four query rows, scaled, for half of its
// positions a lane: sc[i][e] of position 16 (tig >> 1) + gid + 8 i and row (2 tig
// + e) % 4.  Columns 0 to 3 of the products hold the rows' dims of the first
// blocks, 4 to 7 those of the second (qf is zero elsewhere).
template <int D>
__device__ __forceinline__ void fp4_scores_4(uint32_t kt, const uint8_t* ready, bool upper,
                                             const uint32_t (&qf)[D / 16][2],
                                             float (&sc)[2][2]) {
  constexpr int NB = D / 16, W = D / 2, kChunks = D / 32;
  float part[2][4];
  static_for<2>([&](auto half) {
    constexpr int b = decltype(half)::value;
    float s[2][kChunks];  // of tokens gid and gid + 8, the lane's block of each chunk
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* at = ready + (16 * b + 8 * i) * NB * 4;
      if constexpr (kChunks == 2) {
        const float2 v = *reinterpret_cast<const float2*>(at);
        s[i][0] = v.x, s[i][1] = v.y;
      } else {
#pragma unroll
        for (int k = 0; k < kChunks / 4; ++k) {
          const float4 v = reinterpret_cast<const float4*>(at)[k];
          s[i][4 * k] = v.x, s[i][4 * k + 1] = v.y;
          s[i][4 * k + 2] = v.z, s[i][4 * k + 3] = v.w;
        }
      }
    }
#pragma unroll
    for (int cp = 0; cp < kChunks / 2; ++cp) {
      uint32_t r[4];  // (tokens 0-7, 8-15) x (chunks 2 cp, 2 cp + 1): eight dims per register
      ldmatrix_x4_at<16 * b * W>(r, kt ^ (32 * cp));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 2 * cp + i;
        uint32_t x[4], y[4];
        e2m1_to_half8(r[2 * i], x);
        e2m1_to_half8(r[2 * i + 1], y);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t af[4] = {x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1]};
          ElemOps<__half>::mma(o, af, qf[2 * c + k][0], qf[2 * c + k][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          part[b][e] = c == 0 ? o[e] * s[e >> 1][c] : fmaf(o[e], s[e >> 1][c], part[b][e]);
      }
    }
  });
  // the other blocks' sums come from the lane that goes on with the other positions
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float give = upper ? part[0][2 * i + e] : part[1][2 * i + e];
      const float keep = upper ? part[1][2 * i + e] : part[0][2 * i + e];
      sc[i][e] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
}

// The online softmax of those: the weights in the places that fp4_values gives
// them, wb[g] of the unit's 8 tokens 8 g...  rows: (-, V scale, its log2) per
// position, from the lane's first on; scale: the rows' factor (kFactor; else 1).
template <bool kInside, bool kFactor>
__device__ __forceinline__ bool fp4_weights_4(const float (&sc)[2][2], const float4* rows,
                                              const float (&scale)[2], const int2* col_s,
                                              int tok0, int lane, uint32_t sel,
                                              float (&m_run)[2], float (&l_sum)[2],
                                              float (&down)[2], uint32_t (&wb)[4][2]) {
  const int gid = lane >> 2, tig = lane & 3;
  const int first = 8 * (tig & 2) + gid;  // this lane's positions: first, first + 8
  float4 row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) row[i] = rows[8 * i];
  bool rescale = false;
  float w[2][2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float sv[2], mx = -INFINITY;
    bool in[2];
    int2 range = make_int2(0, 0);
    if constexpr (!kInside) range = col_s[(2 * tig + e) & 3];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sv[i] = kFactor ? sc[i][e] * scale[e] : sc[i][e];
      const int t = tok0 + first + 8 * i;
      in[i] = kInside || (t >= range.x && t < range.y);
      mx = fmaxf(mx, in[i] ? sv[i] + row[i].z : -INFINITY);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    const float m_new = fmaxf(m_run[e], mx);
    down[e] = (m_new == -INFINITY) ? 0.f : m_run[e] - m_new;
    rescale |= down[e] != 0.f;
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float p = in[i] ? fast_exp2(sv[i] - m_new) : 0.f;
      l += p;
      w[i][e] = in[i] ? p * row[i].y : 0.f;
    }
    l_sum[e] = l;
    m_run[e] = m_new;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // transposed: tokens 2 tig, 2 tig + 1 of row gid % 4, in the first 16 positions
    // (gid < 4) or the last; the others' from the lane that has them
    const uint32_t x = movmatrix_trans(ElemOps<__half>::pack2(w[i][0], w[i][1]));
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, 16);
    // (the selectors of the even or the odd dims' places, the second token's 16 bits on)
    const bool odd = gid & 4;
    const uint32_t lo = odd ? y : x, hi = odd ? x : y;
    wb[i][0] = __byte_perm(lo, 0u, sel);
    wb[i][1] = __byte_perm(lo, 0u, sel >> 16);
    wb[2 + i][0] = __byte_perm(hi, 0u, sel);
    wb[2 + i][1] = __byte_perm(hi, 0u, sel >> 16);
  }
  return rescale;
}

// Scores of a unit: sc[b] of the positions 16 b + gid (and + 8), columns 2 tig,
// 2 tig + 1.
template <int D, int NJ>
__device__ __forceinline__ void fp4_scores(uint32_t kt, const uint8_t* ready,
                                           const uint32_t (&qf)[NJ][D / 16][2],
                                           float (&sc)[2][NJ][4]) {
  constexpr int NB = D / 16, W = D / 2, kChunks = D / 32;
  static_for<2>([&](auto half) {
    constexpr int b = decltype(half)::value;
#pragma unroll
    for (int j = 0; j < NJ; ++j) sc[b][j][0] = sc[b][j][1] = sc[b][j][2] = sc[b][j][3] = 0.f;
    // this lane's two tokens, gid and gid + 8, and of a chunk the block of dims 8 tig..
    __half2 s[2][NB / 4];
    read_scales<NB>(ready + 16 * b * 2 * NB, s[0]);
    read_scales<NB>(ready + (16 * b + 8) * 2 * NB, s[1]);
#pragma unroll
    for (int cp = 0; cp < kChunks / 2; ++cp) {
      uint32_t r[4];  // (tokens 0-7, 8-15) x (chunks 2 cp, 2 cp + 1): eight dims per register
      ldmatrix_x4_at<16 * b * W>(r, kt ^ (32 * cp));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 s0 = i ? __high2half2(s[0][cp]) : __low2half2(s[0][cp]);
        const __half2 s1 = i ? __high2half2(s[1][cp]) : __low2half2(s[1][cp]);
        uint32_t a[4], c[4];
        e2m1_to_half8(r[2 * i], a);
        e2m1_to_half8(r[2 * i + 1], c);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t af[4] = {hmul2_bits(a[2 * k], s0), hmul2_bits(c[2 * k], s1),
                                  hmul2_bits(a[2 * k + 1], s0), hmul2_bits(c[2 * k + 1], s1)};
          const int ks = 2 * (2 * cp + i) + k;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            ElemOps<__half>::mma(sc[b][j], af, qf[j][ks][0], qf[j][ks][1]);
        }
      }
    }
  });
}

// The online softmax of a unit's scores: weights (with V's row scales) as
// transposed fp16 pairs, tokens 2 tig and 2 tig + 1 of column gid in each 8.
// rows: (K scale times the softmax's, V scale, its log2) per position, from the
// lane's first on; scale: the
// columns' factor (kFactor; else 1).  kInside: every column attends all
// positions, else those of col_s.
template <int NQ, int NJ, bool kInside, bool kFactor>
__device__ __forceinline__ bool fp4_weights(const float (&sc)[2][NJ][4], const float4* rows,
                                            const float (&scale)[NJ][2], const int2* col_s,
                                            int tok0, int lane, float (&m_run)[NJ][2],
                                            float (&l_sum)[NJ][2], float (&down)[NJ][2],
                                            uint32_t (&wt)[4][NJ]) {
  const int gid = lane >> 2, tig = lane & 3;
  float4 row[4];  // this lane's positions: gid + 8 i
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = rows[8 * i];
  bool rescale = false;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    float w[4][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sv[4], mx = -INFINITY;
      bool in[4];
      int2 range = make_int2(0, 0);
      if constexpr (!kInside) range = col_s[(8 * j + 2 * tig + e) % NQ];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sv[i] = sc[i >> 1][j][e + 2 * (i & 1)] * row[i].x;
        if constexpr (kFactor) sv[i] *= scale[j][e];
        const int t = tok0 + gid + 8 * i;
        in[i] = kInside || (t >= range.x && t < range.y);
        mx = fmaxf(mx, in[i] ? sv[i] + row[i].z : -INFINITY);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float m_new = fmaxf(m_run[j][e], mx);
      down[j][e] = (m_new == -INFINITY) ? 0.f : m_run[j][e] - m_new;
      rescale |= down[j][e] != 0.f;
      float l = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = in[i] ? fast_exp2(sv[i] - m_new) : 0.f;
        l += p;
        w[i][e] = in[i] ? p * row[i].y : 0.f;
      }
      l_sum[j][e] = l;
      m_run[j][e] = m_new;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      wt[i][j] = movmatrix_trans(ElemOps<__half>::pack2(w[i][0], w[i][1]));
  }
  return rescale;
}

// out^T += V^T . W^T, 8 tokens at a time: rows gid and gid + 8 of chunk c are the
// dims 32 c + 4 gid (+ 1) and the next two; the contraction's places 2 tig, 2 tig
// + 1 are the even and odd dim of token 2 tig, 2 tig + 8 and + 9 those of token
// 2 tig + 1.
template <int D, int NQ, int NJ, int NP>
__device__ __forceinline__ void fp4_values(uint32_t vt, const uint8_t* ready,
                                           const uint32_t (&wt)[4][NQ == 4 ? 2 : NJ],
                                           float (&acc)[D / 32][NJ][NP][4]) {
  constexpr int NB = D / 16, W = D / 2, kChunks = D / 32;
  // matrices of a load: four chunks of 8 tokens, or (head_dim 64) two of 16
  constexpr bool kFour = kChunks >= 4;
  uint32_t r[4];  // four dims of tokens 2 tig and 2 tig + 1 of a chunk each
  static_for<4>([&](auto group) {
    constexpr int g = decltype(group)::value;
    __half2 s[2][NB / 4];
    read_scales<NB>(ready + 8 * g * 2 * NB, s[0]);
    read_scales<NB>(ready + (8 * g + 1) * 2 * NB, s[1]);
    uint32_t wb[NJ][NP][2];  // the weights in their places
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if constexpr (NQ == 4) {
        wb[j][0][0] = wt[g][0];
        wb[j][0][1] = wt[g][1];
      } else {
        const uint32_t x = wt[g][j];
        wb[j][0][0] = x & 0xffffu;
        wb[j][0][1] = x >> 16;
        wb[j][NP - 1][0] = x << 16;
        wb[j][NP - 1][1] = x & 0xffff0000u;
      }
    }
#pragma unroll
    for (int c0 = 0; c0 < kChunks; c0 += 4) {
      if constexpr (kFour || g % 2 == 0) ldmatrix_x4_trans_at<8 * g * W>(r, vt ^ (16 * c0));
#pragma unroll
      for (int i = 0; i < (kFour ? 4 : 2); ++i) {
        const int c = c0 + i;
        const __half2 s0 = c & 1 ? __high2half2(s[0][c >> 1]) : __low2half2(s[0][c >> 1]);
        const __half2 s1 = c & 1 ? __high2half2(s[1][c >> 1]) : __low2half2(s[1][c >> 1]);
        uint32_t a[4];
        e2m1_to_half8(r[kFour ? i : 2 * (g & 1) + i], a);
        const uint32_t af[4] = {hmul2_bits(a[0], s0), hmul2_bits(a[1], s0),
                                hmul2_bits(a[2], s1), hmul2_bits(a[3], s1)};
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int p = 0; p < NP; ++p)
            ElemOps<__half>::mma(acc[c][j][p], af, wb[j][p][0], wb[j][p][1]);
      }
    }
  });
}

// A row of q as fp16 fragments, 8 consecutive dims per lane and 32-dim chunk;
// returns the power of two taken out of a bf16 row (as load_q_row).
template <int D, class E>
__device__ __forceinline__ float fp4_load_q_row(const uint16_t* row, bool live, int tig,
                                                uint32_t (&qf)[D / 16][2]) {
  uint4 raw[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    raw[c] = live ? *reinterpret_cast<const uint4*>(row + c * 32 + 8 * tig)
                  : make_uint4(0u, 0u, 0u, 0u);
  float amax = 0.f;
  if constexpr (!std::is_same<E, __half>::value) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      for (uint32_t w : {raw[c].x, raw[c].y, raw[c].z, raw[c].w}) {
        const float2 f = ElemOps<E>::unpack2(w);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  }
  // 2^(E - 14) of the row's largest value, 2^E at least, as for the 8-bit cache
  const uint32_t e = min(max((__float_as_uint(amax) >> 23) & 255u, 27u), 253u) - 14u;
  const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t& to = qf[2 * c + (i >> 1)][i & 1];
      if constexpr (std::is_same<E, __half>::value) {
        to = w[i];
      } else {
        const float2 f = ElemOps<E>::unpack2(w[i]);
        to = ElemOps<__half>::pack2(f.x * inv, f.y * inv);
      }
    }
  }
  return std::is_same<E, __half>::value ? 1.f : __uint_as_float(e << 23);
}

// CL: a cluster plan, as in split_mma_body.
template <int D, int NQ, class E, bool CL, int HC>
__global__ void __launch_bounds__(Fp4Cfg<D, NQ, HC>::kThreads, Fp4Cfg<D, NQ, HC>::kCtas)
    fp4_split_kernel(const Fp4Args fa) {
  using C = Fp4Cfg<D, NQ, HC>;
  using Loader = Fp4Loader<D>;
  constexpr int KS = D / 16, NB = D / 16, kWarps = C::kWarps, GP = NQ;
  constexpr int NJ = (NQ + 7) / 8, NP = NQ == 4 ? 1 : 2, kChunks = D / 32, kQuads = D / 4;
  const SplitArgs& a = fa.s;

  __shared__ __align__(8) uint64_t recv_bar;
  __shared__ int32_t coord_s[kMaxPieces];
  __shared__ int2 col_s[NQ];  // positions a head's query row attends
  __shared__ float2 ml_s[kWarps][GP];
  __shared__ float cw_s[kWarps][GP];
  __shared__ float2 row_s[GP * HC];
  __shared__ Fp4Wild<GP * HC> wild_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (used as declared, so that the compiler sees shared memory: rounded as an integer
  // it gave generic loads and 64-bit addresses, 5 % of the instructions)
  extern __shared__ __align__(128) uint8_t fp4_smem[];
  uint8_t* ring = fp4_smem;

  if constexpr (CL) {
    if (threadIdx.x == 0) {
      mbar_init(smem_u32(&recv_bar), cluster_size());
      fence_mbar_init();
    }
    __syncthreads();
    cluster_arrive_relaxed();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int capacity = a.max_pages * a.page_size;
  const int box_t = a.box_tokens, box_shift = __ffs(box_t) - 1;
  const int R = a.T * a.G, R1 = a.T * fa.G1;  // query rows of the CTA, of one head
  const int gid = lane >> 2, tig = lane & 3;
  uint8_t* recv = ring + C::kRingBytes;
  // this warp's head, and its place among the warps of that head
  const int head = warp % HC, first = warp / HC;
  constexpr int kStep = kWarps / HC;
  uint8_t* mine = ring + warp * C::kWarpBytes;
  uint8_t* ready_k = mine + 2 * C::kSlotBytes;
  uint8_t* ready_v = ready_k;
  float4* ready_row = reinterpret_cast<float4*>(ready_k + C::kReadyK);
  // the lane's places: in a slot's K and V codes (ldmatrix: matrix bit 0 of K tokens
  // 8.., bit 1 dims 32..; V's four chunks, or at head_dim 64 chunks and tokens 8..),
  // in the scales made ready, and the weights' selectors
  const int mat = lane >> 3, mrow = lane & 7;
  uint32_t k_at = fp4_offset<D / 2>(mrow + (mat & 1 ? 8 : 0), mat >> 1);
  uint32_t v_at = kChunks >= 4 ? fp4_offset<D / 2>(mrow, mat)
                               : fp4_offset<D / 2>(mrow + (mat & 2 ? 8 : 0), mat & 1);
  v_at += Loader::kV;
  uint32_t ks_at = NQ == 4 ? (gid * NB + (tig >> 1) * kChunks) * 4
                           : gid * 2 * NB + (tig >> 1) * NB;
  uint32_t vs_at = 2 * tig * 2 * NB + (gid >> 2) * NB;
  uint32_t sel = gid & 4 ? 0x32441044u : 0x44324410u;
  uint32_t slots = smem_u32(mine);
  keep(k_at);
  keep(v_at);
  keep(ks_at);
  keep(vs_at);
  keep(sel);
  keep(slots);
  const float4* my_rows = ready_row + (NQ == 4 ? 8 * (tig & 2) + gid : gid);
  // query row rr of the head (token rr / G1) among the CTA's rows
  auto cta_row = [&](int rr, int hd) {
    return HC == 1 ? rr : rr / fa.G1 * a.G + hd * fa.G1 + rr % fa.G1;
  };

  const int h = a.head_fastest ? blockIdx.x : blockIdx.y;
  const int s = a.head_fastest ? blockIdx.y : blockIdx.x;
  const int b = blockIdx.z;
  // the page id of this thread's first piece, read together with the length under
  // the guess that the sequence is as long as the plan's bound
  int spec_lo = -1, spec_phys = -1;
  {
    const SeqRange g =
        seq_range(a.len_hint, a.window, capacity, a.chunk, a.max_shards, a.T, a.balanced);
    if (g.status == 0 && s < g.nshards) {
      spec_lo = g.base + s * g.chunk;
      const int ptok = spec_lo + threadIdx.x * box_t;
      const size_t pi = (size_t)b * a.max_pages + (ptok >> a.page_shift);
      if (ptok < capacity && PGD_IN(pi, (size_t)a.batch * a.max_pages, a.err))
        spec_phys = ld_global_s32(a.page_table + pi);
    }
  }
  // q, too, comes beside the length
  uint32_t qf[NJ][KS][2];
  float acc[kChunks][NJ][NP][4];
  float m_run[NJ][2], l_part[NJ][2], scale[NJ][2];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int rr = NQ == 4 ? gid & 3 : 8 * j + gid;  // (four rows: twice)
    size_t qr = group_row(b, h, cta_row(rr < R1 ? rr : 0, head), a.T, a.G, a.Hq);
    if (!PGD_IN(qr, (size_t)a.batch * a.T * a.Hq, a.err)) qr = 0;
    const float f = fp4_load_q_row<D, E>(static_cast<const uint16_t*>(a.q) + qr * D,
                                         rr < R1, tig, qf[j]);
    if (NQ == 4 && (gid >> 2) != (tig >> 1)) {  // a column's dims of the other blocks
#pragma unroll
      for (int k = 0; k < KS; ++k) qf[j][k][0] = qf[j][k][1] = 0u;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // this lane's score columns are rows 8 j + 2 tig + e
      scale[j][e] = __shfl_sync(0xffffffffu, f, (2 * tig + e) * 4);
      m_run[j][e] = -INFINITY;
      l_part[j][e] = 0.f;
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int p = 0; p < NP; ++p)
        acc[c][j][p][0] = acc[c][j][p][1] = acc[c][j][p][2] = acc[c][j][p][3] = 0.f;
  const SeqRange r = seq_range(ld_global_s32(a.seq_lens + b), a.window, capacity, a.chunk,
                               a.max_shards, a.T, a.balanced);
  if (r.status != 0 || s >= r.nshards) {
    if (s == 0 && r.status != 0 && threadIdx.x == 0) raise_error(a.err, r.status);
    if constexpr (CL) {  // an empty partial still takes part in the exchange
      const ClusterXchg x(recv, R, D);
      cluster_wait();
      for (int e = threadIdx.x; e < R * kQuads; e += C::kThreads)
        x.push(e, make_float4(0.f, 0.f, 0.f, 0.f));
      for (int g = threadIdx.x; g < R; g += C::kThreads)
        x.push_ml(g, make_float2(-INFINITY, 0.f));
      cluster_finish<D, E>(a, x, b, h, smem_u32(&recv_bar), recv, C::kThreads);
    } else if (s == 0) {
      zero_group_rows<D, GP * HC>(a, b, h);
    }
    return;
  }
  const int shard_lo = r.base + s * r.chunk;
  const int lo = max(r.start, shard_lo), hi = min(r.end, shard_lo + r.chunk);
  if (threadIdx.x < GP * HC) wild_s.bits[threadIdx.x] = 0u;
  if (threadIdx.x == 0) wild_s.any = 0;
  if (threadIdx.x < NQ) {
    // query rows past R1 are zeros and attend what the last one does
    const int t = (int)threadIdx.x < R1 ? threadIdx.x / fa.G1 : a.T - 1;
    const int end = r.end - a.T + t + 1;
    col_s[threadIdx.x] = make_int2(a.window > 0 ? max(0, end - a.window) : 0, end);
  }
  Loader load(fa, coord_s, lane, h * HC + head, box_shift);
  // positions that every query row attends
  const int in_hi = min(hi, r.end - a.T + 1);
  const int in_lo = max(lo, a.window > 0 ? r.end - a.window : 0);
  const int n_units = (hi - shard_lo + kUnit - 1) / kUnit;
  const int n_pieces = (n_units * kUnit + box_t - 1) >> box_shift;
  int any_bad = 0;
  for (int i = threadIdx.x; i < n_pieces; i += C::kThreads) {
    const int ptok = shard_lo + i * box_t;
    int coord = 0;  // (a piece that no row attends)
    if (ptok < hi && ptok + box_t > lo) {
      int phys;
      if (i == (int)threadIdx.x && shard_lo == spec_lo) {
        phys = spec_phys;
      } else {
        const size_t pi = (size_t)b * a.max_pages + (ptok >> a.page_shift);
        phys = PGD_IN(pi, (size_t)a.batch * a.max_pages, a.err) ? a.page_table[pi] : -1;
      }
      if (phys < 0 || phys >= a.num_pages)
        any_bad = 1;
      else
        coord = phys * a.page_size + (ptok & (a.page_size - 1));
    }
    coord_s[i] = coord;
  }
  const bool bad = __syncthreads_or(any_bad);
  if (bad && threadIdx.x == 0) raise_error(a.err, DECODE_ATTN_DEV_BAD_PAGE);
  const int units = bad ? 0 : n_units;
  // groups in order: K, V of the first unit, K, V of the second, ...; two units ahead
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int u = first + n * kStep;
    if (u < units) {
      load.k(slots + n * C::kSlotBytes, u);
      load.v(slots + n * C::kSlotBytes);
    } else {
      cp_async_commit();
      cp_async_commit();
    }
  }
#pragma unroll 1
  for (int n = 0, u = first; u < units; ++n, u += kStep) {
    const int tok0 = shard_lo + u * kUnit;
    const uint32_t slot_at = (n & 1) * C::kSlotBytes;
    uint8_t* slot = mine + slot_at;
    const uint32_t to = slots + slot_at;
    const bool inside = tok0 >= in_lo && tok0 + kUnit <= in_hi;
    const int next = u + 2 * kStep;
    uint32_t words[NB / 4];
    cp_async_wait<3>();  // K of this unit, and the row scales
    __syncwarp();
    load_words<NB>(slot + Loader::kKb + lane * NB, words);
    {
      const float ks = a.scale_log2 * reinterpret_cast<const float*>(slot + Loader::kKr)[lane];
      if constexpr (NQ == 4)
        ready_scales_f32<NB>(words, ks, ready_k + lane * 4 * NB);
      else
        ready_scales<NB>(words, ready_k + lane * 2 * NB);
      const float vs = reinterpret_cast<const float*>(slot + Loader::kVr)[lane];
      // (a NaN, too, fails the comparison)
      ready_row[lane] =
          make_float4(ks, fabsf(vs) < kHugeScale ? vs : __int_as_float(0x7fffffff),
                      scale_log2_of(fminf(fabsf(vs), kHugeScale)), 0.f);
    }
    __syncwarp();
    float sc[2][NQ == 4 ? 1 : NJ][NQ == 4 ? 2 : 4];
    if constexpr (NQ == 4)
      fp4_scores_4<D>(to + k_at, ready_k + ks_at, tig & 2, qf[0],
                      reinterpret_cast<float(&)[2][2]>(sc));
    else
      fp4_scores<D, NJ>(to + k_at, ready_k + ks_at, qf, sc);
    __syncwarp();
    if (next < units)
      load.k(to, next);
    else
      cp_async_commit();
    cp_async_wait<3>();  // V of this unit
    __syncwarp();
    load_words<NB>(slot + Loader::kVb + lane * NB, words);
    if (!inside) {
      // V rows outside the range become zeros: a zero weight meets no NaN
      const int t = tok0 + lane;
      if (t < lo || t >= hi) {
#pragma unroll
        for (int w = 0; w < NB / 4; ++w) words[w] = 0u;
      } else if (a.T > 1) {
        // NaN blocks are noted for the rows that attend them and cleared: a zero
        // weight would carry them to the others
        uint32_t nan = 0;
#pragma unroll
        for (int w = 0; w < NB / 4; ++w) {
          const uint32_t four = __vcmpeq4(words[w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
#pragma unroll
          for (int k = 0; k < 4; ++k) nan |= (four >> (8 * k) & 1u) << (4 * w + k);
          words[w] &= ~four;
        }
        for (int rr = 0; nan != 0u && rr < R1; ++rr)
          if (t >= col_s[rr].x && t < col_s[rr].y) {
            wild_s.any = 1;
            atomicOr(&wild_s.bits[head * GP + rr], nan);
          }
      }
    }
    ready_scales<NB>(words, ready_v + lane * 2 * NB);
    uint32_t wt[4][NQ == 4 ? 2 : NJ];
    float l_sum[NJ][2], down[NJ][2];
    constexpr bool kFactor = !std::is_same<E, __half>::value;
    bool rescale;
    auto weights = [&](auto whole) {
      if constexpr (NQ == 4)
        rescale = fp4_weights_4<decltype(whole)::value, kFactor>(
            reinterpret_cast<float(&)[2][2]>(sc), my_rows, scale[0], col_s, tok0, lane, sel,
            m_run[0], l_sum[0], down[0], wt);
      else
        rescale = fp4_weights<NQ, NJ, decltype(whole)::value, kFactor>(
            sc, my_rows, scale, col_s, tok0, lane, m_run, l_sum, down, wt);
    };
    if (inside)
      weights(std::true_type{});
    else
      weights(std::false_type{});
    if (__any_sync(0xffffffffu, rescale)) {
      float alpha[NJ][2];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          alpha[j][e] = fast_exp2(down[j][e]);
          l_part[j][e] = carry_sum(l_part[j][e], down[j][e], alpha[j][e]);
        }
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            acc[c][j][p][0] *= alpha[j][0];
            acc[c][j][p][1] *= alpha[j][1];
            acc[c][j][p][2] *= alpha[j][0];
            acc[c][j][p][3] *= alpha[j][1];
          }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) l_part[j][e] += l_sum[j][e];
    __syncwarp();
    fp4_values<D, NQ, NJ, NP>(to + v_at, ready_v + vs_at, wt, acc);
    __syncwarp();
    if (next < units)
      load.v(to);
    else
      cp_async_commit();
  }
  cp_async_wait<0>();
  __syncthreads();  // every warp is done with the table and the ring

  // ---- fold the consumer warps in fixed order (deterministic) -----------
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_part[j][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if constexpr (NQ == 4) l += __shfl_xor_sync(0xffffffffu, l, 2);
      l_part[j][e] = l;
    }
  // the padding sends a fragment's stores to distinct banks, where it fits
  constexpr int kRowStride = kWarps * GP * (D + 4) * 4 <= C::kRingBytes ? D + 4 : D;
  static_assert(kWarps * GP * kRowStride * 4 <= C::kRingBytes, "warp states fit in the ring");
  float* acc_s = reinterpret_cast<float*>(ring);
  if (gid == 0 && (NQ > 4 || tig < 2)) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        ml_s[warp][8 * j + 2 * tig + e] = make_float2(m_run[j][e], l_part[j][e]);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float* to = acc_s + (warp * GP + (8 * j + 2 * tig) % NQ) * kRowStride + 32 * c + 4 * gid;
      if constexpr (NQ == 4) {  // columns 4 to 7 are the odd dims of the same rows
        const float(&o)[4] = acc[c][j][0];
        to += tig >> 1;
        to[0] = o[0];
        to[2] = o[2];
        to[kRowStride] = o[1];
        to[kRowStride + 2] = o[3];
      } else {
        const float(&o)[4] = acc[c][j][0];
        const float(&odd)[4] = acc[c][j][NP - 1];
        *reinterpret_cast<float4*>(to) = make_float4(o[0], odd[0], o[2], odd[2]);
        *reinterpret_cast<float4*>(to + kRowStride) = make_float4(o[1], odd[1], o[3], odd[3]);
      }
    }
  named_barrier_sync(1, kWarps * 32);
  // the CTA's row r: its head and the row among the head's
  auto head_row = [&](int r, int& hd) {
    if (HC == 1) {
      hd = 0;
      return r;
    }
    hd = r % a.G / fa.G1;
    return r / a.G * fa.G1 + r % fa.G1;
  };
  if ((int)threadIdx.x < R) {
    int hd;
    const int g = head_row(threadIdx.x, hd);
    const float2 ML = fold_states<kWarps, HC, GP>(ml_s, cw_s, hd, g);
    const float M = ML.x, L = ML.y;
    // (positions whose scores are no numbers alone leave no maximum, and would
    // pass for none in the merge)
    row_s[threadIdx.x] = make_float2(L != L ? fmaxf(M, -3e38f) : M, L);
  }
  named_barrier_sync(1, kWarps * 32);
  ClusterXchg x;
  if constexpr (CL) {
    x = ClusterXchg(recv, R, D);
    cluster_wait();
  }
  for (int e = threadIdx.x; e < R * kQuads; e += kWarps * 32) {
    const int rc = e / kQuads, q = e % kQuads;
    int hd;
    const int g = head_row(rc, hd);
    const float2 ML = row_s[rc];
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; w += HC) {
      const float c = cw_s[w + hd][g];
      if (c < 0.f) continue;
      const float4 v =
          *reinterpret_cast<const float4*>(acc_s + ((w + hd) * GP + g) * kRowStride + 4 * q);
      O.x += c * v.x;
      O.y += c * v.y;
      O.z += c * v.z;
      O.w += c * v.w;
    }
    if (wild_s.any && (wild_s.bits[hd * GP + g] >> (q >> 2) & 1u))
      O.x = O.y = O.z = O.w = __int_as_float(0x7fffffff);
    if (bad) O = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t row = group_row(b, h, rc, a.T, a.G, a.Hq);
    if (!a.split) {
      if (!PGD_IN(row, (size_t)a.batch * a.T * a.Hq, a.err)) continue;
      const bool z = bad || ML.y == 0.f;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + 4 * q) = make_uint2(
          ElemOps<E>::pack2(z ? 0.f : O.x / ML.y, z ? 0.f : O.y / ML.y),
          ElemOps<E>::pack2(z ? 0.f : O.z / ML.y, z ? 0.f : O.w / ML.y));
      continue;
    }
    const float2 part = make_float2(ML.x, bad ? -1.f : ML.y);
    if constexpr (CL) {
      x.push(e, O);
      if (q == 0) x.push_ml(rc, part);
    } else {
      const size_t at = row * a.max_shards + s;
      if (!PGD_IN(at, (size_t)a.batch * a.T * a.Hq * a.max_shards, a.err)) continue;
      *reinterpret_cast<float4*>(a.ws_acc + at * D + 4 * q) = O;
      if (q == 0) a.ws_ml[at] = part;
    }
  }
  if (!a.split) return;
  if constexpr (CL)
    cluster_finish<D, E>(a, x, b, h, smem_u32(&recv_bar), recv, kWarps * 32);
  else
    merge_if_last<D, E, 16>(a, r, b, h, ring, kWarps * 32);
}

}  // namespace pgd
