// Decode attention over an 8-bit cache (e4m3 codes, one fp32 scale per
// (position, KV head) row of K and of V): out = sum_t p_t vs_t vc_t with
// scores scale * ks_t * (q . kc_t).
//
// The shape of the 16-bit split kernel (split_mma.cuh): one CTA per (shard,
// KV head or two, sequence), one or two producer warps filling a shared-memory
// ring by TMA, pairs of consumer warps that take its stages in turn, mma.sync
// with the tokens on M and the group's query rows on N, and the same merges
// (workspace, or a cluster's distributed shared memory).  What differs is what
// a stage holds and how the fragments come out of it:
//  * A stage is 64 positions of codes (half the bytes), so twice the stages
//    are in flight; the scales of its positions follow by cp.async, 16 bytes
//    (4 positions of one head; they lie [P][Hkv][PS]) per lane.
//  * Codes become fp16 in registers, exactly: ldmatrix moves pairs of codes,
//    a K register of four dims gives two A registers (the order of the
//    contraction is free, so q is loaded in the same order), and a transposed
//    V register of (2 tokens x 2 dims) gives, after two conversions and two
//    byte permutations, the registers of two output dims.
//  * The products are fp16 for either element type of q: a bf16 row of q is
//    scaled by a power of two to magnitudes below 2^15 (the largest above
//    2^14), where fp16 holds all 8 bits of a value down to 2^-31 of the row's
//    largest and 2^-39 of it absolutely, and the scores take the factor back.
//  * The scales enter in fp32, ks with the scores.  vs goes into the weight
//    w_t = p_t vs_t: the running maximum is taken over log2(p_t vs_t), less 14,
//    so that the largest w_t is 2^14 whatever the magnitude of V, while the sum
//    keeps p_t.  w is split into an fp16 head and remainder (two products),
//    whose last place is 2^-24: 22 bits of a weight down to 2^-16 of the
//    largest, 11 down to 2^-28, nothing below 2^-39 (with a largest w of 1 the
//    weights of a context far below one token's would end at 2^-25).
//
// Measured (GB300): four sequences of 131072 positions, 64 heads over 8, 187 us
// (5.9 TB/s; 195 run after run), 64 of U[1, 8192] 109 us, one of 3060 9.1 us.  The
// copies bound it: with consumers that only release the stages the long step
// takes 170 to 185 us, since a head's row is one 128-byte line of the eight that
// lie together.
#pragma once

#include <type_traits>

#include "e4m3.cuh"
#include "split_mma.cuh"
#include "tcgen05.cuh"  // mbar_wait_hot

namespace pgd {

// A CTA takes HC = 1 or 2 neighbouring KV heads.  Two, where one head's box of
// a page's piece is too small for the copy engine: a box costs about 45 ns
// whatever it brings, and a box can hold the rows of several heads (GB300,
// pages of 16: 64 sequences of U[1, 8192] positions 125 -> 114 us, a thousand
// of U[1, 512] 193 -> 140 us, head_dim 256 118 -> 108 us).  A stage then
// holds half the positions, and the two warps that share it take a head each.
// Everything after the streams sees one KV head with twice the query
// heads.
struct QuantArgs {
  SplitArgs s;            // as for the 16-bit split kernel; G and Hkv of HC heads as one
  const float* k_scales;  // [P][Hkv][PS]
  const float* v_scales;
  int32_t G1, heads;      // query heads per KV head, KV heads
};

template <int D, int NT8 = 1, int HC = 1>
struct QuantCfg {
  // Consumer warps: pairs that share a stage, 32 positions a warp, the pairs
  // taking the stages in turn.  Turning codes into fragments is a long chain
  // of short instructions, so each warp gets two independent blocks of 16
  // positions, and there are as many pairs as the registers and the ring
  // (whose stages every pair must return to) allow.
  static constexpr int kWarps = NT8 == 2 && D <= 128 ? 4 : 6;
  // Warps that fill the ring.  The smaller stages of two heads' CTAs come twice
  // as often, and two warps share them (64 sequences of U[1, 8192] positions
  // 120 -> 115 us); with one head's the second only takes issue slots from the
  // consumers (four sequences of 131072 201 -> 206 us).
  static constexpr int kProducers = HC;
  static constexpr int kThreads = (kWarps + kProducers) * 32;
  // CTAs of an SM: two, and one with twice the ring at D = 256, whose
  // accumulators and fragments need more registers than two leave.
  static constexpr int kCtas = D == 256 ? 1 : 2;
  static constexpr int kWidth = D < 128 ? D : 128;   // bytes of a swizzled row
  static constexpr int kTileBytes = kTile * D;       // K or V codes of a stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = (192 / kCtas) * 1024 / kStageBytes;  // 12, 6, 6
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kSmemBytes = kRingBytes + 1024;
  // static shared memory (scales, row coordinates, warps' states), and what is
  // left of a CTA's share of the SM's 228 KB for a cluster's receive buffer
  static constexpr int kTableBytes =
      kStages * 2 * kTile * 4 + kMaxPieces * 4 + D * 4 + (D == 256 ? 1408 : 1120);
  static constexpr int kRecvRoom = 228 * 1024 / kCtas - 1024 - kSmemBytes - kTableBytes;
};

// Byte offset of (token t, 16-byte chunk c) of a CTA's head in a tile of codes
// made of pieces of 2^ps rows, each [D / kWidth][HC heads][2^ps rows][kWidth]
// with the 128-byte (or at D = 64 the 64-byte) swizzle.
template <int D, int HC>
__device__ __forceinline__ uint32_t code_offset(int t, int c, int head, int ps) {
  constexpr int W = QuantCfg<D>::kWidth, kChunks = W / 16;
  const int rows = 1 << ps, r = t & (rows - 1);
  const int key = W == 128 ? (r & 7) : ((r >> 1) & 3);
  return (uint32_t)((t >> ps) * (rows * D * HC) + ((c / kChunks) * HC + head) * (rows * W) +
                    r * W + (((c % kChunks) ^ key) << 4));
}

// log2 of a V scale for the running maximum, less 14 (above).  At least that of
// 2^-90, so that a zero row (scale 0) makes no sum overflow: p is at most 2^104
// then, the sum of a shard's 65536 at most 2^120.  No bound
// above: the weights of a larger scale would pass fp16's range (an Inf, less
// itself in the remainder: a row of NaN).  A largest weight of scale 2^119
// leaves p = 2^-105 in the sum, which holds 2^-21 of that (it ends at 2^-126).
__device__ __forceinline__ float scale_log2_of(float v) {
  const float a = fmaxf(fabsf(v), 0x1p-90f);
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(a));
  return y - 14.f;
}

// V rows with a scale from here on take no part in the maximum and the
// products, where the other positions would be left without a weight: the
// append writes 2^120 for a row with an Inf.  (The test takes 0.9 % of the long
// step's time, 1.3 of the mix's, 5 at head_dim 64; ahead of the block 2, 4 and 4.
// With 16 query rows it goes there, 64 -> 68 us on 16 sequences of 8192, since
// in the middle it takes the registers of the products: 74.)
constexpr float kHugeScale = 0x1p120f;

// Dims of the CTA's rows (row g of head hd at hd * GP + g) that an Inf (1), a
// -Inf (2) or a NaN (both) reaches, kept beside the accumulators: the products
// would carry them to rows that do not attend them.
template <int D, int GP, int HC>
struct QuantWild {
  uint32_t bits[GP * HC][D / 16];  // two bits per dim
  int32_t any;
};

// Notes what position t (row tr of the tile) adds to the rows that attend it
// beside the products: with a huge scale an Inf in the dims whose code is not
// zero, with a scale of 0 a NaN where the code is one.
template <int D, int NT8, int HC>
__device__ __forceinline__ void note_row(QuantWild<D, 8 * NT8, HC>& wild, const uint8_t* kt,
                                         float scale, int tr, int head, int lane, int t,
                                         const int (&col_lo)[NT8][2],
                                         const int (&col_hi)[NT8][2], int ps) {
  wild.any = 1;
#pragma unroll 1
  for (int mi = 0; mi < D / 16; ++mi) {
    const uint16_t codes = *reinterpret_cast<const uint16_t*>(
        kt + QuantCfg<D>::kTileBytes + code_offset<D, HC>(tr, mi, head, ps) + 2 * (lane >> 2));
    const float2 x = ElemOps<__half>::unpack2(e4m3_to_half2(codes));
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float v = (i ? x.y : x.x) * scale;
      const uint32_t two = v != v ? 3u : v > 0.f ? 1u : v < 0.f ? 2u : 0u;
      bits |= two << (4 * (lane >> 2) + 2 * i);
    }
#pragma unroll
    for (int j = 0; j < NT8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (bits != 0u && t >= col_lo[j][e] && t < col_hi[j][e])
          atomicOr(&wild.bits[head * 8 * NT8 + 8 * j + 2 * (lane & 3) + e][mi], bits);
  }
}

// One consumer warp's 32 positions of a staged tile (K codes at kt, V codes
// behind them, ks / vs the scales of its positions), as two blocks of 16:
// mma_block's counterpart.  They are the tile's positions t0.. of head `head`.
// inside: every column attends all 32.
template <int D, int NT8, int HC, bool MT>
__device__ __forceinline__ void quant_block(uint8_t* kt, const float* ks_s, float* vs_s,
                                            int t0, int head, int lane, int tok0, int lo, int hi,
                                            bool inside, const int (&col_lo)[NT8][2],
                                            const int (&col_hi)[NT8][2],
                                            const uint32_t (&qf)[NT8][D / 16][2],
                                            const float (&col_scale)[NT8][2],
                                            float (&acc)[D / 16][NT8][4], float (&m_run)[NT8][2],
                                            float (&l_part)[NT8][2], int ps,
                                            QuantWild<D, 8 * NT8, HC>& wild) {
  using H = ElemOps<__half>;
  const int gid = lane >> 2;
  const int mat = lane >> 3, mrow = lane & 7;
  const int tok = t0 + mrow + ((mat & 1) ? 8 : 0);  // matrix bit 0: tokens 8..15 of a block
  const int hd = mat >> 1;                          // matrix bit 1: dims 16..31
  const uint32_t kbase = smem_u32(kt);
  const uint32_t vbase = kbase + QuantCfg<D>::kTileBytes;
  if (tok0 < lo || tok0 + 32 > hi) {
    // V codes outside the range become zeros: a zero weight meets no NaN
    uint8_t* vt = kt + QuantCfg<D>::kTileBytes;
    for (int e = lane; e < 32 * (D / 16); e += 32) {
      const int t = e / (D / 16), c = e % (D / 16);
      if (tok0 + t < lo || tok0 + t >= hi)
        *reinterpret_cast<uint4*>(vt + code_offset<D, HC>(t0 + t, c, head, ps)) =
            make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncwarp();
  }
  if (MT && !inside) {
    // NaN codes of V become zeros and are noted for the rows that attend them:
    // a zero weight would carry them to the others
    uint8_t* vt = kt + QuantCfg<D>::kTileBytes;
    bool nan = false;
    for (int c = 0; c < D / 16; ++c) {
      const uint4 v =
          *reinterpret_cast<const uint4*>(vt + code_offset<D, HC>(t0 + lane, c, head, ps));
      for (uint32_t w : {v.x, v.y, v.z, v.w})
        nan |= __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u;
    }
    uint32_t rows = __ballot_sync(0xffffffffu, nan);
    for (uint32_t left = rows; left != 0u; left &= left - 1) {
      const int t = __ffs(left) - 1;
      note_row<D, NT8, HC>(wild, kt, 0.f, t0 + t, head, lane, tok0 + t, col_lo, col_hi, ps);
    }
    if (rows != 0u) {
      __syncwarp();
      if (nan)
        for (int c = 0; c < D / 16; ++c) {
          uint4* at = reinterpret_cast<uint4*>(vt + code_offset<D, HC>(t0 + lane, c, head, ps));
          uint4 v = *at;
          for (uint32_t* w : {&v.x, &v.y, &v.z, &v.w})
            *w &= ~__vcmpeq4(*w & 0x7f7f7f7fu, 0x7f7f7f7fu);
          *at = v;
        }
      fence_proxy_async_smem();
      __syncwarp();
    }
  }
  // notes the rows of a huge scale; a bit per position
  auto note_huge_rows = [&] {
    const uint32_t apart = __ballot_sync(0xffffffffu, fabsf(vs_s[lane]) >= kHugeScale);
    for (uint32_t left = apart; left != 0u; left &= left - 1) {
      const int t = __ffs(left) - 1;
      if (tok0 + t >= lo && tok0 + t < hi)
        note_row<D, NT8, HC>(wild, kt, vs_s[t], t0 + t, head, lane, tok0 + t, col_lo, col_hi, ps);
    }
    return apart;
  };
  if constexpr (NT8 == 2)
    if (__any_sync(0xffffffffu, fabsf(vs_s[lane]) >= kHugeScale)) {
      const uint32_t apart = note_huge_rows();
      __syncwarp();
      if (apart >> lane & 1u) vs_s[lane] = 0.f;
      __syncwarp();
    }
  float sc[2][NT8][4];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int j = 0; j < NT8; ++j) sc[b][j][0] = sc[b][j][1] = sc[b][j][2] = sc[b][j][3] = 0.f;
#pragma unroll
  for (int kb = 0; kb < D / 32; ++kb)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t r[4];  // (tokens 0-7, 8-15) x (dims 0-15, 16-31): four dims per register
      ldmatrix_x4(r, kbase + code_offset<D, HC>(tok + 16 * b, 2 * kb + hd, head, ps));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t af[4] = {e4m3_to_half2(r[2 * i] & 0xffffu),
                                e4m3_to_half2(r[2 * i + 1] & 0xffffu),
                                e4m3_to_half2(r[2 * i] >> 16), e4m3_to_half2(r[2 * i + 1] >> 16)};
#pragma unroll
        for (int j = 0; j < NT8; ++j)
          H::mma(sc[b][j], af, qf[j][2 * kb + i][0], qf[j][2 * kb + i][1]);
      }
    }
  // this lane's positions: gid + 8 i of the 32
  float ks[4], vs[4], lv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ks[i] = ks_s[gid + 8 * i];
    vs[i] = vs_s[gid + 8 * i];
    lv[i] = scale_log2_of(vs[i]);
  }
  if constexpr (NT8 == 1) {
    const float top = fmaxf(fmaxf(fabsf(vs[0]), fabsf(vs[1])), fmaxf(fabsf(vs[2]), fabsf(vs[3])));
    if (__any_sync(0xffffffffu, top >= kHugeScale)) {
      const uint32_t apart = note_huge_rows();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (apart >> (gid + 8 * i) & 1u) {
          vs[i] = 0.f;
          lv[i] = scale_log2_of(0.f);
        }
    }
  }
  uint32_t pb_hi[2][NT8][2], pb_lo[2][NT8][2];
  bool rescale = false;
  float alpha[NT8][2];
#pragma unroll
  for (int j = 0; j < NT8; ++j) {
    float w[4][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sv[4], mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sv[i] = sc[i >> 1][j][e + 2 * (i & 1)] * (col_scale[j][e] * ks[i]);
        if (!inside) {
          const int t = tok0 + gid + 8 * i;
          if (t < col_lo[j][e] || t >= col_hi[j][e]) sv[i] = -INFINITY;
        }
        mx = fmaxf(mx, sv[i] + (inside || sv[i] != -INFINITY ? lv[i] : 0.f));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float m_new = fmaxf(m_run[j][e], mx);
      alpha[j][e] = (m_new == -INFINITY) ? 1.f : fast_exp2(m_run[j][e] - m_new);
      rescale |= alpha[j][e] != 1.f;
      float l = l_part[j][e] * alpha[j][e];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = inside || sv[i] != -INFINITY;
        const float p = in ? fast_exp2(sv[i] - m_new) : 0.f;
        l += p;
        w[i][e] = in ? p * vs[i] : 0.f;
      }
      l_part[j][e] = l;
      m_run[j][e] = m_new;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = H::pack2(w[i][0], w[i][1]);
      const float2 f = H::unpack2(h);
      pb_hi[i >> 1][j][i & 1] = movmatrix_trans(h);
      pb_lo[i >> 1][j][i & 1] = movmatrix_trans(H::pack2(w[i][0] - f.x, w[i][1] - f.y));
    }
  }
  if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
    for (int mi = 0; mi < D / 16; ++mi)
#pragma unroll
      for (int j = 0; j < NT8; ++j) {
        acc[mi][j][0] *= alpha[j][0];
        acc[mi][j][1] *= alpha[j][1];
        acc[mi][j][2] *= alpha[j][0];
        acc[mi][j][3] *= alpha[j][1];
      }
  }
  // out^T += V^T . W^T: row gid of a tile of 16 dims is dim 2 gid, row gid + 8
  // dim 2 gid + 1
#pragma unroll
  for (int kb = 0; kb < D / 32; ++kb)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t r[4];  // as for K, transposed: (2 tokens x 2 dims) per register
      ldmatrix_x4_trans(r, vbase + code_offset<D, HC>(tok + 16 * b, 2 * kb + hd, head, ps));
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = __byte_perm(r[i], 0u, 0x3120);  // (2 dims x 2 tokens)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t af[4] = {e4m3_to_half2(r[2 * i] & 0xffffu), e4m3_to_half2(r[2 * i] >> 16),
                                e4m3_to_half2(r[2 * i + 1] & 0xffffu),
                                e4m3_to_half2(r[2 * i + 1] >> 16)};
#pragma unroll
        for (int j = 0; j < NT8; ++j) {
          H::mma(acc[2 * kb + i][j], af, pb_hi[b][j][0], pb_hi[b][j][1]);
          H::mma(acc[2 * kb + i][j], af, pb_lo[b][j][0], pb_lo[b][j][1]);
        }
      }
    }
}

// A row of q as fp16 fragments, 4 consecutive dims per lane and 16-dim step;
// returns the power of two taken out of a bf16 row.
template <int D, class E>
__device__ __forceinline__ float load_q_row(const uint16_t* row, bool live, int tig,
                                            uint32_t (&qf)[D / 16][2]) {
  uint2 raw[D / 16];
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    raw[ks] = live ? *reinterpret_cast<const uint2*>(row + ks * 16 + 4 * tig) : make_uint2(0u, 0u);
  if constexpr (std::is_same<E, __half>::value) {
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[ks][0] = raw[ks].x;
      qf[ks][1] = raw[ks].y;
    }
    return 1.f;
  } else {
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const float2 a = ElemOps<E>::unpack2(raw[ks].x), b = ElemOps<E>::unpack2(raw[ks].y);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^(E - 14) of the row's largest value, 2^E at least (a tiny row stays, an
    // Inf stays Inf; bf16's largest is scaled to 65280)
    const uint32_t e = min(max((__float_as_uint(amax) >> 23) & 255u, 27u), 253u) - 14u;
    const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const float2 a = ElemOps<E>::unpack2(raw[ks].x), b = ElemOps<E>::unpack2(raw[ks].y);
      qf[ks][0] = ElemOps<__half>::pack2(a.x * inv, a.y * inv);
      qf[ks][1] = ElemOps<__half>::pack2(b.x * inv, b.y * inv);
    }
    return __uint_as_float(e << 23);
  }
}

// CL: a cluster plan, as in split_mma_body.  MT: several new tokens per sequence
// (a kernel of its own: with the test in one kernel the steps of single tokens
// took 0.5 to 1.5 % longer).
template <int D, int NT8, class E, bool CL, int HC, bool MT>
__global__ void __launch_bounds__(QuantCfg<D, NT8, HC>::kThreads, QuantCfg<D, NT8, HC>::kCtas)
    quant_split_kernel(const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const QuantArgs qa) {
  using C = QuantCfg<D, NT8, HC>;
  constexpr int kPairs = C::kWarps / 2;
  static_assert(C::kStages % kPairs == 0, "a pair sees every phase of its stages");
  constexpr int KS = D / 16, kWarps = C::kWarps, GP = 8 * NT8;
  constexpr int kStagePos = kTile / HC;
  const SplitArgs& a = qa.s;

  __shared__ __align__(8) uint64_t full_bar[C::kStages];
  __shared__ __align__(8) uint64_t empty_bar[C::kStages];
  __shared__ __align__(8) uint64_t recv_bar;
  __shared__ __align__(16) float scale_s[C::kStages][2][kTile];
  __shared__ int32_t coord_s[kMaxPieces];
  __shared__ float2 ml_s[kWarps][GP];
  __shared__ float cw_s[kWarps][GP];
  __shared__ float2 row_s[GP * HC];
  __shared__ QuantWild<D, GP, HC> wild_s;
  __shared__ int32_t bad_s;
  __shared__ volatile int32_t abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (written so that the code of one producer stays as it is without this)
  const bool producer = C::kProducers == 1 ? warp == kWarps : warp >= kWarps;
  const int part = C::kProducers == 1 ? 0 : warp - kWarps;
  uint8_t* ring = ring_base();

  if (threadIdx.x == kWarps * 32) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    for (int st = 0; st < C::kStages; ++st) {
      // the boxes' arrival, and one of each producer lane for its scales
      mbar_init(smem_u32(&full_bar[st]), 1 + 32);
      mbar_init(smem_u32(&empty_bar[st]), 2);
    }
    if constexpr (CL) mbar_init(smem_u32(&recv_bar), cluster_size());
    fence_mbar_init();
    abort_s = 0;
    bad_s = 0;
    wild_s.any = 0;
  }
  for (int i = threadIdx.x; i < GP * HC * (D / 16); i += C::kThreads)
    wild_s.bits[i / (D / 16)][i % (D / 16)] = 0u;
  __syncthreads();
  if constexpr (CL) cluster_arrive_relaxed();
  grid_dependency_wait();
  grid_launch_dependents();
  const int h = a.head_fastest ? blockIdx.x : blockIdx.y;
  const int s = a.head_fastest ? blockIdx.y : blockIdx.x;
  const int b = blockIdx.z;
  const int capacity = a.max_pages * a.page_size;
  const int box_t = a.box_tokens;
  // page ids of the first 32 pieces, read together with the length under the
  // guess that the sequence is as long as the plan's bound
  int spec_lo = -1, spec_phys = -1;
  if (producer) {
    const SeqRange g =
        seq_range(a.len_hint, a.window, capacity, a.chunk, a.max_shards, a.T, a.balanced);
    if (g.status == 0 && s < g.nshards) {
      spec_lo = g.base + s * g.chunk;
      const int ptok = spec_lo + lane * box_t;
      const size_t pi = (size_t)b * a.max_pages + (ptok >> a.page_shift);
      if (ptok < capacity && PGD_IN(pi, (size_t)a.batch * a.max_pages, a.err))
        spec_phys = ld_global_s32(a.page_table + pi);
    }
  }
  const SeqRange r = seq_range(ld_global_s32(a.seq_lens + b), a.window, capacity, a.chunk,
                               a.max_shards, a.T, a.balanced);
  const int R = a.T * a.G, R1 = a.T * qa.G1;  // query rows of the CTA, of one head
  const int gid = lane >> 2, tig = lane & 3;
  uint8_t* recv = ring + C::kRingBytes;

  if (r.status != 0 || s >= r.nshards) {
    if (s == 0 && r.status != 0 && threadIdx.x == 0) raise_error(a.err, r.status);
    if constexpr (CL) {
      if (warp < kWarps) {  // an empty partial still takes part in the exchange
        const ClusterXchg x(recv, R, D);
        cluster_wait();
        for (int e = threadIdx.x; e < R * (D / 4); e += kWarps * 32)
          x.push(e, make_float4(0.f, 0.f, 0.f, 0.f));
        for (int g = threadIdx.x; g < R; g += kWarps * 32)
          x.push_ml(g, make_float2(-INFINITY, 0.f));
        cluster_finish<D, E>(a, x, b, h, smem_u32(&recv_bar), recv, kWarps * 32);
      }
    } else if (s == 0) {
      zero_group_rows<D, GP * HC>(a, b, h);
    }
    return;
  }

  const int shard_lo = r.base + s * r.chunk;
  const int lo = max(r.start, shard_lo);
  const int hi = min(r.end, shard_lo + r.chunk);
  const int n_tiles = (hi - shard_lo + kStagePos - 1) / kStagePos;
  const int pieces = kStagePos / box_t, n_pieces = n_tiles * pieces;

  if (producer) {
    const int pool_rows = a.num_pages * a.page_size;  // past the pool: zeros
    int any_bad = 0;
#pragma unroll 4
    for (int i = lane; i < n_pieces; i += 32) {
      const int ptok = shard_lo + i * box_t;
      int coord = pool_rows;
      if (ptok < hi && ptok + box_t > lo) {
        int phys;
        if (i == lane && shard_lo == spec_lo) {
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
    if (__any_sync(0xffffffffu, any_bad)) {
      // no copy is issued; the consumers' first wait completes on plain
      // arrivals and they find the flag
      if (part > 0) return;
      if (lane == 0) {
        bad_s = 1;
        raise_error(a.err, DECODE_ATTN_DEV_BAD_PAGE);
      }
      __syncwarp();
      for (int i = 0; i < kPairs; ++i) {  // each pair's first stage
        mbar_arrive(smem_u32(&full_bar[i]));
        if (lane == 0) mbar_arrive(smem_u32(&full_bar[i]));
      }
      return;
    }
    __syncwarp();
    const uint64_t policy = l2_evict_first_policy();
    const float* scales = lane < 16 ? qa.k_scales : qa.v_scales;
    int issued = 0;
    for (int i = part; i < n_tiles; i += C::kProducers) {
      const int st = i % C::kStages;
      if (i >= C::kStages) {
        int go = 1;
        if (lane == 0) {
          if (!mbar_wait_hot(smem_u32(&empty_bar[st]), ((i / C::kStages) & 1) ^ 1)) {
            abort_s = 1;
            raise_error(a.err, DECODE_ATTN_DEV_TIMEOUT);
          }
          go = abort_s ? 0 : 1;
        }
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
      }
      const uint32_t fb = smem_u32(&full_bar[st]);
      if (lane == 0) mbar_arrive_expect_tx(fb, C::kStageBytes + (i == 0 ? a.stall_tx : 0));
      __syncwarp();
      if (lane < 2 * pieces) {  // at most 16 boxes: pieces of 8 positions or more
        const int coord = coord_s[i * pieces + (lane >> 1)];
        const bool in =
            PGD_IN(coord == pool_rows ? 0 : (int64_t)coord + box_t - 1, pool_rows, a.err);
        tma_load_4d_hint(smem_u32(ring + st * C::kStageBytes) + (lane & 1) * C::kTileBytes +
                             (lane >> 1) * box_t * D * HC,
                         (lane & 1) ? &tmap_v : &tmap_k, 0, in ? coord : pool_rows, h * HC, 0,
                         fb, policy);
      }
      {
        // this lane's 4 positions' scales (lanes 0-15 K, 16-31 V; of 16 lanes
        // the upper 8 the second head's); zeros where no position is attended
        const int t = 4 * (lane & (kStagePos / 4 - 1));
        const int hd = h * HC + (HC == 2 ? (lane >> 3) & 1 : 0);
        const int coord = coord_s[i * pieces + t / box_t];
        const bool in = coord < pool_rows;
        const int row = (in ? coord : 0) + (in ? t % box_t : 0);
        const size_t at = ((size_t)(row >> a.page_shift) * qa.heads + hd) * a.page_size +
                          (row & (a.page_size - 1));
        const bool ok = PGD_IN(at + 3, (size_t)pool_rows * qa.heads, a.err);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(&scale_s[st][lane >> 4][4 * (lane & 15)])),
                     "l"(scales + (ok ? at : 0)), "r"(in && ok ? 16 : 0)
                     : "memory");
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
      }
      issued = i + 1;
    }
    // this CTA's copies in flight have landed before the warp exits
    for (int i = max(0, issued - C::kStages); i < issued; ++i)
      if (i % C::kProducers == part)
        mbar_wait_hot(smem_u32(&full_bar[i % C::kStages]), (i / C::kStages) & 1);
    return;
  }

  // ------------------------------------------------------------ consumers
  uint32_t qf[NT8][KS][2];
  float acc[KS][NT8][4];
  int col_lo[NT8][2], col_hi[NT8][2];
  float m_run[NT8][2], l_part[NT8][2], col_scale[NT8][2];
  // this warp's positions of a stage, or head of the CTA
  const int half = warp & 1, head = HC == 2 ? half : 0;
  // query row rr of the head (token rr / G1) among the CTA's rows
  auto cta_row = [&](int rr, int hd) {
    return HC == 1 ? rr : rr / qa.G1 * a.G + hd * qa.G1 + rr % qa.G1;
  };
#pragma unroll
  for (int j = 0; j < NT8; ++j) {
    const int rr = 8 * j + gid;
    size_t qr = group_row(b, h, cta_row(rr < R1 ? rr : 0, head), a.T, a.G, a.Hq);
    if (!PGD_IN(qr, (size_t)a.batch * a.T * a.Hq, a.err)) qr = 0;
    const float f =
        load_q_row<D, E>(static_cast<const uint16_t*>(a.q) + qr * D, rr < R1, tig, qf[j]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // this lane's score columns are rows 8j + 2 tig + e
      col_scale[j][e] = a.scale_log2 * __shfl_sync(0xffffffffu, f, (2 * tig + e) * 4);
      const int cr = 8 * j + 2 * tig + e;
      const int t = cr < R1 ? cr / qa.G1 : a.T - 1;
      col_hi[j][e] = r.end - a.T + t + 1;
      col_lo[j][e] = a.window > 0 ? max(0, col_hi[j][e] - a.window) : 0;
      m_run[j][e] = -INFINITY;
      l_part[j][e] = 0.f;
    }
  }
#pragma unroll
  for (int mi = 0; mi < KS; ++mi)
#pragma unroll
    for (int j = 0; j < NT8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mi][j][e] = 0.f;
  const int piece_shift = __ffs(box_t) - 1;
  // positions that every query row attends
  const int in_hi = r.end - a.T + 1, in_lo = a.window > 0 ? r.end - a.window : 0;
  for (int i = warp >> 1; i < n_tiles; i += kPairs) {
    const int st = i % C::kStages;
    if (!mbar_wait_hot(smem_u32(&full_bar[st]), (i / C::kStages) & 1)) {
      abort_s = 1;
      raise_error(a.err, DECODE_ATTN_DEV_TIMEOUT);
      break;
    }
    if (bad_s || abort_s) break;
    const int t0 = HC == 1 ? 32 * half : 0;
    const int tok0 = shard_lo + i * kStagePos + t0;
    if (tok0 + 32 > lo && tok0 < hi) {
      const bool inside = tok0 >= max(lo, in_lo) && tok0 + 32 <= min(hi, in_hi);
      quant_block<D, NT8, HC, MT>(ring + st * C::kStageBytes, &scale_s[st][0][32 * half],
                                  &scale_s[st][1][32 * half], t0, head, lane, tok0, lo, hi, inside,
                                  col_lo, col_hi, qf, col_scale, acc, m_run, l_part, piece_shift,
                                  wild_s);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&empty_bar[st]));
  }

  // ---- fold the consumer warps in fixed order (deterministic) -----------
#pragma unroll
  for (int j = 0; j < NT8; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_part[j][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      l_part[j][e] = l;
    }
  named_barrier_sync(1, kWarps * 32);  // every consumer is done with the ring
  // the padding sends a fragment's stores to distinct banks, where it fits
  constexpr int kRowStride = kWarps * GP * (D + 4) * 4 <= C::kRingBytes ? D + 4 : D;
  static_assert(kWarps * GP * kRowStride * 4 <= C::kRingBytes, "warp states fit in the ring");
  float* acc_s = reinterpret_cast<float*>(ring);
  if (gid == 0) {
#pragma unroll
    for (int j = 0; j < NT8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        ml_s[warp][8 * j + 2 * tig + e] = make_float2(m_run[j][e], l_part[j][e]);
  }
#pragma unroll
  for (int mi = 0; mi < KS; ++mi)
#pragma unroll
    for (int j = 0; j < NT8; ++j) {
      const int hd = 8 * j + 2 * tig, d = 16 * mi + 2 * gid;
      float* base = acc_s + (warp * GP) * kRowStride;
      *reinterpret_cast<float2*>(base + hd * kRowStride + d) =
          make_float2(acc[mi][j][0], acc[mi][j][2]);
      *reinterpret_cast<float2*>(base + (hd + 1) * kRowStride + d) =
          make_float2(acc[mi][j][1], acc[mi][j][3]);
    }
  named_barrier_sync(1, kWarps * 32);
  // the CTA's row r: its head and the row among the head's
  auto head_row = [&](int r, int& hd) {
    if (HC == 1) {
      hd = 0;
      return r;
    }
    hd = r % a.G / qa.G1;
    return r / a.G * qa.G1 + r % qa.G1;
  };
  if (threadIdx.x < R) {
    int hd;
    const int g = head_row(threadIdx.x, hd);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; w += HC) M = fmaxf(M, ml_s[w + hd][g].x);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w += HC) {
      const float2 ml = ml_s[w + hd][g];
      const float c = ml.y == 0.f ? 0.f : fast_exp2(ml.x - M);
      if (ml.y != 0.f) L += c * ml.y;
      cw_s[w + hd][g] = c;
    }
    row_s[threadIdx.x] = make_float2(M, L);
  }
  named_barrier_sync(1, kWarps * 32);
  const bool dead = bad_s != 0 || abort_s != 0;
  ClusterXchg x;
  if constexpr (CL) {
    x = ClusterXchg(recv, R, D);
    cluster_wait();
  }
  constexpr int kQuads = D / 4;
  for (int e = threadIdx.x; e < R * kQuads; e += kWarps * 32) {
    const int rc = e / kQuads, q = e % kQuads;
    int hd;
    const int g = head_row(rc, hd);
    const float2 ML = row_s[rc];
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; w += HC) {
      const float c = cw_s[w + hd][g];
      if (c == 0.f) continue;
      const float4 v =
          *reinterpret_cast<const float4*>(acc_s + ((w + hd) * GP + g) * kRowStride + 4 * q);
      O.x += c * v.x;
      O.y += c * v.y;
      O.z += c * v.z;
      O.w += c * v.w;
    }
    if (wild_s.any) {
      const uint32_t bits = wild_s.bits[hd * GP + g][q >> 2] >> (8 * (q & 3));
      auto add = [&](float& o, uint32_t two) {
        if (two & 1u) o += INFINITY;
        if (two & 2u) o -= INFINITY;
      };
      add(O.x, bits);
      add(O.y, bits >> 2);
      add(O.z, bits >> 4);
      add(O.w, bits >> 6);
    }
    const size_t row = group_row(b, h, rc, a.T, a.G, a.Hq);
    if (!a.split) {
      if (!PGD_IN(row, (size_t)a.batch * a.T * a.Hq, a.err)) continue;
      const bool z = dead || ML.y == 0.f;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + 4 * q) = make_uint2(
          ElemOps<E>::pack2(z ? 0.f : O.x / ML.y, z ? 0.f : O.y / ML.y),
          ElemOps<E>::pack2(z ? 0.f : O.z / ML.y, z ? 0.f : O.w / ML.y));
      continue;
    }
    const float4 Ow = dead ? make_float4(0.f, 0.f, 0.f, 0.f) : O;
    const float2 MLw = make_float2(ML.x, dead ? -1.f : ML.y);
    if constexpr (CL) {
      x.push(e, Ow);
      if (q == 0) x.push_ml(rc, MLw);
    } else {
      const size_t slot = row * a.max_shards + s;
      if (!PGD_IN(slot, (size_t)a.batch * a.T * a.Hq * a.max_shards, a.err)) continue;
      *reinterpret_cast<float4*>(a.ws_acc + slot * D + 4 * q) = Ow;
      if (q == 0) a.ws_ml[slot] = MLw;
    }
  }
  if (!a.split) return;
  if constexpr (CL)
    cluster_finish<D, E>(a, x, b, h, smem_u32(&recv_bar), recv, kWarps * 32);
  else
    merge_if_last<D, E, 16>(a, r, b, h, ring, kWarps * 32);
}

}  // namespace pgd
