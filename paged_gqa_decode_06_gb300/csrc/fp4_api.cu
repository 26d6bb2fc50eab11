// decode_attn_fp4: argument checks, the host planner for a 4-bit cache and the
// launch.
#include <algorithm>
#include <cstring>

#include "fp4_launch.h"
#include "host_common.h"
#include "quant_plan.h"

using namespace pgd;

namespace {

constexpr int kDefaultSplitMin = 256;
constexpr int kLargeChunkCap = 2048;
constexpr int64_t kPairBytes = 32 << 20;
// Up to four sequences take one head a CTA and few_shards; more, two heads and pieces of
// 1.7 waves.  Of lengths all alike the first way is quicker to eight (32/8 heads of 128,
// 65536 positions: 4 sequences 67 us and 83, 6 96 and 114, 8 123 and 132); of U[1, L] the
// second is from five on (64/8 of 131072: 4 sequences 92 and 114, 5 114 and 100, 8 216 and
// 153), and the lengths are not known here.
constexpr int kFewSequences = 4;
constexpr double kSmallStep = 1280 * 1024;   // bytes per SM
constexpr double kSmallPiece = 96 * 1024;    // bytes per CTA slot
constexpr double kSmRingBytes = 152 * 1024;  // in flight per SM
// Of a few long sequences: what an SM takes for a position of one head with 1, 2, 3
// or 4 CTAs at once (ns at head_dim 128, up to 4 query rows; 8 rows take 1.15 times
// as long; other head_dims by their size and 16 rows as 8, which is no measurement: four
// sequences of 32768 take 68 us so with 16 rows and 65 at head_dim 256, by pieces 74 and
// 75), and what the merge takes per shard and query row (one sequence of 131072 positions
// by 38, 57 and 76 shards 45, 42 and 42 us).
constexpr double kRowNs[4] = {5.7, 4.6, 4.1, 3.95};
constexpr double kMergeNs = 20;

int queries(const decode_attn_params* p) { return p->num_queries > 1 ? p->num_queries : 1; }

// Bytes of a position's K and V of one head.
double row_bytes_of(int D) { return 2.0 * (D / 2 + D / 16 + 4); }

// The positions that a sequence attends at most, the tiles' start included, and
// the KV heads of a CTA: two, whose codes of a position lie side by side, where the
// step is large and of several sequences (64 of 8192: 127 us, 131 with one; short ones,
// U[1, 512], 88 and 101); a small step has too few CTAs as it is, and for a few long
// sequences the shards' partials of two heads cost more to merge (one of 131072 42
// us, 52 with two).
struct Work {
  int64_t attended, span;
  int heads;
};
Work work_of(const decode_attn_params* p) {
  const int T = queries(p), rows = T * (p->num_q_heads / p->num_kv_heads);
  const int64_t capacity = (int64_t)p->max_pages_per_seq * p->page_size;
  const int64_t max_len =
      p->max_seq_len > 0 ? std::min<int64_t>(p->max_seq_len, capacity) : capacity;
  Work w{};
  w.attended = p->window > 0 ? std::min<int64_t>(max_len, (int64_t)p->window + T - 1) : max_len;
  w.span = std::max<int64_t>(1, p->window > 0 ? w.attended + kTile - 1 : max_len);
  const double bytes =
      (double)p->batch * p->num_kv_heads * (double)w.span * row_bytes_of(p->head_dim);
  w.heads = rows <= 8 && p->num_kv_heads % 2 == 0 && p->head_dim < 256 && bytes >= kPairBytes &&
                    p->batch > kFewSequences
                ? 2
                : 1;
  return w;
}

// What the kernel for `rows` query rows and `heads` KV heads per CTA takes.
struct Shape {
  int room, ctas, warps;  // query rows, CTAs of an SM, warps of a CTA
  int recv_room;          // bytes left for a cluster's receive buffer
};
template <int D, int NQ, int HC>
Shape shape_as() {
  using C = Fp4Cfg<D, NQ, HC>;
  return Shape{NQ, C::kCtas, C::kWarps, C::kRecvRoom};
}
template <int D>
Shape shape_of(int rows, int heads) {
  constexpr int kTwo = D < 256 ? 2 : 1;
  if (rows > 8) return shape_as<D, 16, 1>();
  if (rows > 4) return heads == 2 ? shape_as<D, 8, kTwo>() : shape_as<D, 8, 1>();
  return heads == 2 ? shape_as<D, 4, kTwo>() : shape_as<D, 4, 1>();
}
Shape shape_of(int D, int rows, int heads) {
  return D == 64 ? shape_of<64>(rows, heads)
                 : D == 128 ? shape_of<128>(rows, heads) : shape_of<256>(rows, heads);
}

// Shards of each of a few long sequences, all in one wave: the CTAs of the fullest
// SM, as quick as that many are together, and the merge.
int64_t few_shards(int64_t units, int64_t sms, int ctas_per_sm, int64_t span, int64_t max_chunk,
                   int rows, int D) {
  const int64_t lo = std::max<int64_t>(2, ceil_div(span, max_chunk));
  const int64_t hi = std::max(lo, std::min(sms * ctas_per_sm / units, ceil_div(span, kMinChunk)));
  int64_t best = lo;
  double best_t = 1e300;
  for (int64_t s = lo; s <= hi; ++s) {
    const int64_t chunk = round_up(ceil_div(span, s), kTile);
    if (chunk > max_chunk) continue;
    const int64_t got = ceil_div(span, chunk);
    const int64_t per_sm = ceil_div(units * got, sms);
    const double row_ns = kRowNs[std::min<int64_t>(per_sm, 4) - 1] * D / 128 * (rows > 4 ? 1.15 : 1);
    const double t = (double)(per_sm * chunk) * row_ns + kMergeNs * (double)(got * rows);
    if (t < best_t) {
      best = got;
      best_t = t;
    }
  }
  return best;
}

}  // namespace

extern "C" int decode_attn_fp4_make_plan(const decode_attn_params* p, int32_t num_sms,
                                         decode_attn_plan* plan) {
  int st = validate_params(p);
  if (st) return st;
  if (!plan) return DECODE_ATTN_ERR_NULL;
  if (num_sms <= 0) return DECODE_ATTN_ERR_SHAPE;
  std::memset(plan, 0, sizeof(*plan));
  const int G = p->num_q_heads / p->num_kv_heads, T = queries(p), D = p->head_dim;
  if (p->variant != DECODE_ATTN_VARIANT_AUTO && p->variant != DECODE_ATTN_VARIANT_MMA)
    return DECODE_ATTN_ERR_VARIANT;
  if (T * G > 16) return DECODE_ATTN_ERR_VARIANT;

  const Work work = work_of(p);
  const int64_t attended = work.attended, span = work.span;
  const int HC = work.heads;
  const Shape shape = shape_of(D, T * G, HC);
  const int kv_heads = p->num_kv_heads / HC;
  const int64_t max_chunk = (int64_t)kMaxPieces * std::min(p->page_size, kTile);
  const int64_t units = std::max<int64_t>(1, (int64_t)p->batch * kv_heads);
  const int ctas_per_sm = shape.ctas;
  const int64_t slots = (int64_t)num_sms * ctas_per_sm;
  const double row_bytes = HC * row_bytes_of(D);
  const double bytes = (double)units * span * row_bytes;
  const int split_min = p->split_min > 0 ? p->split_min : kDefaultSplitMin;

  int64_t chunk;
  if (p->force_chunk > 0) {
    chunk = round_up(p->force_chunk, kTile);
    if (chunk > max_chunk) return DECODE_ATTN_ERR_SHAPE;
  } else if (attended <= split_min) {
    chunk = std::min(round_up(span, kTile), max_chunk);
  } else {
    int64_t s;
    // one wave of equal shards for small steps, by the 8-bit cache's rule, and for a
    // few long sequences; pieces that the SMs take as they come for large steps of more
    const bool several = 2 * units <= (int64_t)(kOneWaveFill * (double)slots);
    if (several && p->batch <= kFewSequences && bytes > (double)kPairBytes) {
      s = few_shards(units, num_sms, ctas_per_sm, span, max_chunk, T * G, D);
    } else if (several && bytes <= num_sms * kSmallStep) {
      s = one_wave(units, slots, span, row_bytes, max_chunk, kSmRingBytes / ctas_per_sm);
    } else if (!several && bytes <= (double)slots * kSmallPiece) {
      s = std::max<int64_t>(1, std::min(slots / units, ceil_div(span, kMinChunk)));
    } else {
      // about 1.7 waves; pieces short enough to balance mixed lengths
      const int64_t target = std::max<int64_t>(1, (17 * slots + 5 * units) / (10 * units));
      const int64_t cap = std::max<int64_t>(kLargeChunkCap, round_up(ceil_div(span, 16), kTile));
      s = std::max(target, ceil_div(span, cap));
    }
    chunk = std::min(round_up(ceil_div(span, s), kTile), max_chunk);
  }
  const int64_t shards = ceil_div(span, chunk);
  if (shards > 65535) return DECODE_ATTN_ERR_SHAPE;
  const int64_t ctas = (int64_t)p->batch * kv_heads * shards;
  const bool one_wave_grid = ctas <= slots;

  plan->variant = DECODE_ATTN_VARIANT_MMA;
  plan->group_pad = shape.room;
  plan->tile_tokens = kTile;
  plan->chunk_tokens = (int32_t)chunk;
  plan->max_shards = (int32_t)shards;
  plan->split = shards > 1 ? 1 : 0;
  plan->balanced = plan->split && one_wave_grid && p->force_chunk <= 0 ? 1 : 0;
  plan->ctas_per_sm = ctas_per_sm;
  plan->ring_stages = 2 * shape.warps;  // units of 32 positions of one head in flight
  // the merge, by the 8-bit planner's rule
  plan->grid_z = p->batch;
  const int recv = ClusterRecv::of(T * G * HC, D, (int)std::min<int64_t>(shards, 16)).bytes;
  const bool cluster_ok =
      plan->split && one_wave_grid && (shards <= 8 || (shards <= 16 && ctas <= 64));
  if (p->schedule == DECODE_ATTN_SCHEDULE_CLUSTER && !cluster_ok) return DECODE_ATTN_ERR_VARIANT;
  if (p->schedule == DECODE_ATTN_SCHEDULE_CLUSTER ||
      (p->schedule == DECODE_ATTN_SCHEDULE_AUTO && cluster_ok &&
       (ctas_per_sm > 1 || shards <= 4 || ctas <= 64) && recv <= shape.recv_room &&
       ((ctas * 5 >= slots * 4 && bytes <= (double)(256 << 20)) ||
        bytes <= (double)(32 << 20))))
    plan->cluster = (int32_t)shards;
  plan->head_fastest = plan->cluster ? 0 : 1;
  plan->grid_x = plan->head_fastest ? kv_heads : (int32_t)shards;
  plan->grid_y = plan->head_fastest ? (int32_t)shards : kv_heads;
  if (plan->split) {
    const size_t rows = (size_t)p->batch * T * p->num_q_heads * (size_t)shards;
    plan->workspace_bytes =
        ticket_bytes(p) + round_up(rows * sizeof(float2), 256) + round_up(rows * D * 4, 256);
  }
  return DECODE_ATTN_OK;
}

extern "C" size_t decode_attn_fp4_workspace_size(const decode_attn_params* p, int device) {
  int sms = 0;
  decode_attn_plan plan;
  if (device_sms(device, &sms) || decode_attn_fp4_make_plan(p, sms, &plan)) return 0;
  return plan.workspace_bytes;
}

extern "C" int decode_attn_fp4(const decode_attn_params* p, const decode_kv_cache* cache,
                               const void* q, const int32_t* page_table, const int32_t* seq_lens,
                               void* out, void* workspace, size_t workspace_bytes,
                               int32_t* err_flag, void* stream) {
  int st = validate_params(p);
  if (st) return st;
  if (!cache) return DECODE_ATTN_ERR_NULL;
  if (cache->kv_format != DECODE_ATTN_KV_E2M1) return DECODE_ATTN_ERR_SHAPE;
  if (p->batch == 0) return DECODE_ATTN_OK;
  const void* need[] = {q, cache->k_pages, cache->v_pages, cache->k_scales, cache->v_scales,
                        cache->k_blocks, cache->v_blocks, out, page_table, seq_lens};
  for (const void* ptr : need)
    if (!ptr) return DECODE_ATTN_ERR_NULL;
  for (int i = 0; i < 8; ++i)
    if (!aligned16(need[i])) return DECODE_ATTN_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DECODE_ATTN_ERR_CUDA;
  if ((st = device_sms(dev, &sms))) return st;
  decode_attn_plan plan;
  if ((st = decode_attn_fp4_make_plan(p, sms, &plan))) return st;
  if (plan.split && (!workspace || workspace_bytes < plan.workspace_bytes ||
                     (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return DECODE_ATTN_ERR_WORKSPACE;

  const int D = p->head_dim;
  const int HC = work_of(p).heads;
  const int kv_heads = p->num_kv_heads / HC;
  const int box_t = std::min(p->page_size, kTile);
  Fp4Launch L{};
  L.args.codes[0] = static_cast<const uint8_t*>(cache->k_pages);
  L.args.codes[1] = static_cast<const uint8_t*>(cache->v_pages);
  L.args.scales[0] = cache->k_scales;
  L.args.scales[1] = cache->v_scales;
  L.args.blocks[0] = cache->k_blocks;
  L.args.blocks[1] = cache->v_blocks;
  SplitArgs& a = L.args.s;
  a.q = q;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.err = err_flag;
  if (plan.split) {
    const size_t slots =
        (size_t)p->batch * queries(p) * p->num_q_heads * (size_t)plan.max_shards;
    char* base = static_cast<char*>(workspace);
    const size_t tickets = ticket_bytes(p);
    a.counters = reinterpret_cast<int32_t*>(base);
    a.ws_ml = reinterpret_cast<float2*>(base + tickets);
    a.ws_acc = reinterpret_cast<float*>(base + tickets + round_up(slots * sizeof(float2), 256));
    if (!plan.cluster &&
        (st = clear_far_tickets(base, (int64_t)p->batch * kv_heads,
                                static_cast<cudaStream_t>(stream))))
      return st;
  }
  a.Hq = p->num_q_heads;
  a.Hkv = kv_heads;
  a.G = p->num_q_heads / kv_heads;
  L.args.G1 = p->num_q_heads / p->num_kv_heads;
  L.args.heads = p->num_kv_heads;
  a.max_pages = p->max_pages_per_seq;
  a.num_pages = p->num_pages;
  a.page_size = p->page_size;
  a.page_shift = ilog2(p->page_size);
  a.box_tokens = box_t;
  a.window = p->window > 0 ? p->window : 0;
  a.chunk = plan.chunk_tokens;
  a.max_shards = plan.max_shards;
  a.balanced = plan.balanced;
  a.split = plan.split;
  a.T = queries(p);
  a.head_fastest = plan.head_fastest;
  a.batch = p->batch;
  const int64_t cap = (int64_t)p->max_pages_per_seq * p->page_size;
  a.len_hint = (int32_t)(p->max_seq_len > 0 ? std::min<int64_t>(p->max_seq_len, cap) : cap);
  a.scale_log2 = p->scale * kLog2e;
  L.grid = dim3(plan.grid_x, plan.grid_y, plan.grid_z);
  L.group_pad = plan.group_pad;
  L.dtype = p->dtype;
  L.cluster = plan.cluster;
  L.stream = static_cast<cudaStream_t>(stream);
  switch (D) {
    case 64: return cuda_status(launch_fp4_d64(L));
    case 128: return cuda_status(launch_fp4_d128(L));
    default: return cuda_status(launch_fp4_d256(L));
  }
}
