// decode_attn_quant: argument checks, the host planner for an 8-bit cache,
// the TMA descriptors and the launch.
#include <algorithm>
#include <cstring>

#include "host_common.h"
#include "quant_launch.h"

using namespace pgd;

namespace {

constexpr int kDefaultSplitMin = 256;
constexpr int kMinChunk = 128;
constexpr int kLargeChunkCap = 2048;
constexpr int64_t kPairBytes = 64 << 20;
constexpr int kFewSequences = 4;
constexpr double kSmallStep = 1280 * 1024;  // bytes per SM
constexpr double kSmRingBytes = 192 * 1024;  // in flight per SM
// The one-wave cost model of the 16-bit planner: the read rate, the loaded
// round trip in which a CTA moves its ring, the merge per 8 shards, and the
// share of the CTA slots a one-wave grid fills.
constexpr double kStreamBytesPerS = 7.0e12, kRoundTripS = 3.0e-6, kMergeStepS = 1.2e-6;
constexpr double kOneWaveFill = 0.85;

int queries(const decode_attn_params* p) { return p->num_queries > 1 ? p->num_queries : 1; }

// KV heads of a CTA: two where the box of a page's piece of one head is at most
// 4 KB and the step is large (QuantArgs).  With boxes of 8 KB it depends on the
// plan (four sequences of 131072 positions 198 -> 191 us, one of them 61 -> 75:
// half the units, so twice the shards to merge), and a small step has too few
// CTAs as it is.
int heads_per_cta(const decode_attn_params* p, int64_t span) {
  const int rows = queries(p) * (p->num_q_heads / p->num_kv_heads);
  const int64_t box = (int64_t)std::min(p->page_size, kTile) * p->head_dim;
  const int64_t bytes = (int64_t)p->batch * p->num_kv_heads * span * 2 * p->head_dim;
  return rows <= 8 && p->num_kv_heads % 2 == 0 && box <= 4096 && bytes >= kPairBytes ? 2 : 1;
}

// Shards of a sequence when the grid is one wave: least t(S) = bytes /
// min(read rate, CTAs * ring / round trip) + the merge, ties to more CTAs.
int64_t one_wave(int64_t units, int64_t slots, int64_t span, double row_bytes, int64_t max_chunk,
                 double ring_bytes) {
  const double bytes = (double)units * (double)span * row_bytes;
  const int64_t s_lo = std::max<int64_t>(2, ceil_div(span, max_chunk));
  const int64_t fill = std::max<int64_t>(1, (int64_t)(kOneWaveFill * (double)slots) / units);
  const int64_t s_hi = std::max(s_lo, std::min(fill, ceil_div(span, kMinChunk)));
  int64_t best = s_lo;
  double best_t = 1e300;
  for (int64_t s = s_lo; s <= s_hi; ++s) {
    const int64_t chunk = round_up(ceil_div(span, s), kTile);
    if (chunk > max_chunk) continue;
    const int64_t got = ceil_div(span, chunk);
    const double rate =
        std::min(kStreamBytesPerS, (double)(units * got) * ring_bytes / kRoundTripS);
    const double t = bytes / rate + (got > 1 ? kMergeStepS * (double)ceil_div(got, 8) : 0.0);
    if (t < best_t * (1 - 1e-3) || (t <= best_t * (1 + 1e-3) && got > best)) {
      best = got;
      best_t = std::min(best_t, t);
    }
  }
  return best;
}

}  // namespace

extern "C" int decode_attn_quant_make_plan(const decode_attn_params* p, int32_t kv_format,
                                           int32_t num_sms, decode_attn_plan* plan) {
  int st = validate_params(p);
  if (st) return st;
  if (!plan) return DECODE_ATTN_ERR_NULL;
  if (num_sms <= 0 || kv_format != DECODE_ATTN_KV_E4M3) return DECODE_ATTN_ERR_SHAPE;
  std::memset(plan, 0, sizeof(*plan));
  const int G = p->num_q_heads / p->num_kv_heads, T = queries(p), D = p->head_dim;
  if (p->variant != DECODE_ATTN_VARIANT_AUTO && p->variant != DECODE_ATTN_VARIANT_MMA)
    return DECODE_ATTN_ERR_VARIANT;
  if (T * G > 16) return DECODE_ATTN_ERR_VARIANT;

  const int64_t capacity = (int64_t)p->max_pages_per_seq * p->page_size;
  const int64_t max_len =
      p->max_seq_len > 0 ? std::min<int64_t>(p->max_seq_len, capacity) : capacity;
  const int64_t attended =
      p->window > 0 ? std::min<int64_t>(max_len, (int64_t)p->window + T - 1) : max_len;
  const int64_t span = std::max<int64_t>(1, p->window > 0 ? attended + kTile - 1 : max_len);
  const int HC = heads_per_cta(p, span);
  const int kv_heads = p->num_kv_heads / HC;
  const int64_t max_chunk = (int64_t)kMaxPieces * std::min(p->page_size, kTile / HC);
  const int64_t units = std::max<int64_t>(1, (int64_t)p->batch * kv_heads);
  const int ctas_per_sm = D == 256 ? QuantCfg<256>::kCtas : QuantCfg<128>::kCtas;
  const int64_t slots = (int64_t)num_sms * ctas_per_sm;
  const double row_bytes = HC * (2.0 * D + 8);  // a position's K and V codes and scales
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
    // One wave of equal shards is the quickest where the sequences are equally
    // long, and the host knows only their bound; where a large step has more
    // than a few, pieces that the SMs take as they come cost little then and
    // save much otherwise (16 sequences of 32768, head_dim 64: 63 us by one
    // wave, 68 by pieces; of U[1, 32768] 55 and 37 us.  8 of 65536, 64 heads:
    // 198 and 190 us).
    const bool several = 2 * units <= (int64_t)(kOneWaveFill * (double)slots);
    if (several && (bytes <= num_sms * kSmallStep || p->batch <= kFewSequences)) {
      s = one_wave(units, slots, span, row_bytes, max_chunk, kSmRingBytes / ctas_per_sm);
    } else if (!several && bytes <= (double)slots * (1 << 20)) {
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
  plan->group_pad = T * G <= 8 ? 8 : 16;
  plan->tile_tokens = kTile;
  plan->chunk_tokens = (int32_t)chunk;
  plan->max_shards = (int32_t)shards;
  plan->split = shards > 1 ? 1 : 0;
  plan->balanced = plan->split && one_wave_grid && p->force_chunk <= 0 ? 1 : 0;
  plan->ctas_per_sm = ctas_per_sm;
  plan->ring_stages = D == 64 ? QuantCfg<64>::kStages
                              : D == 128 ? QuantCfg<128>::kStages : QuantCfg<256>::kStages;
  // the merge, by the 16-bit planner's rule: a cluster for one-wave plans of
  // 2..8 shards (16 on grids of at most 64 CTAs) that fill 4/5 of the slots,
  // or of small steps.  Not of long ones, where a cluster's CTAs, shards of one
  // head, start together and not the heads (four sequences of 131072: 198 us;
  // 16 of 4096: 33 us, without clusters 35); and only where the receive buffer
  // leaves room for the CTAs of an SM (16 rows of head_dim 128 do not: 8
  // sequences of 65536, pages of 16, 346 us by clusters, one CTA per SM, and
  // 195 us through the workspace)
  const int recv = ClusterRecv::of(T * G * HC, D, (int)std::min<int64_t>(shards, 16)).bytes;
  // One CTA per SM leaves GPCs without room for a second cluster of 8 (2
  // sequences of 16384, head_dim 256: 50 us by clusters, 30 us without).
  const bool cluster_ok =
      plan->split && one_wave_grid && (shards <= 8 || (shards <= 16 && ctas <= 64));
  if (p->schedule == DECODE_ATTN_SCHEDULE_CLUSTER && !cluster_ok) return DECODE_ATTN_ERR_VARIANT;
  if (p->schedule == DECODE_ATTN_SCHEDULE_CLUSTER ||
      (p->schedule == DECODE_ATTN_SCHEDULE_AUTO && cluster_ok &&
       (ctas_per_sm > 1 || shards <= 4 || ctas <= 64) &&
       recv <= (D == 64 ? QuantCfg<64>::kRecvRoom
                        : D == 128 ? QuantCfg<128>::kRecvRoom : QuantCfg<256>::kRecvRoom) &&
       ((ctas * 5 >= slots * 4 && bytes <= (double)(256 << 20)) ||
        bytes <= (double)(32 << 20))))
    plan->cluster = (int32_t)shards;
  // The heads of a shard side by side: their rows of a position are neighbours
  // in memory, which the DRAM answers better when they are asked for together
  // (four sequences of 131072: 192 us, 207 with the shards side by side, as a
  // cluster's have to be).
  plan->head_fastest = plan->cluster ? 0 : 1;
  plan->grid_x = plan->head_fastest ? kv_heads : (int32_t)shards;
  plan->grid_y = plan->head_fastest ? (int32_t)shards : kv_heads;
  plan->grid_z = p->batch;
  if (plan->split) {
    const size_t rows = (size_t)p->batch * T * p->num_q_heads * (size_t)shards;
    plan->workspace_bytes =
        ticket_bytes(p) + round_up(rows * sizeof(float2), 256) + round_up(rows * D * 4, 256);
  }
  return DECODE_ATTN_OK;
}

extern "C" size_t decode_attn_quant_workspace_size(const decode_attn_params* p, int32_t kv_format,
                                                   int device) {
  int sms = 0;
  decode_attn_plan plan;
  if (device_sms(device, &sms) || decode_attn_quant_make_plan(p, kv_format, sms, &plan)) return 0;
  return plan.workspace_bytes;
}

extern "C" int decode_attn_quant(const decode_attn_params* p, int32_t kv_format, const void* q,
                                 const void* k_pages, const void* v_pages, const float* k_scales,
                                 const float* v_scales, const int32_t* page_table,
                                 const int32_t* seq_lens, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* err_flag, void* stream) {
  int st = validate_params(p);
  if (st) return st;
  if (kv_format != DECODE_ATTN_KV_E4M3) return DECODE_ATTN_ERR_SHAPE;
  if (p->batch == 0) return DECODE_ATTN_OK;
  if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !page_table || !seq_lens || !out)
    return DECODE_ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_scales) ||
      !aligned16(v_scales) || !aligned16(out))
    return DECODE_ATTN_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DECODE_ATTN_ERR_CUDA;
  if ((st = device_sms(dev, &sms))) return st;
  decode_attn_plan plan;
  if ((st = decode_attn_quant_make_plan(p, kv_format, sms, &plan))) return st;
  if (plan.split && (!workspace || workspace_bytes < plan.workspace_bytes ||
                     (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return DECODE_ATTN_ERR_WORKSPACE;

  const int D = p->head_dim;
  const int kv_heads = plan.head_fastest ? plan.grid_x : plan.grid_y;
  const int HC = p->num_kv_heads / kv_heads;
  const int box_t = std::min(p->page_size, kTile / HC);
  QuantLaunch L{};
  for (int i = 0; i < 2; ++i) {
    // [P][PS][Hkv][D] codes as (up to 128 dims, row, head, chunk of 128
    // dims): one box = a page's piece with all its dims
    const uint64_t w = std::min(D, 128), row = (uint64_t)p->num_kv_heads * D;
    const uint64_t dims[4] = {w, (uint64_t)p->num_pages * p->page_size,
                              (uint64_t)p->num_kv_heads, (uint64_t)D / w};
    const uint64_t strides[3] = {row, (uint64_t)D, w};
    const uint32_t box[4] = {(uint32_t)w, (uint32_t)box_t, (uint32_t)HC, (uint32_t)(D / w)};
    st = encode_map(i ? &L.tmap_v : &L.tmap_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                    i ? v_pages : k_pages, dims, strides, box);
    if (st) return st;
  }
  L.args.k_scales = k_scales;
  L.args.v_scales = v_scales;
  SplitArgs& a = L.args.s;
  a.q = q;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.err = err_flag;
  if (plan.split) {
    const size_t rows = (size_t)p->batch * queries(p) * p->num_q_heads * (size_t)plan.max_shards;
    char* base = static_cast<char*>(workspace);
    const size_t tickets = ticket_bytes(p);
    a.counters = reinterpret_cast<int32_t*>(base);
    a.ws_ml = reinterpret_cast<float2*>(base + tickets);
    a.ws_acc = reinterpret_cast<float*>(base + tickets + round_up(rows * sizeof(float2), 256));
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
  a.stall_tx = env_positive("DECODE_ATTN_TEST_STALL_TX");  // a test's hook; unset in normal use
  a.scale_log2 = p->scale * kLog2e;
  L.grid = dim3(plan.grid_x, plan.grid_y, plan.grid_z);
  L.group_pad = plan.group_pad;
  L.dtype = p->dtype;
  L.cluster = plan.cluster;
  L.stream = static_cast<cudaStream_t>(stream);
  switch (D) {
    case 64: return cuda_status(launch_quant_d64(L));
    case 128: return cuda_status(launch_quant_d128(L));
    default: return cuda_status(launch_quant_d256(L));
  }
}
