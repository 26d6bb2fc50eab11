// C entry points of the chunk attention: argument checks, the host planner,
// the TMA descriptors and the launches.
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled

#include <algorithm>
#include <cstdlib>
#include <cstring>

#include "chunk_launch.h"
#include "host_common.h"

using namespace pgd;

namespace {

// Scratch starts where decode_attn's shard tickets end (they are never
// written here), so one zeroed buffer serves both.
constexpr size_t kTickets = 64 * 1024;
constexpr int64_t kMaxPartialBytes = int64_t(512) << 20;  // of a split plan
constexpr int kMaxShards = 128;
// Cost model of a plan (GB300): the rate of the products and a tile's latency,
// the read rate of the cache, a CTA's fixed time (launch, first loads, output)
// and that of one without work, the merge kernel's, and the rate at which
// partials are written and read back.  Fitted to 309 random calls at 1 to 128
// shards: the plan's time is 1.7 % above the best of them in the mean, and
// more than 1.2 times the best in 9 (with a fixed time of 3 us, no time for
// empty CTAs and whole waves only 3.3 % and 18).
constexpr double kFlops = 1.1e15, kTileS = 0.25e-6, kReadBytes = 7.0e12, kFixedS = 9.5e-6,
                 kEmptyS = 3.5e-6, kMergeS = 3.0e-6, kPartialBytes = 2.5e12;
// More waves than this overlap: the last one counts for kTailWave.
constexpr double kFullWaves = 3.0, kTailWave = 0.35;
// Of the longest sequence's tiles the share that a CTA has when there are more
// sequences and more CTAs than SMs.
constexpr double kRagged = 0.9;

int tile_keys(int head_dim) {
  return head_dim == 256 ? ChunkCfg<256>::kKeys : ChunkCfg<128>::kKeys;
}
int streams(int head_dim) {
  return head_dim == 256 ? ChunkCfg<256>::kStreams : ChunkCfg<128>::kStreams;
}

// The window, 0 for none; one as long as the table's capacity is none, so that
// the kernel's positions minus a window stay in 32 bits (a token before
// position 0 has a negative one).
int32_t window_of(const decode_attn_params* p) {
  const int64_t capacity = (int64_t)p->max_pages_per_seq * p->page_size;
  return p->window > 0 && p->window < capacity ? p->window : 0;
}

int run_chunk(const decode_attn_params* p, const decode_attn_chunk_plan& plan, int32_t total,
              const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
              const int32_t* query_offsets, const int32_t* seq_lens, void* out, void* workspace,
              int32_t* err_flag, cudaStream_t stream) {
  const int D = p->head_dim, G = p->num_q_heads / p->num_kv_heads;
  ChunkLaunch L{};
  ChunkArgs& a = L.args;
  a.page_table = page_table;
  a.offsets = query_offsets;
  a.seq_lens = seq_lens;
  a.v_pages = v_pages;
  a.out = out;
  a.err = err_flag;
  a.B = p->batch;
  a.total = total;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = G;
  a.max_pages = p->max_pages_per_seq;
  a.num_pages = p->num_pages;
  a.page_size = p->page_size;
  a.page_shift = ilog2(p->page_size);
  a.box_t = std::min(p->page_size, tile_keys(D));
  a.window = window_of(p);
  a.tile_tok = plan.tile_tokens;
  a.item_tok = plan.item_tokens;
  a.slots = plan.slots;
  a.max_shards = plan.max_shards;
  a.shard_tiles = plan.shard_keys / tile_keys(D);
  a.by_item = FastDiv::of(a.item_tok);
  a.by_heads = FastDiv::of(a.Hkv);
  a.by_shards = FastDiv::of(a.max_shards);
  a.by_shard_tiles = FastDiv::of(a.shard_tiles);
  a.by_group = FastDiv::of(G);
  a.stall_tx = env_positive("DECODE_ATTN_TEST_STALL_TX");  // a test's hook; unset in normal use
  a.scale_log2 = p->scale * kLog2e;
  if (plan.max_shards > 1) {
    char* ws = static_cast<char*>(workspace) + kTickets;
    a.ws_ml = reinterpret_cast<float2*>(ws);
    a.ws_acc = reinterpret_cast<float*>(
        ws + round_up((int64_t)total * p->num_q_heads * plan.max_shards * 8, 256));
  }

  const CUtensorMapDataType et = p->dtype == DECODE_ATTN_DTYPE_BF16
                                     ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  {
    // [total][Hq][D] as (64 dims, head, token, chunk of 64 dims): one box =
    // the group's heads of tile_tok tokens, rows token * G + g
    const uint64_t dims[4] = {64, (uint64_t)p->num_q_heads, (uint64_t)total, (uint64_t)D / 64};
    const uint64_t strides[3] = {(uint64_t)D * 2, (uint64_t)p->num_q_heads * D * 2, 128};
    const uint32_t box[4] = {64, (uint32_t)G, (uint32_t)a.tile_tok, 1};
    int st = encode_map(&L.tmap_q, et, 4, q, dims, strides, box);
    if (st) return st;
  }
  for (int i = 0; i < 2; ++i) {
    // [P][PS][Hkv][D] as (64 dims, token of 8, chunk of 64 dims, group of 8
    // tokens, head): one box = a piece of a page with all its dims
    const uint64_t row = (uint64_t)p->num_kv_heads * D * 2;
    const uint64_t dims[5] = {64, 8, (uint64_t)D / 64,
                              (uint64_t)p->num_pages * p->page_size / 8,
                              (uint64_t)p->num_kv_heads};
    const uint64_t strides[4] = {row, 128, row * 8, (uint64_t)D * 2};
    const uint32_t box[5] = {64, 8, (uint32_t)D / 64, (uint32_t)a.box_t / 8, 1};
    int st = encode_map(i ? &L.tmap_v : &L.tmap_k, et, 5, i ? v_pages : k_pages, dims, strides,
                        box);
    if (st) return st;
  }
  L.grid = (unsigned)plan.grid;
  L.combine_grid = 0;
  if (plan.max_shards > 1) {
    const int64_t blocks = ceil_div((int64_t)plan.item_tokens * G, kChunkCombineRows);
    L.combine_grid = (unsigned)(blocks * p->num_kv_heads * plan.slots);
  }
  L.dtype = p->dtype;
  L.stream = stream;
  switch (D) {
    case 64: return cuda_status(launch_chunk_d64(L));
    case 128: return cuda_status(launch_chunk_d128(L));
    default: return cuda_status(launch_chunk_d256(L));
  }
}

}  // namespace

extern "C" int decode_attn_chunk_make_plan(const decode_attn_params* p, int32_t total_queries,
                                           int32_t num_sms, decode_attn_chunk_plan* plan) {
  int st = validate_params(p);
  if (st) return st;
  if (!plan) return DECODE_ATTN_ERR_NULL;
  if (num_sms <= 0 || total_queries < 0) return DECODE_ATTN_ERR_SHAPE;
  std::memset(plan, 0, sizeof(*plan));
  const int D = p->head_dim, G = p->num_q_heads / p->num_kv_heads;
  const int KT = tile_keys(D), NS = streams(D);
  plan->tile_tokens = 128 / G;
  plan->item_tokens = NS * plan->tile_tokens;
  const int64_t slots = (int64_t)total_queries / plan->item_tokens + p->batch;
  const int64_t capacity = (int64_t)p->max_pages_per_seq * p->page_size;
  const int32_t window = window_of(p);
  const int64_t max_len =
      p->max_seq_len > 0 ? std::min<int64_t>(p->max_seq_len, capacity) : capacity;

  // The typical CTA: the average sequence's tokens over the longest range.
  const int64_t avg = p->batch > 0 ? std::max<int64_t>(1, ceil_div(total_queries, p->batch)) : 1;
  const int64_t items = std::max<int64_t>(
      1, (int64_t)p->batch * ceil_div(avg, plan->item_tokens) * p->num_kv_heads);
  const int64_t tokens = std::min<int64_t>(avg, plan->item_tokens);
  const int64_t span =
      window > 0 ? std::min<int64_t>(max_len, (int64_t)window + tokens) : max_len;
  const int64_t tiles = std::max<int64_t>(1, ceil_div(span, KT) + (window > 0 ? 1 : 0));
  const int ns = tokens > plan->tile_tokens ? NS : 1;

  int64_t shards = 1;
  if (p->force_chunk > 0) {
    const int64_t per = std::min<int64_t>(tiles, ceil_div(p->force_chunk, KT));
    shards = std::min<int64_t>(kMaxShards, ceil_div(tiles, per));
  } else {
    // Shards of the key range: a CTA's time is its tiles at the products'
    // rate or the cache's read rate, whichever is slower, and a fixed part;
    // CTAs run in waves of one per SM; splitting adds the merge.
    const double rows = (double)total_queries * p->num_q_heads;
    const double mma = 4.0 * 128 * ns * KT * D / (kFlops / num_sms) + kTileS;
    double best = 1e300;
    for (int64_t s = 1; s <= std::min<int64_t>(tiles, kMaxShards); ++s) {
      if (s > 1 && rows * s * (D + 2) * 4 > (double)kMaxPartialBytes) break;
      const int64_t ctas = items * s;
      const int64_t empty = std::max<int64_t>(0, slots * p->num_kv_heads * s - ctas);
      const double read = 4.0 * KT * D / (kReadBytes / (double)std::min<int64_t>(ctas, num_sms));
      const double waves = ctas <= kFullWaves * num_sms ? (double)ceil_div(ctas, num_sms)
                                                        : (double)ctas / num_sms + kTailWave;
      const double share = p->batch > 1 && ctas > num_sms ? kRagged : 1.0;
      const double t =
          waves * (share * (double)ceil_div(tiles, s) * std::max(mma, read) + kFixedS) +
          (double)empty / num_sms * kEmptyS +
          (s > 1 ? kMergeS + 2 * rows * s * D * 4 / kPartialBytes : 0.0);
      if (t < best * (1 - 1e-3)) {
        best = t;
        shards = s;
      }
    }
  }
  plan->max_shards = (int32_t)shards;
  plan->shard_keys = (int32_t)(ceil_div(tiles, shards) * KT);
  const int64_t grid = slots * shards * p->num_kv_heads;
  const int64_t combine = ceil_div((int64_t)plan->item_tokens * G, kChunkCombineRows) *
                          p->num_kv_heads * slots;
  if (slots > INT32_MAX || grid > INT32_MAX || (shards > 1 && combine > INT32_MAX))
    return DECODE_ATTN_ERR_SHAPE;
  plan->slots = (int32_t)slots;
  plan->grid = (int32_t)grid;
  if (shards > 1) {
    const int64_t rows = (int64_t)total_queries * p->num_q_heads * shards;
    plan->workspace_bytes =
        kTickets + (size_t)round_up(rows * 8, 256) + (size_t)round_up(rows * D * 4, 256);
  }
  return DECODE_ATTN_OK;
}

extern "C" size_t decode_attn_chunk_workspace_size(const decode_attn_params* p,
                                                   int32_t total_queries, int device) {
  int sms = 0;
  decode_attn_chunk_plan plan;
  if (device_sms(device, &sms) || decode_attn_chunk_make_plan(p, total_queries, sms, &plan))
    return 0;
  return plan.workspace_bytes;
}

extern "C" int decode_attn_chunk(const decode_attn_params* p, int32_t total_queries, const void* q,
                                 const void* k_pages, const void* v_pages,
                                 const int32_t* page_table, const int32_t* query_offsets,
                                 const int32_t* seq_lens, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* err_flag, void* stream) {
  int st = validate_params(p);
  if (st) return st;
  if (total_queries < 0) return DECODE_ATTN_ERR_SHAPE;
  if (p->batch == 0 || total_queries == 0) return DECODE_ATTN_OK;
  if (!q || !k_pages || !v_pages || !page_table || !query_offsets || !seq_lens || !out)
    return DECODE_ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
    return DECODE_ATTN_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DECODE_ATTN_ERR_CUDA;
  if ((st = device_sms(dev, &sms))) return st;
  decode_attn_chunk_plan plan;
  if ((st = decode_attn_chunk_make_plan(p, total_queries, sms, &plan))) return st;
  if (plan.workspace_bytes > 0 && (!workspace || workspace_bytes < plan.workspace_bytes ||
                                   (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return DECODE_ATTN_ERR_WORKSPACE;
  return run_chunk(p, plan, total_queries, q, k_pages, v_pages, page_table, query_offsets,
                   seq_lens, out, workspace, err_flag, static_cast<cudaStream_t>(stream));
}
