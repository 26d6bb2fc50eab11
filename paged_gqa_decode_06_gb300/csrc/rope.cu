// decode_rope_freqs, decode_rope_table, decode_rope: the frequencies of rotary
// positions (on the host), their table of cosines and sines, and rows rotated
// by it.
//
// The rotation moves memory: each value is read and written once, a table row
// once per position.  A thread takes one unit of 16 values (rope.cuh) of two
// neighbouring heads, so that four 16-byte loads are in flight before its
// position's table row, which the two share.  A prompt of 8192 positions of 32 heads
// of 128, called run after run: 22.3 us (6.2 TB/s), DRAM.  (Replayed on the same rows
// 17.6 us, less than DRAM allows: L2 holds part of them.)
#include <cmath>

#include "chunk_launch.h"
#include "host_common.h"
#include "ragged.cuh"
#include "rope.cuh"

namespace pgd {
namespace {

constexpr int kThreads = 256;

struct RopeRows {
  RopeArgs rope;
  const void* x;
  void* out;
  const int32_t* positions;
  int32_t* err;
  int64_t x_stride, out_stride;  // in 8-value items
  int32_t rows, heads, units;    // units of 16 values in a head
  int64_t items;                 // rows * pairs of heads * units
  FastDiv by_unit, by_pair;
};

template <class E>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const RopeRows a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (e >= a.items) return;
  const int pair = (int)a.by_unit.div((uint32_t)e), unit = (int)e - pair * a.units;
  const int row = (int)a.by_pair.div(pair), h = 2 * (pair - row * (int)a.by_pair.d);
  const int2 item = rope_items(a.rope, unit);
  const int per_head = 2 * a.units;
  const bool two = h + 1 < a.heads;
  const uint4* src = static_cast<const uint4*>(a.x) + row * a.x_stride + h * per_head;
  uint4 x[2][2] = {};
  x[0][0] = __ldcs(src + item.x);
  x[0][1] = __ldcs(src + item.y);
  if (two) {
    x[1][0] = __ldcs(src + per_head + item.x);
    x[1][1] = __ldcs(src + per_head + item.y);
  }
  const int pos = ld_global_s32(a.positions + row);
  if (pos < 0 || pos >= a.rope.rows) {
    if (h == 0 && unit == 0) raise_error(a.err, DECODE_ATTN_DEV_BAD_LEN);
    x[0][0] = x[0][1] = x[1][0] = x[1][1] = make_uint4(0u, 0u, 0u, 0u);
  } else if (16 * unit < a.rope.rot) {
    RopePairs p;
    rope_load(p, a.rope, pos, unit);
    rope_unit<E>(x[0][0], x[0][1], p, a.rope.interleaved);
    rope_unit<E>(x[1][0], x[1][1], p, a.rope.interleaved);
  }
  uint4* dst = static_cast<uint4*>(a.out) + row * a.out_stride + h * per_head;
  dst[item.x] = x[0][0];
  dst[item.y] = x[0][1];
  if (two) {
    dst[per_head + item.x] = x[1][0];
    dst[per_head + item.y] = x[1][1];
  }
}

// A thread per frequency and position.  The 64-bit sine and cosine bound it (131072
// positions of 128 dims 472 us; writing them would take 9.9): the angles of far
// positions need the bits, and a table is made once.
__global__ void __launch_bounds__(kThreads)
    rope_table_kernel(const double* inv_freq, int half, int positions, double amplitude,
                      float* table) {
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (e >= (int64_t)positions * half) return;
  const int64_t p = e / half;
  const int i = (int)(e - p * half);
  double s, c;
  sincos((double)p * inv_freq[i], &s, &c);
  float* row = table + p * 2 * half;
  row[i] = (float)(amplitude * c);
  row[half + i] = (float)(amplitude * s);
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" int decode_rope_freqs(const decode_rope_scaling* s, int32_t rot_dim, double base,
                                 double* inv_freq, double* amplitude) {
  if (!inv_freq || !amplitude) return DECODE_ATTN_ERR_NULL;
  const int kind = s ? s->kind : DECODE_ROPE_SCALE_NONE;
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 65536 || !(base > 1.0) || !std::isfinite(base) ||
      kind < DECODE_ROPE_SCALE_NONE || kind > DECODE_ROPE_SCALE_WAVELENGTH)
    return DECODE_ATTN_ERR_SHAPE;
  const double pi2 = 6.283185307179586476925286766559;
  const double f = s && kind ? s->factor : 1.0;
  double slow = 0, fast = 0, len = 0;
  if (kind && (!(f >= 1.0) || !std::isfinite(f))) return DECODE_ATTN_ERR_SHAPE;
  if (kind == DECODE_ROPE_SCALE_NTK) {
    if (rot_dim < 4) return DECODE_ATTN_ERR_SHAPE;
    base *= std::pow(f, (double)rot_dim / (rot_dim - 2));
    if (!std::isfinite(base)) return DECODE_ATTN_ERR_SHAPE;
  }
  if (kind == DECODE_ROPE_SCALE_YARN || kind == DECODE_ROPE_SCALE_WAVELENGTH) {
    const bool yarn = kind == DECODE_ROPE_SCALE_YARN;
    len = s->original_len;
    slow = s->low > 0 ? s->low : 1.0;
    fast = s->high > 0 ? s->high : yarn ? 32.0 : 4.0;
    if (!(len >= 1.0) || !std::isfinite(len) || !(fast > slow) || !std::isfinite(fast))
      return DECODE_ATTN_ERR_SHAPE;
  }
  // the dim whose pair turns `turns` times over the original length
  const auto dim_of = [&](double turns) {
    return rot_dim * std::log(len / (turns * pi2)) / (2.0 * std::log(base));
  };
  double lo = 0, hi = 0;
  if (kind == DECODE_ROPE_SCALE_YARN) {
    lo = std::fmax(std::floor(dim_of(fast)), 0.0);
    hi = std::fmin(std::ceil(dim_of(slow)), rot_dim - 1.0);
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rot_dim);
    if (kind == DECODE_ROPE_SCALE_LINEAR) {
      w /= f;
    } else if (kind == DECODE_ROPE_SCALE_YARN) {
      const double ramp = std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);
      w = w * (1.0 - ramp) + w / f * ramp;
    } else if (kind == DECODE_ROPE_SCALE_WAVELENGTH) {
      const double turns = len * w / pi2;  // over the original length
      const double keep = std::fmin(std::fmax((turns - slow) / (fast - slow), 0.0), 1.0);
      w = w * keep + w / f * (1.0 - keep);
    }
    inv_freq[i] = w;
  }
  *amplitude = kind == DECODE_ROPE_SCALE_YARN ? 0.1 * std::log(f) + 1.0 : 1.0;
  return DECODE_ATTN_OK;
}

extern "C" int decode_rope_table(const double* inv_freq, int32_t rot_dim, int32_t num_positions,
                                 double amplitude, float* table, void* stream) {
  if (rot_dim < 16 || rot_dim % 16 || rot_dim > 512 || num_positions < 0 ||
      !std::isfinite(amplitude))
    return DECODE_ATTN_ERR_SHAPE;
  if (num_positions == 0) return DECODE_ATTN_OK;
  if (!inv_freq || !table) return DECODE_ATTN_ERR_NULL;
  if (!aligned16(inv_freq) || !aligned16(table)) return DECODE_ATTN_ERR_ALIGN;
  const int64_t blocks = ceil_div((int64_t)num_positions * (rot_dim / 2), kThreads);
  if (blocks > INT32_MAX) return DECODE_ATTN_ERR_SHAPE;
  rope_table_kernel<<<(unsigned)blocks, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      inv_freq, rot_dim / 2, num_positions, amplitude, table);
  return cuda_status(cudaGetLastError());
}

extern "C" int decode_rope(const decode_rope_params* p, const void* x, int64_t x_stride,
                           const int32_t* positions, const float* table, void* out,
                           int64_t out_stride, int32_t* err_flag, void* stream) {
  if (!p) return DECODE_ATTN_ERR_NULL;
  if (p->rows < 0 || p->heads <= 0 || p->head_dim < 16 || p->head_dim % 16 ||
      p->head_dim > 512 || p->rot_dim < 16 || p->rot_dim % 16 || p->rot_dim > p->head_dim ||
      p->table_rows <= 0 || (p->dtype != DECODE_ATTN_DTYPE_FP16 &&
                             p->dtype != DECODE_ATTN_DTYPE_BF16))
    return DECODE_ATTN_ERR_SHAPE;
  const int64_t width = (int64_t)p->heads * p->head_dim;
  if (x_stride == 0) x_stride = width;
  if (out_stride == 0) out_stride = width;
  if (x_stride < width || out_stride < width) return DECODE_ATTN_ERR_SHAPE;
  if (x_stride % 8 || out_stride % 8) return DECODE_ATTN_ERR_ALIGN;
  RopeRows a{};
  a.units = p->head_dim / 16;
  const int32_t pairs = p->heads / 2 + p->heads % 2;
  a.items = (int64_t)p->rows * pairs * a.units;
  if (a.items > INT32_MAX) return DECODE_ATTN_ERR_SHAPE;
  if (p->rows == 0) return DECODE_ATTN_OK;
  if (!x || !positions || !table || !out) return DECODE_ATTN_ERR_NULL;
  if (!aligned16(x) || !aligned16(table) || !aligned16(out)) return DECODE_ATTN_ERR_ALIGN;
  a.rope = RopeArgs{table, p->table_rows, p->rot_dim, p->interleaved != 0, p->backward != 0};
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.err = err_flag;
  a.x_stride = x_stride / 8;
  a.out_stride = out_stride / 8;
  a.rows = p->rows;
  a.heads = p->heads;
  a.by_unit = FastDiv::of(a.units);
  a.by_pair = FastDiv::of(pairs);
  static std::atomic<uint64_t> done{0};
  const unsigned blocks = (unsigned)ceil_div(a.items, kThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(p->dtype == DECODE_ATTN_DTYPE_BF16
                         ? launch_pdl(rope_rows_kernel<__nv_bfloat16>, done, blocks, kThreads, 0,
                                      s, a)
                         : launch_pdl(rope_rows_kernel<__half>, done, blocks, kThreads, 0, s, a));
}
