// Host helpers of the entry points outside api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/decode_attn.h"

namespace pgd {

// The argument checks decode_attn_make_plan starts with (api.cu): shapes,
// head dim, page size, group, dtype, schedule; no device call.
int validate_params(const decode_attn_params* p);

// Bytes of the shard tickets at the start of a workspace, 64 KiB or more, and
// the clearing of a call's tickets beyond 64 KiB, where other calls keep
// partials (api.cu).
size_t ticket_bytes(const decode_attn_params* p);
int clear_far_tickets(void* tickets, int64_t groups, cudaStream_t stream);

// SM count of a device, looked up once.
int device_sms(int device, int* sms);

// A positive integer from the environment, read on every call; else 0.
int env_positive(const char* name);

// A tiled tensor map with the 128-byte swizzle (or 64-byte, when the inner
// extent of the box is 64 bytes), zero fill outside the tensor.
int encode_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
               const uint64_t* dims, const uint64_t* strides, const uint32_t* box);

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0; }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t ceil_div(int64_t x, int64_t m) { return (x + m - 1) / m; }
inline int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}
inline int cuda_status(cudaError_t e) {
  return e == cudaSuccess ? DECODE_ATTN_OK : DECODE_ATTN_ERR_CUDA;
}

}  // namespace pgd
