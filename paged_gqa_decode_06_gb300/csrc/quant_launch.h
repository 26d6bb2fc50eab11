// Host-side interface between decode_attn_quant (quant_api.cu) and the
// per-head-dim translation units that instantiate its kernel.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "quant_split.cuh"

namespace pgd {

struct QuantLaunch {
  CUtensorMap tmap_k, tmap_v;
  QuantArgs args;
  dim3 grid;
  int group_pad;  // 8 or 16 query rows per KV row
  int dtype;
  int cluster;    // > 0: CTAs per cluster along x
  cudaStream_t stream;
};

cudaError_t launch_quant_d64(const QuantLaunch& L);
cudaError_t launch_quant_d128(const QuantLaunch& L);
cudaError_t launch_quant_d256(const QuantLaunch& L);

}  // namespace pgd
