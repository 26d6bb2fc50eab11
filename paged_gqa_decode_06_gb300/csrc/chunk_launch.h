// Host-side interface between the chunk entry points (chunk_api.cu) and the
// per-head-dim translation units that instantiate the chunk kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "chunk_attn.cuh"

namespace pgd {

struct ChunkLaunch {
  CUtensorMap tmap_q, tmap_k, tmap_v;
  ChunkArgs args;
  unsigned grid;          // CTAs of the attention kernel
  unsigned combine_grid;  // CTAs of the merge; 0 for a plan without shards
  int dtype;
  cudaStream_t stream;
};

cudaError_t launch_chunk_d64(const ChunkLaunch& L);
cudaError_t launch_chunk_d128(const ChunkLaunch& L);
cudaError_t launch_chunk_d256(const ChunkLaunch& L);

// Launches `kern` as a programmatic dependent of the preceding kernel on the
// stream; `done` remembers the devices whose shared-memory limit is raised
// already, so that launches under stream capture make no attribute calls.
template <class Kernel, class... Args>
cudaError_t launch_pdl(Kernel kern, std::atomic<uint64_t>& done, unsigned grid, int threads,
                       int smem, cudaStream_t stream, const Args&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (smem > 48 * 1024 && !(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace pgd
