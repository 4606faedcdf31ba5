// Launching the kernels of h3attn_lowp.h: what the host would otherwise ask the runtime
// on every call is kept per kernel and device, and every launch may begin before the
// work ahead of it in the stream is done (programmatic dependent launch): the kernels
// set up barriers and tensor memory first and read or write no global memory before
// pdl_wait() (a prefetch into L2 aside).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.hpp"

namespace h3 {

constexpr int kLaunchDevices = 64;

// Per kernel (a function-local static of its launcher).  Threads that race write the same
// values.
struct KernelState {
  std::atomic<uint64_t> smem_set{0};                  // devices whose limit is raised
  std::atomic<uint64_t> occupancy[kLaunchDevices]{};  // last answer: smem << 24 | threads << 8 | CTAs an SM
  std::atomic<int> clusters[kLaunchDevices]{};        // resident clusters
};

// Allows the kernel `bytes` of dynamic shared memory; the same `bytes` on every call.
template <class Kernel>
cudaError_t allow_smem(KernelState* s, Kernel kern, size_t bytes, const DevCtx& ctx) {
  const uint64_t bit = uint64_t(1) << ctx.dev;
  if (s->smem_set.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess) s->smem_set.fetch_or(bit, std::memory_order_release);
  return e;
}

// CTAs that fit an SM, at least 1.
template <class Kernel>
cudaError_t ctas_per_sm(KernelState* s, Kernel kern, int threads, size_t smem, const DevCtx& ctx,
                        int* per_sm) {
  const uint64_t key = uint64_t(smem) << 24 | uint64_t(threads) << 8;
  const uint64_t last = s->occupancy[ctx.dev].load(std::memory_order_relaxed);
  if (last != 0 && (last & ~uint64_t(255)) == key) {
    *per_sm = int(last & 255);
    return cudaSuccess;
  }
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, kern, threads, smem);
  if (e != cudaSuccess) return e;
  if (*per_sm < 1) *per_sm = 1;
  s->occupancy[ctx.dev].store(key | uint64_t(*per_sm), std::memory_order_relaxed);
  return cudaSuccess;
}

struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  Launch(unsigned grid, int threads, size_t smem, cudaStream_t st, int cluster = 1) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
  Launch(const Launch&) = delete;   // cfg points into the object
  Launch& operator=(const Launch&) = delete;
};

}  // namespace h3
