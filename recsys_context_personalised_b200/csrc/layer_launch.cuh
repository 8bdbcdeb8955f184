// Shared by the attention layer's operators (rotary, chunk attention, block norm): launches and their checks.
// Apart from gdpa_internal.cuh, which the GDPA kernels' recorded DRAM traffic is tied to.
#pragma once

#include <atomic>

#include "gdpa_internal.cuh"

namespace gdpa {

// Starts the launch count of an entry point (gdpa_last_launch_count).
void reset_launch_count();
// SMs of the current device.
int device_sm_count();
// Allows `kern` `bytes` of dynamic shared memory, once per device (`done`: a bit for each of the first 64).
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 64;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}
// Checks a paged cache's description for a call on B samples.
gdpa_status_t check_cache(const gdpa_cache_t* c, int32_t B);
inline int log2_int(int x) {
  int n = 0;
  while ((1 << (n + 1)) <= x) ++n;
  return n;
}

// Programmatic dependent launch: a kernel launched with launch_dependent has its blocks scheduled as the kernel
// before it ends (from its pdl_trigger on), and waits (pdl_wait) for that one's completion before it reads
// anything of it.
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace gdpa
