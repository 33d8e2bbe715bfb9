// sv_launch.cuh -- launches whose start overlaps the end of the kernel before
// them in the stream (programmatic dependent launch). A kernel launched so
// calls wait_for_stream() before its first access to global memory: it returns
// when every kernel before it has ended and its writes are visible. It calls
// release_stream() where the next such kernel may be brought up. In a row of
// short calls this hides about a microsecond of each launch.
#pragma once

#include "../../include/spec_verify.h"

#include <atomic>
#include <cuda_runtime.h>

namespace sv {

__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_stream() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Such a kernel may have started while the one before it still wrote, so its
// inputs are not read-only for its lifetime: they are read by ordinary loads
// (not .nc, not __ldg), through a pointer that only exists behind the wait, so
// that no load moves ahead of it.
template <typename T>
__device__ __forceinline__ const T* behind_wait(const T* p) {
  asm volatile("" : "+l"(p)::"memory");
  return p;
}
// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_once16(const void* p) {
  uint4 v;
  asm("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// A call's own status, which is returned; the runtime keeps it too, for the
// next one who asks about errors, unless it is taken back.
inline cudaError_t own_error(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

template <typename... K, typename... A>
cudaError_t launch_overlapped(void (*kernel)(K...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st,
                              A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = at;
  return own_error(cudaLaunchKernelEx(&cfg, kernel, static_cast<K>(args)...));
}

// Allows the kernel that much dynamic shared memory, once per device (`done`
// is the caller's static, a bit a device; devices past 63 ask every time).
template <typename F>
cudaError_t allow_smem(F* kernel, size_t bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = own_error(cudaGetDevice(&dev));
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = own_error(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace sv
