// launch.cuh -- launches that overlap the end of the kernel before them on the stream.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace haste {

// Returns once everything before this kernel on its stream is complete and visible.
// A kernel launched with launch_early calls it before it touches memory that others
// write or read.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's CTAs move in once all of this kernel's have started; they
// wait in wait_for_stream until this kernel is complete.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// A launch that may begin before the kernel before it has ended (the kernel waits
// for that itself, griddepcontrol.wait).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Sets a kernel's attribute once per device.
inline cudaError_t set_once(std::atomic<uint64_t>& done, const void* kern, cudaFuncAttribute attr, int value) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, attr, value);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

}  // namespace haste
