// early_launch.cuh -- a kernel's shared-memory limit, and launches whose set-up overlaps the end of
// the work before them in the stream (programmatic stream serialization): the kernel may come up
// early and has to call wait_for_stream() before it touches global memory.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace pa {

// Returns once the kernels before this one in the stream have completed and their writes are
// visible.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr int kMaxLaunchDevices = 64;
// The most dynamic shared memory that a decode plan asks for: 227 KB less the kernel's own barriers.
constexpr int kMaxDecodeSmem = 232448 - 1024;

// Raises a kernel's shared-memory limit once per device. All launches of a kernel name the same
// limit: with limits of their own, two first calls at once could leave the smaller one in force.
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int smem, std::atomic<bool> (&set)[kMaxLaunchDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxLaunchDevices || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxLaunchDevices) set[dev].store(true, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, int smem,
                         cudaStream_t stream, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // reported here, not by a later call
  return e;
}

}  // namespace pa
