// Launches whose start overlaps the end of the launch before them on the stream.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace flce {
namespace {

// In the earlier kernel: the next launch may start as soon as there is room for it.
__device__ __forceinline__ void start_next_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// In the later kernel, before it touches what earlier launches read or write: waits until
// the launch before it has ended and its writes are visible.
__device__ __forceinline__ void wait_for_launch_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches a kernel that calls wait_for_launch_before().
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         A&&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace
}  // namespace flce
