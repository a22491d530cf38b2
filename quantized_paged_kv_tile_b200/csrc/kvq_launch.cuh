// Launches of a call's second kernel.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace kvq {

// Launch `kernel` so that it may be set up while the kernel before it in the
// stream still runs (programmatic stream serialization): its blocks start as
// that one's end and wait in cudaGridDependencySynchronize(), which every
// block calls before it reads what that kernel wrote and before it returns.
// Against a plain launch, calls in a row: a prompt with masses of 2048 tokens, 8
// heads over 2, 38 instead of 42 to 45 us; a decode with masses of 16 sequences
// of 2000, 8 heads over 4, 45.3 instead of 47.6.  Replayed from a graph the two
// are equal (41.2 and 41.3 us).
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t s, Args&&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, std::forward<Args>(args)...);
}

}  // namespace kvq
