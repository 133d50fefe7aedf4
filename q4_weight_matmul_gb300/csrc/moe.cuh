// What the kernels of a layer with routed experts share: the plan, the tiles
// of pairs that share an expert, and launches that overlap the end of the one
// before.
#pragma once

#include "q4k_internal.h"

#include <cstdint>

namespace q4k {

// `kernel` on `s`; it may start while the launch before it ends, and waits for
// that launch's results itself (griddepcontrol.wait).
template <class K, class... A>
inline cudaError_t launch_after(K* kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace q4k
