// What the kernels of a layer with routed experts share: launches that overlap
// the end of the one before, waits, sums over a block.
#pragma once

#include "q4k_internal.h"
#include "tc_ptx.cuh"

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

// v / (1 + exp(-v)), within some 2e-6 of it where it is not negligible; 0 for
// v far below 0 (exp(-v) infinite).
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

// A warp agrees on a wait's outcome, so that its lanes stay together; one that
// gives up raises the block's flag and the device error word.
__device__ __forceinline__ bool agreed(bool ok, volatile int* gave_up, int* err) {
  if (__all_sync(~0u, ok)) return true;
  if ((threadIdx.x & 31) == 0) {
    if (!*gave_up) atomicOr(err, 1);
    *gave_up = 1;
  }
  __syncwarp();
  return false;
}
// (Short: the code of a warp's loop is fetched anew for every turn where the
// warps of a block do different things.)
template <long long kTimeoutCycles = tc::kTimeoutCycles>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* gave_up, int* err) {
  if (__all_sync(~0u, tc::mbar_try_wait(bar, parity))) return true;
  const uint32_t t0 = (uint32_t)(clock64() >> 16);
  while (!__all_sync(~0u, tc::mbar_try_wait(bar, parity)))
    if (!agreed(!*gave_up && (uint32_t)(clock64() >> 16) - t0 < (uint32_t)(kTimeoutCycles >> 16), gave_up, err)) return false;
  return true;
}

// Two barriers, asked together at first.
template <long long kTimeoutCycles = tc::kTimeoutCycles>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2,
                                          volatile int* gave_up, int* err) {
  if (__all_sync(~0u, tc::mbar_try_wait(bar, parity) & tc::mbar_try_wait(bar2, parity2))) return true;
  return warp_wait<kTimeoutCycles>(bar, parity, gave_up, err) && warp_wait<kTimeoutCycles>(bar2, parity2, gave_up, err);
}

using tc::warp_release;

// Exclusive sum of `v` over the block's threads before this one (`most`:
// maximum in place of a sum); every thread gets the whole block's in `all`.
template <int THREADS, bool MOST>
__device__ __forceinline__ int scan_block(int v, int* warps, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int u = __shfl_up_sync(~0u, s, o);
    if (lane >= o) s = MOST ? max(s, u) : s + u;
  }
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int u = warps[w];
    if (w < warp) before = MOST ? max(before, u) : before + u;
    all = MOST ? max(all, u) : all + u;
  }
  const int u = __shfl_up_sync(~0u, s, 1);
  if (lane > 0) before = MOST ? max(before, u) : before + u;
  __syncthreads();
  return before;
}

}  // namespace q4k
