// q4k_lora_add: low-rank adapters of many requests beside projections that
// share the input x.  Two launches: h = A x into the workspace, then
// y = base + scale B h.
#include "q4k_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace q4k {
namespace {

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t v) {
  if constexpr (BF16) return __bfloat162float(__ushort_as_bfloat16(v));
  else return __half2float(__ushort_as_half(v));
}

// The token at place i of the order, and its adapter (-1: none); a token of
// -1 is out of range.
__device__ __forceinline__ void place(const LoraParams& P, int64_t i, int& token, int& adapter) {
  int lo = 0, hi = (int)P.n_seg - 1;               // the last segment that starts at or before i
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (P.seg_start[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  token = P.order[i];
  adapter = P.seg_adapter[lo];
  bool bad = adapter >= P.n_adapters;
  if (bad) adapter = -1;
  if (token < 0 || token >= P.tokens) bad = true, token = -1;
  if (bad && threadIdx.x == 0) atomicOr(P.err, kErrIndex);
  if (adapter < 0) adapter = -1;
}

// One warp per value h[place][m][j].
template <bool BF16>
__global__ void lora_shrink_kernel(const LoraParams P) {
  int token, adapter;
  place(P, blockIdx.x, token, adapter);
  if (token < 0 || adapter < 0) return;
  const int lane = threadIdx.x & 31;
  for (int u = threadIdx.x >> 5; u < P.n * P.rank; u += blockDim.x >> 5) {
    const int m = u / P.rank, j = u - m * P.rank;
    const uint16_t* a = static_cast<const uint16_t*>(P.mat[m].a) + ((int64_t)adapter * P.rank + j) * P.cols;
    const float* x = P.x + (int64_t)token * P.cols;
    float s = 0.f;
    for (int64_t k = lane; k < P.cols; k += 32) s = fmaf(to_float<BF16>(a[k]), x[k], s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) P.work[((int64_t)blockIdx.x * P.n + m) * P.rank + j] = s * P.scale[adapter];
  }
}

template <bool BF16>
__global__ void lora_expand_kernel(const LoraParams P) {
  int token, adapter;
  place(P, blockIdx.x, token, adapter);
  if (token < 0) return;
  const LoraMat w = P.mat[blockIdx.y];
  const float* h = P.work + ((int64_t)blockIdx.x * P.n + blockIdx.y) * P.rank;
  for (int64_t o = threadIdx.x; o < w.rows; o += blockDim.x) {
    float s = 0.f;
    if (adapter >= 0) {
      const uint16_t* b = static_cast<const uint16_t*>(w.b) + ((int64_t)adapter * w.rows + o) * P.rank;
      for (int j = 0; j < P.rank; ++j) s = fmaf(to_float<BF16>(b[j]), h[j], s);
    }
    w.y[(int64_t)token * w.rows + o] = s + (w.base ? w.base[(int64_t)token * w.rows + o] : 0.f);
  }
}

}  // namespace

size_t lora_workspace(int n, int rank, int64_t tokens) {
  return sizeof(float) * (size_t)n * (size_t)rank * (size_t)tokens;
}

cudaError_t launch_lora_add(const LoraParams& p, cudaStream_t s) {
  const unsigned t = (unsigned)p.tokens;
  if (p.bf16) lora_shrink_kernel<true><<<t, 256, 0, s>>>(p);
  else lora_shrink_kernel<false><<<t, 256, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(t, p.n);
  if (p.bf16) lora_expand_kernel<true><<<grid, 256, 0, s>>>(p);
  else lora_expand_kernel<false><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace q4k
