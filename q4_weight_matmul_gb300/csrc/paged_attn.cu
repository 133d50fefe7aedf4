// q4k_paged_attn: causal attention of new tokens over the paged cache.
//
// One warp per (token, head): its lanes share the head's values, the keys
// come one after another with the running maximum and sum of their softmax.
#include "q4k_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace q4k {
namespace {

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t v) {
  if constexpr (BF16) return __bfloat162float(__ushort_as_bfloat16(v));
  else return __half2float(__ushort_as_half(v));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) paged_attn_kernel(const AttnParams P) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= P.tokens * P.heads) return;
  const int t = (int)(row / P.heads), h = (int)(row - (int64_t)t * P.heads);
  const int hk = h / (P.heads / P.kv_heads);
  // the request: the last one that starts at or before t
  int lo = 0, hi = (int)P.n_req - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (P.cu_q[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  int64_t kv = P.kv_len[lo];
  const int64_t most = P.max_pages * P.page_size;
  if (kv < 0 || kv > most || P.cu_q[lo] > t || P.cu_q[lo + 1] <= t || P.cu_q[lo + 1] > P.tokens) {
    if (lane == 0) atomicOr(P.err, kErrIndex);
    kv = kv < 0 ? 0 : min(kv, most);
  }
  const int64_t pos = min(kv - (P.cu_q[lo + 1] - t), kv - 1);   // in range whatever cu_q holds
  const int64_t first = P.window ? max((int64_t)0, pos - P.window + 1) : 0;

  float q[E], o[E], ob[E], m = -INFINITY, l = 0.f, lb = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_float<BF16>(static_cast<const uint16_t*>(P.q)[row * D + lane * E + e]) * P.scale;
    o[e] = ob[e] = 0.f;
  }
  for (int64_t j = first; j <= pos; ++j) {
    const int page = P.page_table[lo * P.max_pages + j / P.page_size];
    float kk[E], vv[E];
    const bool ok = page >= 0 && page < P.num_pages;
    if (!ok && lane == 0) atomicOr(P.err, kErrIndex);
    const int64_t at = (((int64_t)page * P.kv_heads + hk) * P.page_size + j % P.page_size) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      kk[e] = ok ? to_float<BF16>(static_cast<const uint16_t*>(P.k_cache)[at + e]) : 0.f;
      vv[e] = ok ? to_float<BF16>(static_cast<const uint16_t*>(P.v_cache)[at + e]) : 0.f;
      s = fmaf(q[e], kk[e], s);
    }
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    const float top = fmaxf(m, s), a = expf(m - top), p = expf(s - top);
    m = top;
    // sums of 64 keys each, added up: a single running sum of a long context would lose bits
    const bool last = (j & 63) == 63 || j == pos;
    lb = lb * a + p;
    l = l * a + (last ? lb : 0.f);
    if (last) lb = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      ob[e] = ob[e] * a + p * vv[e];
      o[e] = o[e] * a + (last ? ob[e] : 0.f);
      if (last) ob[e] = 0.f;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float v = o[e] * inv;
    const int64_t at = row * D + lane * E + e;
    if (P.out_f32) static_cast<float*>(P.out)[at] = v;
    else if constexpr (BF16) static_cast<__nv_bfloat16*>(P.out)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(P.out)[at] = __float2half_rn(v);
  }
}

}  // namespace

size_t paged_attn_workspace(const AttnParams&) { return 16; }

cudaError_t launch_paged_attn(const AttnParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.tokens * p.heads + 3) / 4);
  if (p.dim == 128) {
    if (p.bf16) paged_attn_kernel<128, true><<<grid, 128, 0, s>>>(p);
    else paged_attn_kernel<128, false><<<grid, 128, 0, s>>>(p);
  } else {
    if (p.bf16) paged_attn_kernel<64, true><<<grid, 128, 0, s>>>(p);
    else paged_attn_kernel<64, false><<<grid, 128, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace q4k
