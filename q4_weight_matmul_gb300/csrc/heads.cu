// q4k_qk_norm_rope: per-head RMS norm and rotation of queries and keys, and
// the store of keys and values into the paged cache.
//
// A row is one head of one token: 4 D bytes in, 2 D bytes out, and about six
// operations a value between them, so HBM bounds it.  D/4 lanes share a row
// (16-byte loads, 8-byte stores); a warp takes kRows row slots of one token
// and has all their loads in flight at once, together with the token's
// cosines and sines, which it then uses for every row.  A row's rotation
// partner sits rot/8 lanes away (or in the same lane when interleaved).
#include "q4k_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace q4k {
namespace {

constexpr int kLoads = 4;   // row loads in flight per lane

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const HeadsParams P) {
  constexpr int kLanes = D / 4;             // lanes of a row
  constexpr int kPerLoad = 32 / kLanes;     // rows of one warp-wide load
  constexpr int kRows = kLoads * kPerLoad;
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  const int rows = P.heads + 2 * P.kv_heads;
  const int groups = (rows + kRows - 1) / kRows;
  const int64_t task = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (task >= P.tokens * groups) return;    // whole warps leave
  const int64_t t = task / groups;
  const int first = (int)(task - t * groups) * kRows + sub;

  float4 x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = first + i * kPerLoad;
    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= rows) continue;
    const float* src;
    if (r < P.heads) src = P.q + (t * P.heads + r) * D;
    else if (r < P.heads + P.kv_heads) src = P.k + (t * P.kv_heads + (r - P.heads)) * D;
    else src = P.v + (t * P.kv_heads + (r - P.heads - P.kv_heads)) * D;
    x[i] = reinterpret_cast<const float4*>(src)[l];
  }

  // where the token's key and value go, and whether its indices are in range
  int64_t slot = P.slot[t];
  int pos = 0;
  if (P.rot) {
    pos = P.pos[t];
    if (pos < 0 || pos >= P.max_pos) {
      if (lane == 0) atomicOr(P.err, kErrIndex);
      return;
    }
  }
  if (slot >= P.num_slots) {
    if (lane == 0) atomicOr(P.err, kErrIndex);
    slot = -1;
  }
  const int64_t page = slot / P.page_size;
  const int cell = (int)(slot - page * P.page_size);

  // the lane's four angles: values 4l..4l+3 of pair index 4l mod rot/2, or
  // pairs 2l and 2l+1 when interleaved
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  int partner = lane;
  if (4 * l < P.rot) {
    const float* row = P.cos_sin + (int64_t)pos * P.rot;
    const int half = P.rot / 2;
    if (P.interleaved) {
      const float2 cc = *reinterpret_cast<const float2*>(row + 2 * l);
      const float2 ss = *reinterpret_cast<const float2*>(row + half + 2 * l);
      c = make_float4(cc.x, cc.x, cc.y, cc.y);
      s = make_float4(-ss.x, ss.x, -ss.y, ss.y);
    } else {
      const bool low = 4 * l < half;
      const int i = low ? 4 * l : 4 * l - half;
      c = *reinterpret_cast<const float4*>(row + i);
      s = *reinterpret_cast<const float4*>(row + half + i);
      if (low) s = make_float4(-s.x, -s.y, -s.z, -s.w);
      partner = low ? lane + P.rot / 8 : lane - P.rot / 8;
    }
  }
  const bool norm = P.q_weight != nullptr;
  float4 wq = make_float4(1.f, 1.f, 1.f, 1.f), wk = wq;
  if (norm) {
    wq = reinterpret_cast<const float4*>(P.q_weight)[l];
    wk = reinterpret_cast<const float4*>(P.k_weight)[l];
  }

#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = first + i * kPerLoad;
    float4 v = x[i];
    const bool value_row = r >= P.heads + P.kv_heads;
    if (norm) {
      float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!value_row) {
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + P.eps);
        const float4 w = r < P.heads ? wq : wk;
        v = make_float4(v.x * inv * w.x, v.y * inv * w.y, v.z * inv * w.z, v.w * inv * w.w);
      }
    }
    if (P.rot) {
      float4 o;
      if (P.interleaved) {
        o = make_float4(v.y, v.x, v.w, v.z);
      } else {
        o.x = __shfl_sync(0xffffffffu, v.x, partner);
        o.y = __shfl_sync(0xffffffffu, v.y, partner);
        o.z = __shfl_sync(0xffffffffu, v.z, partner);
        o.w = __shfl_sync(0xffffffffu, v.w, partner);
      }
      if (!value_row && 4 * l < P.rot)
        v = make_float4(v.x * c.x + o.x * s.x, v.y * c.y + o.y * s.y, v.z * c.z + o.z * s.z, v.w * c.w + o.w * s.w);
    }
    if (r >= rows) continue;
    uint16_t* dst;
    if (r < P.heads) {
      dst = static_cast<uint16_t*>(P.q_out) + (t * P.heads + r) * D;
    } else {
      if (slot < 0) continue;
      const int h = value_row ? r - P.heads - P.kv_heads : r - P.heads;
      dst = static_cast<uint16_t*>(value_row ? P.v_cache : P.k_cache) +
            ((page * P.kv_heads + h) * P.page_size + cell) * D;
    }
    reinterpret_cast<uint2*>(dst)[l] = make_uint2(pack2<BF16>(v.x, v.y), pack2<BF16>(v.z, v.w));
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const HeadsParams& p, cudaStream_t s) {
  const int per = kLoads * (128 / p.dim);
  const int64_t tasks = p.tokens * ((p.heads + 2 * p.kv_heads + per - 1) / per);
  // few tasks: one warp per CTA, so that they spread over the SMs
  const int warps = tasks <= 152 * 4 ? 1 : 8;
  const unsigned grid = (unsigned)((tasks + warps - 1) / warps);
  if (p.dim == 128) {
    if (p.bf16) qk_norm_rope_kernel<128, true><<<grid, 32 * warps, 0, s>>>(p);
    else qk_norm_rope_kernel<128, false><<<grid, 32 * warps, 0, s>>>(p);
  } else {
    if (p.bf16) qk_norm_rope_kernel<64, true><<<grid, 32 * warps, 0, s>>>(p);
    else qk_norm_rope_kernel<64, false><<<grid, 32 * warps, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace q4k
