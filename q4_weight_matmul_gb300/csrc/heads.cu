// q4k_qk_norm_rope: per-head RMS norm and rotation of queries and keys, and
// the store of keys and values into the paged cache.
//
// A row is one head of one token: 4 D bytes in, 2 D bytes out, and some ten
// instructions per 16 bytes between them, so HBM bounds it as long as the
// instructions stay few.  D/8 lanes share a row, each with 4 values of its
// lower half and the 4 at the same place of its upper half (16-byte loads,
// 8-byte stores): where the whole head is rotated by halves (kWhole), or
// neighbours are (kNeighbours), a lane then has both values of its pairs, and
// only the sum of squares crosses lanes.  Rotating a part of the head by
// halves (kPart) takes the partner's value from another lane.  A warp takes kLoads rows per group of
// lanes, all of one token, with their loads in flight at once, and reads the
// token's cosines and sines once for all of them.
//
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128, bfloat16: 54.2 us, 5.6
// TB/s (85 % of the copy rate; two rows' worth of lanes per row, so that the
// pairs of a rotation by halves met across lanes, took 97 us: 67 % of the
// issue slots).  One token: 2.7 us.
#include "q4k_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace q4k {
namespace {

constexpr int kLoads = 4;   // rows in flight per group of lanes

template <bool BF16>
__device__ __forceinline__ uint2 pack4(const float4& v) {
  uint2 r;
  if constexpr (BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    r.x = *reinterpret_cast<const uint32_t*>(&a), r.y = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    r.x = *reinterpret_cast<const uint32_t*>(&a), r.y = *reinterpret_cast<const uint32_t*>(&b);
  }
  return r;
}

__device__ __forceinline__ float4 mul(const float4& a, const float4& b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 mul(const float4& a, float b) { return make_float4(a.x * b, a.y * b, a.z * b, a.w * b); }
// a b + c d
__device__ __forceinline__ float4 mul2(const float4& a, const float4& b, const float4& c, const float4& d) {
  return make_float4(fmaf(a.x, b.x, c.x * d.x), fmaf(a.y, b.y, c.y * d.y), fmaf(a.z, b.z, c.z * d.z),
                     fmaf(a.w, b.w, c.w * d.w));
}
__device__ __forceinline__ float squares(const float4& a) { return a.x * a.x + a.y * a.y + (a.z * a.z + a.w * a.w); }

enum Mode { kWhole, kNeighbours, kPart };

template <int D, bool BF16, Mode MODE>
__global__ void __launch_bounds__(256, 3) qk_norm_rope_kernel(const HeadsParams P, int page_shift) {
  constexpr int kLanes = D / 8;             // lanes of a row
  constexpr int kPerLoad = 32 / kLanes;     // rows of one warp-wide load
  constexpr int kRows = kLoads * kPerLoad;
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  const int rows = P.heads + 2 * P.kv_heads, groups = (rows + kRows - 1) / kRows;
  const int task = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int t = task / groups, first = (task - t * groups) * kRows + sub;
  if (t >= P.tokens) return;                // whole warps leave

  const float* q = P.q + (int64_t)t * P.heads * D + 4 * l;
  const float* k = P.k + (int64_t)t * P.kv_heads * D + 4 * l;
  const float* v = P.v + (int64_t)t * P.kv_heads * D + 4 * l;
  float4 lo[kLoads], hi[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = first + i * kPerLoad, rk = r - P.heads, rv = rk - P.kv_heads;
    const float* src = rk < 0 ? q + r * D : rv < 0 ? k + rk * D : v + rv * D;
    if (r < rows) {
      lo[i] = *reinterpret_cast<const float4*>(src);
      hi[i] = *reinterpret_cast<const float4*>(src + D / 2);
    } else {
      lo[i] = hi[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }

  // where the token's key and value go, and whether its indices are in range
  int slot = P.slot[t], pos = 0;
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
  const int page = slot >> page_shift, cell = slot & (P.page_size - 1);

  // factors of the lane's values (c) and of their partners (s), lower and upper half, where those are rotated (the
  // others are left alone, not multiplied by 1 and 0: an infinity would make its neighbour, or itself, NaN)
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 c0 = zero, s0 = zero, c1 = zero, s1 = zero;
  const bool turn0 = MODE == kWhole ? P.rot != 0 : 4 * l < P.rot, turn1 = 4 * l + D / 2 < P.rot;
  const float* cs = P.cos_sin + (int64_t)pos * P.rot;
  const int half = P.rot / 2;
  int from0 = lane, from1 = lane;           // kPart: the lanes of the partners,
  bool up0 = false, up1 = false;            // and in which of its halves they are
  if constexpr (MODE == kWhole) {
    if (P.rot) {
      c0 = *reinterpret_cast<const float4*>(cs + 4 * l);
      s0 = *reinterpret_cast<const float4*>(cs + D / 2 + 4 * l);
    }
  } else if constexpr (MODE == kNeighbours) {
    auto factors = [&](int i, float4& c, float4& s) {      // values i .. i+3
      if (i >= P.rot) return;
      const float2 cc = *reinterpret_cast<const float2*>(cs + i / 2), ss = *reinterpret_cast<const float2*>(cs + half + i / 2);
      c = make_float4(cc.x, cc.x, cc.y, cc.y);
      s = make_float4(-ss.x, ss.x, -ss.y, ss.y);
    };
    factors(4 * l, c0, s0);
    factors(4 * l + D / 2, c1, s1);
  } else {
    auto factors = [&](int i, float4& c, float4& s, int& from, bool& up) {
      if (i >= P.rot) return;
      const int pair = i < half ? i : i - half, partner = i < half ? i + half : i - half;
      c = *reinterpret_cast<const float4*>(cs + pair);
      s = *reinterpret_cast<const float4*>(cs + half + pair);
      if (i < half) s = mul(s, -1.f);
      up = partner >= D / 2;
      from = sub * kLanes + (partner - (up ? D / 2 : 0)) / 4;
    };
    factors(4 * l, c0, s0, from0, up0);
    factors(4 * l + D / 2, c1, s1, from1, up1);
  }
  const bool norm = P.q_weight != nullptr;
  uint16_t* q_out = static_cast<uint16_t*>(P.q_out) + (int64_t)t * P.heads * D + 4 * l;
  const int64_t cell_at = (((int64_t)page * P.kv_heads) * P.page_size + cell) * D + 4 * l;
  const int head_step = P.page_size * D;

#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = first + i * kPerLoad, rk = r - P.heads, rv = rk - P.kv_heads;
    float4 x = lo[i], y = hi[i];
    // rows of one load may be of two kinds where the head counts are odd, so the lanes meet before they part
    float sum = 0.f;
    if (norm) {
      sum = squares(x) + squares(y);
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (norm && rv < 0) {
      const float inv = rsqrtf(fmaf(sum, 1.0f / D, P.eps));
      const float* w = (rk < 0 ? P.q_weight : P.k_weight) + 4 * l;     // few lines, in L1 after the first rows
      x = mul(mul(x, inv), __ldg(reinterpret_cast<const float4*>(w)));
      y = mul(mul(y, inv), __ldg(reinterpret_cast<const float4*>(w + D / 2)));
    }
    float4 px, py;
    if constexpr (MODE == kPart) {
      auto partner = [&](float a, float b, int from, bool up) {
        const float u = __shfl_sync(0xffffffffu, a, from), w = __shfl_sync(0xffffffffu, b, from);
        return up ? w : u;
      };
      px = make_float4(partner(x.x, y.x, from0, up0), partner(x.y, y.y, from0, up0), partner(x.z, y.z, from0, up0),
                       partner(x.w, y.w, from0, up0));
      py = make_float4(partner(x.x, y.x, from1, up1), partner(x.y, y.y, from1, up1), partner(x.z, y.z, from1, up1),
                       partner(x.w, y.w, from1, up1));
    }
    if (r >= rows) continue;
    uint16_t* dst;
    if (rv < 0) {
      if constexpr (MODE == kWhole) {
        if (turn0) {
          px = mul2(x, c0, mul(y, -1.f), s0);
          y = mul2(y, c0, x, s0);
          x = px;
        }
      } else {
        if constexpr (MODE == kNeighbours)
          px = make_float4(x.y, x.x, x.w, x.z), py = make_float4(y.y, y.x, y.w, y.z);
        if (turn0) x = mul2(x, c0, px, s0);
        if (turn1) y = mul2(y, c1, py, s1);
      }
      dst = rk < 0 ? q_out + r * D : static_cast<uint16_t*>(P.k_cache) + cell_at + (int64_t)rk * head_step;
    } else {
      dst = static_cast<uint16_t*>(P.v_cache) + cell_at + (int64_t)rv * head_step;
    }
    if (rk >= 0 && slot < 0) continue;
    *reinterpret_cast<uint2*>(dst) = pack4<BF16>(x);
    *reinterpret_cast<uint2*>(dst + D / 2) = pack4<BF16>(y);
  }
}

template <int D, bool BF16>
void launch(const HeadsParams& p, int page_shift, unsigned grid, int threads, cudaStream_t s) {
  if (p.rot == 0 || (p.rot == D && !p.interleaved))
    qk_norm_rope_kernel<D, BF16, kWhole><<<grid, threads, 0, s>>>(p, page_shift);
  else if (p.interleaved)
    qk_norm_rope_kernel<D, BF16, kNeighbours><<<grid, threads, 0, s>>>(p, page_shift);
  else
    qk_norm_rope_kernel<D, BF16, kPart><<<grid, threads, 0, s>>>(p, page_shift);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const HeadsParams& p, cudaStream_t s) {
  const int per = kLoads * (256 / p.dim);
  const int64_t tasks = p.tokens * ((p.heads + 2 * p.kv_heads + per - 1) / per);
  // few tasks: one warp per CTA, so that they spread over the SMs
  const int warps = tasks <= 152 * 4 ? 1 : 8;
  const int64_t grid = (tasks + warps - 1) / warps;
  if (tasks > 0x7ffffff0) return cudaErrorInvalidValue;
  int page_shift = 4;
  while ((1 << page_shift) < p.page_size) ++page_shift;
  if (p.dim == 128) {
    if (p.bf16) launch<128, true>(p, page_shift, (unsigned)grid, 32 * warps, s);
    else launch<128, false>(p, page_shift, (unsigned)grid, 32 * warps, s);
  } else {
    if (p.bf16) launch<64, true>(p, page_shift, (unsigned)grid, 32 * warps, s);
    else launch<64, false>(p, page_shift, (unsigned)grid, 32 * warps, s);
  }
  return cudaGetLastError();
}

}  // namespace q4k
