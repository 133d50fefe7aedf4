// q4k_moe_gate_up and q4k_moe_down: products of the experts' quantised
// matrices with the rows of the pairs that chose them.
//
// The simplest form: a CTA takes 8 weight rows (a warp each) of one expert and
// up to 8 of its pairs; a lane dequantises 8 weights of a superblock in fp32
// and multiplies them with each pair's activations.
#include "moe.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace q4k {
namespace {

constexpr int kRows = 8, kPairs = 8, kThreads = 256;

// 8 weights of a Q4_K superblock: 8 * lane .. 8 * lane + 7.
__device__ __forceinline__ void weights_q4(const uint8_t* sb, int lane, float (&w)[8]) {
  const uint4 head = *reinterpret_cast<const uint4*>(sb);
  const float d = __half2float(__ushort_as_half((unsigned short)(head.x & 0xFFFFu))),
              dmin = __half2float(__ushort_as_half((unsigned short)(head.x >> 16)));
  const int j = lane >> 2, shift = 8 * (j & 3);
  uint32_t sc, m;
  if (j < 4) {
    sc = (head.y >> shift) & 63u, m = (head.z >> shift) & 63u;
  } else {
    const uint32_t b = head.w >> shift;
    sc = (b & 15u) | (((head.y >> shift) & 0xC0u) >> 2);
    m = ((b >> 4) & 15u) | (((head.z >> shift) & 0xC0u) >> 2);
  }
  const uint2 q = *reinterpret_cast<const uint2*>(sb + 16 + 32 * (lane >> 3) + 8 * (lane & 3));
  const int nib = (lane & 4) ? 4 : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = ((i < 4 ? q.x : q.y) >> (8 * (i & 3) + nib)) & 15u;
    w[i] = d * (float)sc * (float)v - dmin * (float)m;
  }
}

// 8 weights of a Q6_K superblock (GPU layout) with the row's scale d.
__device__ __forceinline__ void weights_q6(const uint8_t* sb, uint16_t dbits, int lane, float (&w)[8]) {
  const int c = lane >> 3, f = (lane >> 1) & 3, i0 = 8 * (lane & 1);
  const float s = __half2float(__ushort_as_half(dbits)) * (float)(int8_t)sb[lane >> 1];
  const uint8_t* ch = sb + 16 + 48 * c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t lo = (ch[16 * (f & 1) + i0 + i] >> (4 * (f >> 1))) & 15u, hi = ((ch[32 + i0 + i] >> (2 * f)) & 3u) ^ 2u;
    w[i] = s * (float)((int)(lo | (hi << 4)) - 32);
  }
}

template <bool UP, bool Q6>
__global__ void __launch_bounds__(kThreads) moe_simple_kernel(const MoeProduct P, float* out) {
  __shared__ int tile[3];
  const MoePlan& L = P.plan;
  const int64_t pairs = L.tokens * L.top_k;
  if (threadIdx.x == 0) {
    int64_t left = blockIdx.y;
    tile[0] = -1;
    int64_t at = 0;
    for (int e = 0; e < L.experts; ++e) {
      const int64_t a = min(max((int64_t)L.offsets[e], at), pairs), b = min(max((int64_t)L.offsets[e + 1], a), pairs);
      if (a != L.offsets[e] || b != L.offsets[e + 1]) atomicOr(P.err, kErrIndex);
      const int64_t n = (b - a + kPairs - 1) / kPairs;
      if (left < n && tile[0] < 0) {
        tile[0] = e, tile[1] = (int)(a + left * kPairs), tile[2] = (int)min((int64_t)kPairs, b - a - left * kPairs);
      }
      left -= n, at = b;
    }
  }
  __syncthreads();
  const int e = tile[0], first = tile[1], n = tile[2], lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 5);
  if (e < 0 || row >= P.rows) return;
  const int nb = (int)(P.cols / kQK);
  const int64_t pitch = Q6 ? ((int64_t)nb * 210 + 15) / 16 * 16 : (int64_t)nb * kBlockBytes;
  const uint8_t* w = P.w + (e * P.rows + row) * pitch;
  const float* x[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    x[i] = nullptr;
    if (i < n) {
      if constexpr (UP) {
        const int p = L.order[first + i];
        if (p >= 0 && p < pairs) x[i] = P.x + (int64_t)(p / L.top_k) * P.cols;
        else if (lane == 0) atomicOr(P.err, kErrIndex);
      } else {
        x[i] = P.x + (int64_t)(first + i) * P.cols;
      }
    }
  }
  float acc[UP ? 2 : 1][kPairs] = {};
  for (int sb = 0; sb < nb; ++sb) {
    float v[UP ? 2 : 1][8];
    if constexpr (Q6) weights_q6(w + 208 * sb, *reinterpret_cast<const uint16_t*>(w + 208 * nb + 2 * sb), lane, v[0]);
    else weights_q4(w + kBlockBytes * sb, lane, v[0]);
    if constexpr (UP) weights_q4(P.up + (w - P.w) + kBlockBytes * sb, lane, v[1]);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      if (!x[i]) continue;
      const float4* f = reinterpret_cast<const float4*>(x[i] + sb * kQK + 8 * lane);
      const float4 a = f[0], b = f[1];
#pragma unroll
      for (int m = 0; m < (UP ? 2 : 1); ++m)
        acc[m][i] += v[m][0] * a.x + v[m][1] * a.y + v[m][2] * a.z + v[m][3] * a.w + v[m][4] * b.x + v[m][5] * b.y +
                     v[m][6] * b.z + v[m][7] * b.w;
    }
  }
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
#pragma unroll
    for (int m = 0; m < (UP ? 2 : 1); ++m)
#pragma unroll
      for (int o = 16; o > 0; o /= 2) acc[m][i] += __shfl_xor_sync(~0u, acc[m][i], o);
    if (i < n && lane == 0) {
      float r = acc[0][i];
      if constexpr (UP) r = r / (1.0f + expf(-r)) * acc[1][i];
      out[(int64_t)(first + i) * P.rows + row] = r;
    }
  }
}

// y = residual + the weighted rows of z.
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(const MoeProduct P, const float* z) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MoePlan& L = P.plan;
  const int64_t t = blockIdx.x, pairs = L.tokens * L.top_k;
  const int32_t* place = L.place + t * L.top_k;
  if (place[0] == -2) return;
  for (int64_t r = threadIdx.x; r < P.rows; r += kThreads) {
    float y = P.residual ? P.residual[t * P.rows + r] : 0.0f;
    for (int j = 0; j < L.top_k; ++j) {
      const int at = place[j];
      if (at >= 0 && at < pairs) y = fmaf(L.weight[t * L.top_k + j], z[at * P.rows + r], y);
      else if ((at >= pairs || at < -1) && threadIdx.x == 0) atomicOr(P.err, kErrIndex);
    }
    P.out[t * P.rows + r] = y;
  }
}

}  // namespace

size_t moe_gate_up_workspace(int64_t, int, int, int64_t, int64_t) { return 0; }
size_t moe_down_workspace(int64_t tokens, int top_k, int, int64_t rows, int64_t) {
  return sizeof(float) * (size_t)(tokens * top_k) * (size_t)rows;
}

static dim3 simple_grid(const MoeProduct& p) {
  const int64_t pairs = p.plan.tokens * p.plan.top_k;
  return dim3((unsigned)((p.rows + kRows - 1) / kRows), (unsigned)std::min(pairs, pairs / kPairs + p.plan.experts));
}

cudaError_t launch_moe_gate_up(const MoeProduct& p, cudaStream_t s) {
  moe_simple_kernel<true, false><<<simple_grid(p), kThreads, 0, s>>>(p, p.out);
  return cudaGetLastError();
}

cudaError_t launch_moe_down(const MoeProduct& p, cudaStream_t s) {
  float* z = static_cast<float*>(p.workspace);
  if (p.q6k) moe_simple_kernel<false, true><<<simple_grid(p), kThreads, 0, s>>>(p, z);
  else moe_simple_kernel<false, false><<<simple_grid(p), kThreads, 0, s>>>(p, z);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(moe_combine_kernel, dim3((unsigned)p.plan.tokens), kThreads, 0, s, p, (const float*)z);
}

}  // namespace q4k
