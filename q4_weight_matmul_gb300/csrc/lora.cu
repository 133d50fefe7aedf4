// q4k_lora_add: low-rank adapters of many requests beside projections that
// share the input x, in two launches: h = A x (into the workspace), then
// y = base + scale B h.
//
// Both read their big operands once (x and the A; B, base and y), with a
// handful of operations a byte, so HBM bounds them, or latency when tokens
// are few.  A work item is a tile of 16 tokens of one segment, so tokens that
// share an adapter share its loads; each warp finds its tile from seg_start
// by itself.
//
// Products run on mma.sync m16n8k8 with tf32 operands: the adapters' 16-bit
// values are exact in tf32, and a fp32 activation enters as two parts, hi
// (rounded to 11 bits) + lo (the rest, 11 more bits), so products keep 22
// bits or more over fp32's whole range.  The k index of an instruction is free
// to permute, so every lane loads 8 consecutive k of its row (16 bytes of an
// adapter, 32 of x) straight into registers and feeds them to four
// instructions: no shared memory, no transposes.  Sums of 32 k start from
// zero and are added up in fp32 registers (the tensor core's own running sum
// truncates).
#include "q4k_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace q4k {
namespace {

constexpr int kTile = 16;        // tokens of a tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Parts of the columns that the shrink's CTAs split among them: more for few
// tokens, which have few tiles.
int column_parts(int64_t tokens, int64_t cols) {
  const int64_t want = tokens <= 64 ? 8 : tokens <= 512 ? 4 : 2;
  return (int)std::max<int64_t>(1, std::min(want, cols / 256));
}

struct Tile {
  int adapter;                   // -1: none
  int first, n;                  // places of the order
};

// Tile `t` of the segments' tiles in order; n = 0: there are fewer.  One warp.
__device__ __forceinline__ Tile find_tile(const LoraParams& P, int t) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int64_t s0 = 0; s0 < P.n_seg; s0 += 32) {
    const int64_t s = s0 + lane;
    int a = 0, b = 0, adapter = -1;
    if (s < P.n_seg) {
      a = P.seg_start[s];
      b = P.seg_start[s + 1];
      adapter = P.seg_adapter[s];
      if (a < 0 || b < a || b > P.tokens) {
        atomicOr(P.err, kErrIndex);
        a = b = 0;
      }
    }
    int incl = (b - a + kTile - 1) / kTile;
    const int own = incl;
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned here = __ballot_sync(0xffffffffu, t >= base + incl - own && t < base + incl);
    if (here) {
      const int src = __ffs(here) - 1;
      const int k = t - base - __shfl_sync(0xffffffffu, incl - own, src);
      const int sa = __shfl_sync(0xffffffffu, a, src), sb = __shfl_sync(0xffffffffu, b, src);
      adapter = __shfl_sync(0xffffffffu, adapter, src);
      if (adapter >= P.n_adapters) {
        if (lane == 0) atomicOr(P.err, kErrIndex);
        adapter = -1;
      }
      return {max(adapter, -1), sa + k * kTile, min(kTile, sb - sa - k * kTile)};
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return {-1, 0, 0};
}

// The token at place i of the order; -1 if it is out of range.
__device__ __forceinline__ int token_at(const LoraParams& P, int i) {
  const int t = P.order[i];
  if (t >= 0 && t < P.tokens) return t;
  atomicOr(P.err, kErrIndex);
  return -1;
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// v = hi + lo: hi rounded to tf32's 11 bits, lo exact (read to 11 bits).
__device__ __forceinline__ void split(float v, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(v) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(v - __uint_as_float(hi));
}

template <bool BF16>
__device__ __forceinline__ void widen(uint32_t v, uint32_t& x, uint32_t& y) {
  if constexpr (BF16) {
    x = v << 16;
    y = v & 0xffff0000u;
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
    x = __float_as_uint(f.x);
    y = __float_as_uint(f.y);
  }
}

// c += X W^T over 32 k: X rows g and g + 8 as 8 consecutive k each (xa, xb),
// W row g of each tile as 8 consecutive k (w).
template <bool BF16, int NT>
__device__ __forceinline__ void step32(float (&c)[NT][4], const float4 (&xa)[2], const float4 (&xb)[2],
                                       const uint4 (&w)[NT], int tiles) {
  float t[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q) t[q][0] = t[q][1] = t[q][2] = t[q][3] = 0.f;
  const float* a = reinterpret_cast<const float*>(xa);
  const float* b = reinterpret_cast<const float*>(xb);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h0, h1, h2, h3, l0, l1, l2, l3;
    split(a[2 * i], h0, l0);
    split(b[2 * i], h1, l1);
    split(a[2 * i + 1], h2, l2);
    split(b[2 * i + 1], h3, l3);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      if (q < tiles) {
        uint32_t w0, w1;
        widen<BF16>(i == 0 ? w[q].x : i == 1 ? w[q].y : i == 2 ? w[q].z : w[q].w, w0, w1);
        mma_tf32(t[q], h0, h1, h2, h3, w0, w1);
        mma_tf32(t[q], l0, l1, l2, l3, w0, w1);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[q][e] += t[q][e];
}

// h[part][place][m * rank + j], scaled.  Grid: tiles x column parts x groups
// of NT rank tiles (8 ranks each); a CTA's warps split its columns.
template <bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, 2) lora_shrink_kernel(const LoraParams P) {
  __shared__ float part[kWarps][NT * 8][kTile + 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Tile T = find_tile(P, blockIdx.x);
  if (T.n <= 0 || T.adapter < 0) return;                 // the whole block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int all = P.n * P.rank, q0 = blockIdx.z * NT, tiles = min(NT, all / 8 - q0);
  const int ta = g < T.n ? token_at(P, T.first + g) : -1, tb = g + 8 < T.n ? token_at(P, T.first + g + 8) : -1;
  const float* xa = P.x + (int64_t)max(ta, 0) * P.cols + 8 * c;
  const float* xb = P.x + (int64_t)max(tb, 0) * P.cols + 8 * c;
  const uint16_t* wp[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int col = min(q0 + q, all / 8 - 1) * 8, m = col / P.rank, j = col - m * P.rank;
    wp[q] = static_cast<const uint16_t*>(P.mat[m].a) + ((int64_t)T.adapter * P.rank + j + g) * P.cols + 8 * c;
  }
  float acc[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
  // this warp's steps of 32 columns: every (parts * kWarps)-th
  const int steps = (int)(P.cols / 32), stride = gridDim.y * kWarps;
  constexpr int kAhead = NT <= 2 ? 4 : 2;                // steps in flight
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 a[kAhead][2], b[kAhead][2];
  uint4 w[kAhead][NT];
  auto load = [&](int i, int s) {
    const int64_t k = (int64_t)s * 32;
    const bool in = s < steps;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      a[i][e] = in && ta >= 0 ? reinterpret_cast<const float4*>(xa + k)[e] : zero;
      b[i][e] = in && tb >= 0 ? reinterpret_cast<const float4*>(xb + k)[e] : zero;
    }
#pragma unroll
    for (int q = 0; q < NT; ++q)
      if (q < tiles) w[i][q] = in ? __ldg(reinterpret_cast<const uint4*>(wp[q] + k)) : make_uint4(0, 0, 0, 0);
  };
  int s = blockIdx.y * kWarps + warp;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, s + i * stride);
  for (; s < steps; s += kAhead * stride) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      step32<BF16, NT>(acc, a[i], b[i], w[i], tiles);
      load(i, s + (i + kAhead) * stride);
    }
  }
  // the warps' sums, added up in warp order
#pragma unroll
  for (int q = 0; q < NT; ++q) {
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][8 * q + 2 * c + (e & 1)][g + (e >> 1) * 8] = acc[q][e];
  }
  __syncthreads();
  const float scale = P.scale[T.adapter];
  for (int i = threadIdx.x; i < tiles * 8 * T.n; i += kThreads) {
    const int place = i / (tiles * 8), col = i - place * (tiles * 8);
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += part[k][col][place];
    P.work[((int64_t)blockIdx.y * P.tokens + T.first + place) * all + q0 * 8 + col] = v * scale;
  }
}

// y = base + B h.  Grid: tiles x shares of the chunks of kWarps * 32 outputs
// of all projections; a warp has 32 outputs of one projection for the tile's
// tokens at a time.  Output 8 c + 2 q + e of the 32 is column 2 c + e of
// instruction tile q, so a lane holds 8 consecutive outputs of two tokens.
constexpr int kOuts = 32, kChunk = kWarps * kOuts;
constexpr int kMaxRanks = kLoraMaxMats * 128;

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) lora_expand_kernel(const LoraParams P, int parts, int chunks) {
  __shared__ __align__(16) float h[kTile][kMaxRanks + 4];
  const Tile T = find_tile(P, blockIdx.x);
  if (T.n <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int kblocks = (P.rank + 31) / 32, all = P.n * P.rank;
  const int token[2] = {g < T.n ? token_at(P, T.first + g) : -1, g + 8 < T.n ? token_at(P, T.first + g + 8) : -1};

  // where the warp's outputs of a chunk are (projection m, outputs from o0 on), and what they need: base and B
  int m = 0, first = 0;                                   // first chunk of projection m
  int64_t o0 = 0;
  const uint16_t* bp[4];
  uint4 b[4];
  float y[2][8];
  bool vec = false;
  auto load_b = [&](int kb) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      b[q] = bp[q] && kb * 32 + 8 * c < P.rank ? __ldg(reinterpret_cast<const uint4*>(bp[q] + kb * 32))
                                               : make_uint4(0, 0, 0, 0);
  };
  auto load = [&](int chunk) {
    for (;; ++m) {
      const int n = (int)((P.mat[m].rows + kChunk - 1) / kChunk);
      if (chunk < first + n) break;
      first += n;
    }
    const LoraMat& w = P.mat[m];
    o0 = ((int64_t)(chunk - first) * kWarps + warp) * kOuts;
    vec = (w.rows & 3) == 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t o = o0 + 8 * (g >> 1) + 2 * q + (g & 1);
      bp[q] = T.adapter >= 0 && o < w.rows
                  ? static_cast<const uint16_t*>(w.b) + ((int64_t)T.adapter * w.rows + o) * P.rank + 8 * c
                  : nullptr;
    }
    load_b(0);
    const int64_t o = o0 + 8 * c;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[r][e] = 0.f;
      if (token[r] < 0 || !w.base) continue;
      const float* src = w.base + (int64_t)token[r] * w.rows + o;
      if (vec) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (o + 4 * e < w.rows) *reinterpret_cast<float4*>(&y[r][4 * e]) = reinterpret_cast<const float4*>(src)[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (o + e < w.rows) y[r][e] = src[e];
      }
    }
  };

  load(blockIdx.y);                                       // these do not wait for the first kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (T.adapter >= 0) {
    for (int i = threadIdx.x; i < kTile * all; i += kThreads) {
      const int place = i / all, j = i - place * all;
      float v = 0.f;
      if (place < T.n)
        for (int k = 0; k < parts; ++k) v += __ldcg(P.work + ((int64_t)k * P.tokens + T.first + place) * all + j);
      h[place][j] = v;
    }
    __syncthreads();
  }
  for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
    if (chunk != blockIdx.y) load(chunk);
    const LoraMat& w = P.mat[m];
    if (T.adapter >= 0) {
      float acc[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int kb = 0; kb < kblocks; ++kb) {
        const bool in = kb * 32 + 8 * c < P.rank;
        const float4* ha = reinterpret_cast<const float4*>(&h[g][m * P.rank + kb * 32 + 8 * c]);
        const float4* hb = reinterpret_cast<const float4*>(&h[g + 8][m * P.rank + kb * 32 + 8 * c]);
        const float4 xa[2] = {in ? ha[0] : zero, in ? ha[1] : zero}, xb[2] = {in ? hb[0] : zero, in ? hb[1] : zero};
        const uint4 now[4] = {b[0], b[1], b[2], b[3]};
        if (kb + 1 < kblocks) load_b(kb + 1);
        step32<BF16, 4>(acc, xa, xb, now, 4);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) y[r][2 * q + e] += acc[q][2 * r + e];
    } else if (w.y == w.base) {
      continue;                                           // nothing to add, nothing to copy
    }
    const int64_t o = o0 + 8 * c;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (token[r] < 0) continue;
      float* dst = w.y + (int64_t)token[r] * w.rows + o;
      if (vec) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (o + 4 * e < w.rows) reinterpret_cast<float4*>(dst)[e] = *reinterpret_cast<const float4*>(&y[r][4 * e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (o + e < w.rows) dst[e] = y[r][e];
      }
    }
  }
}

template <bool BF16, int NT>
void shrink(const LoraParams& p, unsigned tiles, int parts, cudaStream_t s) {
  const int groups = (p.n * p.rank / 8 + NT - 1) / NT;
  lora_shrink_kernel<BF16, NT><<<dim3(tiles, parts, groups), kThreads, 0, s>>>(p);
}

template <bool BF16>
cudaError_t launch(const LoraParams& p, cudaStream_t s) {
  const unsigned tiles = (unsigned)std::min<int64_t>(p.tokens, p.n_seg + p.tokens / kTile);
  const int parts = column_parts(p.tokens, p.cols);
  // few tokens: one rank tile per CTA for the sake of latency; many: four of
  // them, so that x is read once for 32 ranks
  if (p.tokens <= 16) shrink<BF16, 1>(p, tiles, parts, s);
  else shrink<BF16, 4>(p, tiles, parts, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  unsigned chunks = 0;
  for (int m = 0; m < p.n; ++m) chunks += (unsigned)((p.mat[m].rows + kChunk - 1) / kChunk);
  int dev = 0;
  cudaGetDevice(&dev);
  const unsigned want = (unsigned)std::max(1, 4 * device_info(dev).sm_count / (int)std::min(tiles, 1u << 20));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles, std::min(chunks, want));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_expand_kernel<BF16>, p, parts, (int)chunks);
}

}  // namespace

size_t lora_workspace(int n, int rank, int64_t tokens) {
  return sizeof(float) * (size_t)n * (size_t)rank * (size_t)tokens * (size_t)column_parts(tokens, int64_t(1) << 24);
}

cudaError_t launch_lora_add(const LoraParams& p, cudaStream_t s) {
  return p.bf16 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace q4k
