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
// Products run on mma.sync m16n8k16 with the adapters' 16-bit values as they
// are; a fp32 activation enters as a sum of values of their type: three
// bfloat16 (24 bits), or two binary16 (22 bits) of the activations scaled by
// a power of two, the same for 32 of a row, that puts the largest near 2^14,
// the second part times 2^11.  So binary16 keeps 22 bits down to 2^-29 of the
// largest and 20 down to 2^-31; where a value but zero is smaller, the warp
// makes its sums again with tf32 instructions (22 bits for any value).  That
// and the second scale cost 7 % (2049 tokens, below: 38.6 us without; 45.7 with
// tf32 throughout).  A value that rounding to its type would make infinite is
// cut off instead, and an infinity is its first part alone.  The k index of an
// instruction is free to permute, so every lane loads 8 consecutive k of its
// row (16 bytes of an adapter, 32 of x) and feeds them to two instructions
// without a transpose.  Sums of 32 k start from zero and are added up in fp32
// registers (the tensor core's own running sum truncates).
//
// Measured, binary16 | bfloat16: 2049 tokens of 4 adapters of rank 32 beside
// 2560 x 9728: 41.2 | 40.3 us (3.0 TB/s); 64 tokens of 17 adapters of rank 64
// beside 2 x 9728 x 2560: 25.5 | 26.1 us; one token beside q, k and v: 6.1 | 5.9 us.
#include "mma_sync.cuh"
#include "q4k_internal.h"
#include "tc_ptx.cuh"

#include <algorithm>

namespace q4k {
namespace {

constexpr int kTile = 16;        // tokens of a tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Parts of the columns that the shrink's CTAs split among them: as many as
// give its tiles of 16 tokens a CTA per SM, 2 at least (us with 8, 4, 2 for up
// to 64, 512 and more tokens | this: 80 tokens, rank 48 of 5632 columns 12.9 |
// 11.3; 278, rank 64 of 6912 23.9 | 20.4; 513, 2 x rank 24 of 7424 35.7 | 29.2;
// 1600 the same; twice as many parts: 28.1 for the 513, but 19.4 -> 22.0 for
// 3 x rank 32 of 2560, whose second launch adds them up).
constexpr int kMaxParts = 8;
constexpr int64_t kSplitTokens = 152 * kTile;
int column_parts(int64_t tokens, int64_t cols) {
  const int64_t want = std::max<int64_t>(2, std::min<int64_t>(kMaxParts, kSplitTokens / tokens));
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

constexpr float kLow = 2048.f;   // the second part of a binary16 operand is held times 2^11

// The parts of a s[0] and b s[1] (s = 1: bfloat16).  CUT: the first part of a
// value is cut off, not rounded, so that it is finite where the value is; of an
// infinity it is all, and the others are zero (not its difference from itself).
template <bool BF16, bool CUT>
__device__ __forceinline__ void split_rows(const float (&a)[8], const float (&b)[8], const float (&s)[2],
                                           uint32_t (&p)[BF16 ? 3 : 2][2][4]) {
  auto pack = [](float v, float w, bool cut) {
    return cut ? __float_as_uint(v) >> 16 | (__float_as_uint(w) & 0xffff0000u) : pack2<BF16>(v, w);
  };
  auto rest = [](float v, float part) { return CUT && fabsf(v) == INFINITY ? 0.f : v - part; };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0 = a[2 * i] * s[0], x1 = a[2 * i + 1] * s[0], y0 = b[2 * i] * s[1], y1 = b[2 * i + 1] * s[1];
#pragma unroll
    for (int k = 0; k < (BF16 ? 3 : 2); ++k) {
      if (!BF16 && k == 1) x0 *= kLow, x1 *= kLow, y0 *= kLow, y1 *= kLow;
      const uint32_t x = pack(x0, x1, CUT && k == 0), y = pack(y0, y1, CUT && k == 0);
      const float2 fx = unpack2<BF16>(x), fy = unpack2<BF16>(y);
      x0 = rest(x0, fx.x), x1 = rest(x1, fx.y), y0 = rest(y0, fy.x), y1 = rest(y1, fy.y);
      p[k][i >> 1][2 * (i & 1)] = x;
      p[k][i >> 1][2 * (i & 1) + 1] = y;
    }
  }
}

// The 16-bit parts of the two rows' 8 values each: p[part][i] is the A operand
// of instruction i; `back`: what the products are to be multiplied by.  Bit r
// of the result: a value of this lane in row r is so far below the row's
// largest that the parts do not hold it, and the products are to be made apart
// (below).
template <bool BF16>
__device__ __forceinline__ uint32_t split(const float (&a)[8], const float (&b)[8], uint32_t (&p)[BF16 ? 3 : 2][2][4],
                                      float (&back)[2]) {
  float s[2] = {1.f, 1.f};
  back[0] = back[1] = 1.f;
  uint32_t apart = 0;
  float top = 0.f;
  if constexpr (BF16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(a[e]), fabsf(b[e])));
  } else {
    float top[2] = {0.f, 0.f};
    uint32_t low[2] = {0xffffffffu, 0xffffffffu};                           // twice the least magnitude but zero, less one
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      top[0] = fmaxf(top[0], fabsf(a[e])), top[1] = fmaxf(top[1], fabsf(b[e]));
      low[0] = min(low[0], 2u * __float_as_uint(a[e]) - 1u), low[1] = min(low[1], 2u * __float_as_uint(b[e]) - 1u);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));      // the row's other 24 values
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const uint32_t e = max(__float_as_uint(top[r]) >> 23, 15u);           // biased exponent
      s[r] = __uint_as_float((268u - e) << 23);                             // 2^(14 - exponent)
      back[r] = __uint_as_float((e - 14u) << 23);
      if (e > 30u && (low[r] < (e - 30u) << 24 || e == 255u)) apart |= 1u << r;      // below 2^-16 when scaled; infinite
    }
  }
  if constexpr (BF16) {
    if (top > 0x1.fep127f) split_rows<true, true>(a, b, s, p);       // bfloat16's largest value
    else split_rows<true, false>(a, b, s, p);
    __syncwarp();                                                    // the products are the whole warp's
  } else {
    split_rows<false, false>(a, b, s, p);
  }
  return apart;
}

// c += X W^T over 32 k: X as split() made it, W row g of each tile as 8
// consecutive k (w).
template <bool BF16, int NT>
__device__ __forceinline__ void products(float (&c)[NT][4], const uint32_t (&p)[BF16 ? 3 : 2][2][4],
                                         const float (&back)[2], const uint4 (&w)[NT], int tiles) {
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    if (q < tiles) {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (BF16) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          mma16816<BF16>(t, p[k][0], w[q].x, w[q].y);
          mma16816<BF16>(t, p[k][1], w[q].z, w[q].w);
        }
      } else {
        float u[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816<BF16>(t, p[0][0], w[q].x, w[q].y);
        mma16816<BF16>(u, p[1][0], w[q].x, w[q].y);
        mma16816<BF16>(t, p[0][1], w[q].z, w[q].w);
        mma16816<BF16>(u, p[1][1], w[q].z, w[q].w);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = fmaf(u[e], 1.f / kLow, t[e]);
      }
      c[q][0] = fmaf(t[0], back[0], c[q][0]), c[q][1] = fmaf(t[1], back[0], c[q][1]);
      c[q][2] = fmaf(t[2], back[1], c[q][2]), c[q][3] = fmaf(t[3], back[1], c[q][3]);
    }
  }
}

// The same with X rows g and g + 8 as 8 consecutive k each (xa, xb); result as split()'s.
template <bool BF16, int NT>
__device__ __forceinline__ uint32_t step32(float (&c)[NT][4], const float4 (&xa)[2], const float4 (&xb)[2],
                                       const uint4 (&w)[NT], int tiles) {
  const float a[8] = {xa[0].x, xa[0].y, xa[0].z, xa[0].w, xa[1].x, xa[1].y, xa[1].z, xa[1].w};
  const float b[8] = {xb[0].x, xb[0].y, xb[0].z, xb[0].w, xb[1].x, xb[1].y, xb[1].z, xb[1].w};
  uint32_t p[BF16 ? 3 : 2][2][4];
  float back[2];
  const uint32_t apart = split<BF16>(a, b, p, back);
  products<BF16, NT>(c, p, back, w, tiles);
  return apart;
}

// Products of binary16 adapters with activations that are too far apart for
// one scale: tf32 instructions, twice as many, whose operands have fp32's
// exponents and hold binary16 exactly.
__device__ __forceinline__ uint32_t to_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
// C += A B, 16 x 8 x 8: A holds rows g (a[0], a[2]) and g + 8 (a[1], a[3]) at
// k = c and c + 4, B column g at the same k, C as mma16816's.
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
// c += X W^T over 32 k for one tile of W's rows, a and b rows g and g + 8 of X.
__device__ __forceinline__ void step32_apart(float (&c)[4], const float (&a)[8], const float (&b)[8], const uint4& w) {
  const float2 f[4] = {unpack2<false>(w.x), unpack2<false>(w.y), unpack2<false>(w.z), unpack2<false>(w.w)};
  float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4] = {a[2 * i], b[2 * i], a[2 * i + 1], b[2 * i + 1]};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float size = fabsf(x[e]);                  // past tf32's largest value: cut off; infinite: this part is all
        p[e] = size > 0x1.ffcp127f ? __float_as_uint(x[e]) & 0xffffe000u : to_tf32(x[e]);
        x[e] = size == INFINITY ? 0.f : x[e] - __uint_as_float(p[e]);
      }
      mma1688(t, p, f[i].x, f[i].y);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += t[e];
}
__device__ __forceinline__ void load8(float (&x)[8], const float* from) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 v = from ? reinterpret_cast<const float4*>(from)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
    x[4 * e] = v.x, x[4 * e + 1] = v.y, x[4 * e + 2] = v.z, x[4 * e + 3] = v.w;
  }
}

// h[part][place][m * rank + j], scaled.  Grid: tiles x column parts x groups
// of NT rank tiles (8 ranks each); a CTA's warps split its columns.

// The warps' sums, added up in warp order; part: [warp][NT * 8][kTile + 1].
template <int NT>
__device__ __forceinline__ void store_h(const LoraParams& P, const Tile& T, float (*part)[NT * 8][kTile + 1],
                                        const float (&acc)[NT][4], int q0, int tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, all = P.n * P.rank;
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

// Row `col` of the adapter's A, all projections after one another.
__device__ __forceinline__ const uint16_t* a_row(const LoraParams& P, int adapter, int col) {
  const int m = col / P.rank, j = col - m * P.rank;
  return static_cast<const uint16_t*>(P.mat[m].a) + ((int64_t)adapter * P.rank + j) * P.cols;
}

// A warp's sums again, all products made apart; its steps of 32 columns are
// every (parts * kWarps)-th in both kernels.
template <int NT>
struct Sums {
  float v[NT][4];
};
template <int NT>
__device__ __noinline__ Sums<NT> sums_apart(const LoraParams& P, int adapter, int ta, int tb, int q0, int tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const float* xa = ta >= 0 ? P.x + (int64_t)ta * P.cols + 8 * c : nullptr;
  const float* xb = tb >= 0 ? P.x + (int64_t)tb * P.cols + 8 * c : nullptr;
  const int64_t stride = (int64_t)gridDim.y * kWarps;
  Sums<NT> sum{};
  for (int64_t s = blockIdx.y * kWarps + warp; s < P.cols / 32; s += stride) {
    float a[8], b[8];
    load8(a, xa ? xa + s * 32 : nullptr);
    load8(b, xb ? xb + s * 32 : nullptr);
#pragma unroll
    for (int q = 0; q < NT; ++q)
      if (q < tiles)
        step32_apart(sum.v[q], a, b,
                     __ldg(reinterpret_cast<const uint4*>(a_row(P, adapter, (q0 + q) * 8 + g) + 8 * c + s * 32)));
  }
  return sum;
}
template <bool BF16, int NT>
__device__ __forceinline__ void replace_apart(const LoraParams& P, const Tile& T, float (&acc)[NT][4], int q0, int tiles,
                                              uint32_t apart) {
  const int g = (threadIdx.x & 31) >> 2;
  const uint32_t there = (g < T.n ? 1u : 0u) | (g + 8 < T.n ? 2u : 0u);      // other rows hold anything
  if (BF16 || !__any_sync(0xffffffffu, apart & there)) return;
  const int ta = g < T.n ? token_at(P, T.first + g) : -1, tb = g + 8 < T.n ? token_at(P, T.first + g + 8) : -1;
  const Sums<NT> sum = sums_apart<NT>(P, T.adapter, ta, tb, q0, tiles);
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[q][e] = sum.v[q][e];
}

// Few tokens: latency counts.  Operands straight into registers, one rank
// tile per CTA.  Up to 16 tokens; both sides, us for the whole call, this |
// the kernel below:
//   tokens                                 1          4          8           16          32          64
//   rank 16, (4096 + 2 x 1024) x 2560   6.1 | 7.9  7.7 | 7.9  7.7 | 8.1   7.7 | 8.6   8.8 | 9.6   11.0 | 11.2
//   rank 64, 2 x 9728 x 2560            8.6 | 9.0             13.2 | 10.8 14.4 | 11.8 15.5 | 13.4 19.9 | 16.8
template <bool BF16>
__global__ void __launch_bounds__(kThreads) lora_shrink_few_kernel(const __grid_constant__ LoraParams P) {
  __shared__ float part[kWarps][8][kTile + 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Tile T = find_tile(P, blockIdx.x);
  if (T.n <= 0 || T.adapter < 0) return;                 // the whole block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int ta = g < T.n ? token_at(P, T.first + g) : -1, tb = g + 8 < T.n ? token_at(P, T.first + g + 8) : -1;
  const float* xa = P.x + (int64_t)max(ta, 0) * P.cols + 8 * c;
  const float* xb = P.x + (int64_t)max(tb, 0) * P.cols + 8 * c;
  const uint16_t* wp = a_row(P, T.adapter, blockIdx.z * 8 + g) + 8 * c;
  float acc[1][4] = {{0.f, 0.f, 0.f, 0.f}};
  // this warp's steps of 32 columns: every (parts * kWarps)-th
  const int steps = (int)(P.cols / 32), stride = gridDim.y * kWarps;
  constexpr int kAhead = 4;                              // steps in flight
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 a[kAhead][2], b[kAhead][2];
  uint4 w[kAhead][1];
  auto load = [&](int i, int s) {
    const int64_t k = (int64_t)s * 32;
    const bool in = s < steps;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      a[i][e] = in && ta >= 0 ? reinterpret_cast<const float4*>(xa + k)[e] : zero;
      b[i][e] = in && tb >= 0 ? reinterpret_cast<const float4*>(xb + k)[e] : zero;
    }
    w[i][0] = in ? __ldg(reinterpret_cast<const uint4*>(wp + k)) : make_uint4(0, 0, 0, 0);
  };
  int s = blockIdx.y * kWarps + warp;
  uint32_t apart = 0;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, s + i * stride);
  for (; s < steps; s += kAhead * stride) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      apart |= step32<BF16, 1>(acc, a[i], b[i], w[i], 1);
      load(i, s + (i + kAhead) * stride);
    }
  }
  replace_apart<BF16, 1>(P, T, acc, blockIdx.z, 1, apart);
  store_h<1>(P, T, part, acc, blockIdx.z, 1);
}

// Many tokens: bandwidth counts.  Stages of 256 columns (the tile's rows of x
// and the rank rows of A, from wherever a row lies) go through a ring in
// shared memory by 16-byte asynchronous copies, all threads sharing them
// (bulk copies of single rows, 48 to a stage, took longer to issue than to
// arrive); warp w has columns 32 w .. of every stage.  Rows are padded so
// that the lanes of a load meet different banks.
constexpr int kCols = 256;
constexpr int kXRow = kCols * 4 + 16, kARow = kCols * 2 + 64;      // bytes of a row in shared memory

template <int NT>
struct Shrink {
  static constexpr int kStage = kTile * kXRow + NT * 8 * kARow;
  static constexpr int kPart = kWarps * NT * 8 * (kTile + 1) * 4;
  static constexpr int kStages = 112 * 1024 / kStage > 4 ? 4 : 112 * 1024 / kStage;      // two CTAs per SM
  static constexpr int kSmem = kStages * kStage > kPart ? kStages * kStage : kPart;
};

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
// The first `bytes` of 16, then zeros.
__device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

template <bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, 2) lora_shrink_kernel(const __grid_constant__ LoraParams P) {
  using S = Shrink<NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Tile T = find_tile(P, blockIdx.x);
  if (T.n <= 0 || T.adapter < 0) return;                 // the whole block
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int q0 = blockIdx.z * NT, tiles = min(NT, P.n * P.rank / 8 - q0);
  // this CTA's stages: blockIdx.y, + parts, ...
  const int parts = gridDim.y, stages = (int)(P.cols / kCols), mine = (stages - (int)blockIdx.y + parts - 1) / parts;

  // what a thread copies of a stage: 16 bytes of x rows tid / 64 + 4 i, and of A rows tid / 32 + 8 i
  constexpr int XN = kTile / 4;
  const float* xs[XN];
  const uint16_t* as[NT];
#pragma unroll
  for (int i = 0; i < XN; ++i) {
    const int r = tid / 64 + 4 * i, t = r < T.n ? token_at(P, T.first + r) : -1;
    xs[i] = t >= 0 ? P.x + (int64_t)t * P.cols + 4 * (tid % 64) : nullptr;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
    as[i] = i < tiles ? a_row(P, T.adapter, (q0 + i) * 8 + tid / 32) + 8 * (tid % 32) : nullptr;
  // rows that are not there keep what shared memory held: an output row takes nothing from another's input row
  auto copy = [&](int i) {
    if (i < mine) {
      uint8_t* at = smem + (i % S::kStages) * S::kStage;
      const int64_t k = ((int64_t)blockIdx.y + (int64_t)i * parts) * kCols;
#pragma unroll
      for (int j = 0; j < XN; ++j)
        if (xs[j]) copy16(at + (tid / 64 + 4 * j) * kXRow + 16 * (tid % 64), xs[j] + k);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (as[j]) copy16(at + kTile * kXRow + (8 * j + tid / 32) * kARow + 16 * (tid % 32), as[j] + k);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");       // an empty one past the last stage
  };
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) copy(i);

  uint32_t apart = 0;
  float acc[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
  for (int i = 0; i < mine; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
    __syncthreads();                                     // stage i is there, and stage i - 1 has been used
    copy(i + S::kStages - 1);
    const uint8_t* at = smem + (i % S::kStages) * S::kStage;
    const uint8_t* x = at + g * kXRow + warp * 128 + c * 32;
    const uint8_t* a = at + kTile * kXRow + g * kARow + warp * 64 + c * 16;
    float4 xa[2], xb[2];
    uint4 w[NT];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      xa[e] = reinterpret_cast<const float4*>(x)[e];
      xb[e] = reinterpret_cast<const float4*>(x + 8 * kXRow)[e];
    }
#pragma unroll
    for (int q = 0; q < NT; ++q) w[q] = *reinterpret_cast<const uint4*>(a + q * 8 * kARow);
    apart |= step32<BF16, NT>(acc, xa, xb, w, tiles);
  }
  replace_apart<BF16, NT>(P, T, acc, q0, tiles, apart);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  store_h<NT>(P, T, reinterpret_cast<float(*)[NT * 8][kTile + 1]>(smem), acc, q0, tiles);
}

// y = base + B h.  Grid: tiles x shares of the chunks of kWarps * 32 outputs
// of all projections; a warp has 32 outputs of one projection for the tile's
// tokens at a time.  Output 8 c + 2 q + e of the 32 is column 2 c + e of
// instruction tile q, so a lane holds 8 consecutive outputs of two tokens.
// The parts of h are made once per CTA and lie in shared memory as the lanes
// take them (making them again for every 32 outputs cost as many
// instructions as all the rest).
constexpr int kOuts = 32, kChunk = kWarps * kOuts;

// Blocks of 32 ranks of all projections, and the bytes of one's parts.
__host__ __device__ constexpr int rank_blocks(int n, int rank) { return n * ((rank + 31) / 32); }
template <bool BF16>
__host__ __device__ constexpr int block_bytes() { return (BF16 ? 3 : 2) * 2 * 32 * 16 + 2 * 32 * 4; }

// A ring slot: base of the tile's tokens for a chunk (rows as in the shrink),
// and 32 ranks of the chunk's rows of B.  The copies of two CTAs keep some
// 130 KB in flight on an SM; with base and B loaded into registers one chunk
// ahead (32 KB in flight) plain copying of base to y took 2.4 TB/s.
constexpr int kBRow = 64;
constexpr int kSlot = kTile * kXRow + kChunk * kBRow;

// A CTA's outputs with all products made apart, operands straight from global
// memory; output 8 q + 2 c + e of a warp's 32 is column 2 c + e of tile q.
__device__ __noinline__ void expand_apart(const LoraParams& P, const Tile& T, int ta, int tb, int parts, int chunks) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, all = P.n * P.rank;
  const int token[2] = {ta, tb};
  int m = 0, first = 0;
  for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
    for (;; ++m) {
      const int n = (int)((P.mat[m].rows + kChunk - 1) / kChunk);
      if (chunk < first + n) break;
      first += n;
    }
    const LoraMat& w = P.mat[m];
    const int64_t o0 = (int64_t)(chunk - first) * kChunk + warp * kOuts;
    float y[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t o = o0 + 8 * q + 2 * c + (e & 1), t = token[e >> 1];
        y[q][e] = w.base && t >= 0 && o < w.rows ? w.base[t * w.rows + o] : 0.f;
      }
    for (int j0 = 0; j0 < P.rank; j0 += 32) {
      const int j = j0 + 8 * c;
      float x[2][8] = {};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (g + 8 * r >= T.n || j >= P.rank) continue;
        const float* from = P.work + ((int64_t)T.first + g + 8 * r) * all + m * P.rank + j;
        for (int k = 0; k < parts; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[r][e] += __ldcg(from + (int64_t)k * P.tokens * all + e);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t o = o0 + 8 * q + g;
        const uint16_t* from = static_cast<const uint16_t*>(w.b) + ((int64_t)T.adapter * w.rows + o) * P.rank + j;
        const uint4 b = o < w.rows && j < P.rank ? __ldg(reinterpret_cast<const uint4*>(from)) : make_uint4(0, 0, 0, 0);
        step32_apart(y[q], x[0], x[1], b);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t o = o0 + 8 * q + 2 * c + (e & 1), t = token[e >> 1];
        if (t >= 0 && o < w.rows) w.y[t * w.rows + o] = y[q][e];
      }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) lora_expand_kernel(const __grid_constant__ LoraParams P, int parts, int chunks, int slots) {
  // [block]: parts [part][instruction][lane], back [row][lane]; then the ring
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int PARTS = BF16 ? 3 : 2;
  const Tile T = find_tile(P, blockIdx.x);
  if (T.n <= 0) {                                        // as the others, not before the first kernel has ended
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int all = P.n * P.rank, rank_blocks_m = (P.rank + 31) / 32, kblocks = T.adapter >= 0 ? rank_blocks_m : 1;
  uint8_t* ring = smem + P.n * rank_blocks_m * block_bytes<BF16>();
  const int token[2] = {g < T.n ? token_at(P, T.first + g) : -1, g + 8 < T.n ? token_at(P, T.first + g + 8) : -1};
  int copy_token[kTile / 4];                             // of the base rows that this thread copies 16 bytes of
#pragma unroll
  for (int i = 0; i < kTile / 4; ++i)
    copy_token[i] = tid / 64 + 4 * i < T.n ? token_at(P, T.first + tid / 64 + 4 * i) : -1;

  // where a chunk is: projection m, whose first chunk is `first`
  struct Place {
    int chunk, m, first, kb;
  };
  auto find = [&](Place& at) {
    for (;; ++at.m) {
      const int n = (int)((P.mat[at.m].rows + kChunk - 1) / kChunk);
      if (at.chunk < at.first + n) break;
      at.first += n;
    }
  };
  auto advance = [&](Place& at) {
    if (++at.kb < kblocks) return;
    at.kb = 0;
    at.chunk += gridDim.y;
    if (at.chunk < chunks) find(at);
  };
  Place ahead{(int)blockIdx.y, 0, 0, 0};
  find(ahead);
  auto copy = [&](int slot) {
    if (ahead.chunk < chunks) {
      const LoraMat& w = P.mat[ahead.m];
      const int64_t o0 = (int64_t)(ahead.chunk - ahead.first) * kChunk;
      uint8_t* at = ring + slot * kSlot;
      if (ahead.kb == 0 && w.base && (w.rows & 3) == 0) {
        if (o0 + 4 * (tid % 64) < w.rows)
#pragma unroll
          for (int i = 0; i < kTile / 4; ++i)
            if (copy_token[i] >= 0)
              copy16(at + (tid / 64 + 4 * i) * kXRow + 16 * (tid % 64),
                     w.base + (int64_t)copy_token[i] * w.rows + o0 + 4 * (tid % 64));
      } else if (ahead.kb == 0 && w.base) {               // rows of base start anywhere
        const int rows = (int)w.rows, n = rows - (int)o0 - tid % 64;
#pragma unroll
        for (int i = 0; i < kTile / 4; ++i) {
          if (copy_token[i] < 0) continue;
          const float* from = w.base + (int64_t)copy_token[i] * rows + o0 + tid % 64;
          const uint32_t to = tc::smem_u32(at + (tid / 64 + 4 * i) * kXRow + 4 * (tid % 64));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (64 * e < n)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 256 * e), "l"(from + 64 * e) : "memory");
        }
      }
      if (T.adapter >= 0) {
        const int j = ahead.kb * 32 + 8 * (tid % 4);
#pragma unroll
        for (int i = 0; i < kChunk / 64; ++i) {
          const int r = tid / 4 + 64 * i;
          const bool in = o0 + r < w.rows && j < P.rank;       // zeros elsewhere
          const uint16_t* from = static_cast<const uint16_t*>(w.b) +
                                 (in ? ((int64_t)T.adapter * w.rows + o0 + r) * P.rank + j : 0);
          copy16(at + kTile * kXRow + r * kBRow + 16 * (tid % 4), from, in ? 16 : 0);
        }
      }
      advance(ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");       // an empty one past the last step
  };
  // the first copies do not wait for the first kernel
  int put = 0;
  for (int i = 0; i < slots - 1; ++i) copy(put++);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (T.adapter >= 0) {
    uint32_t apart = 0;
    // a warp per block: lane (g, c) has 8 ranks of places g and g + 8
    for (int i = warp; i < P.n * kblocks; i += kWarps) {
      const int j = 32 * (i % kblocks) + 8 * c;
      float x[2][8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool in = g + 8 * r < T.n && j < P.rank;
        const float* from = P.work + ((int64_t)T.first + g + 8 * r) * all + i / kblocks * P.rank + j;
        float4 v[kMaxParts][2];
#pragma unroll
        for (int k = 0; k < kMaxParts; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            v[k][e] = in && k < parts ? __ldcg(reinterpret_cast<const float4*>(from + (int64_t)k * P.tokens * all) + e)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int k = 1; k < kMaxParts; ++k)
            v[0][e].x += v[k][e].x, v[0][e].y += v[k][e].y, v[0][e].z += v[k][e].z, v[0][e].w += v[k][e].w;
          x[r][4 * e] = v[0][e].x, x[r][4 * e + 1] = v[0][e].y, x[r][4 * e + 2] = v[0][e].z, x[r][4 * e + 3] = v[0][e].w;
        }
      }
      uint32_t p[PARTS][2][4];
      float back[2];
      apart |= split<BF16>(x[0], x[1], p, back);
      uint8_t* at = smem + i * block_bytes<BF16>();
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          reinterpret_cast<uint4*>(at)[(k * 2 + e) * 32 + lane] = make_uint4(p[k][e][0], p[k][e][1], p[k][e][2], p[k][e][3]);
      float* scale = reinterpret_cast<float*>(at + PARTS * 2 * 32 * 16);
      scale[lane] = back[0];
      scale[32 + lane] = back[1];
    }
    if (!BF16 && __syncthreads_or(apart)) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      expand_apart(P, T, token[0], token[1], parts, chunks);
      return;
    }
  }

  Place now{(int)blockIdx.y, 0, 0, 0};
  find(now);
  float y[4][4];                                          // [instruction tile][token g: two outputs, token g + 8: two]
  int get = 0;
  while (now.chunk < chunks) {
    if (slots == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                                      // this step's copies are there, the last step's slot is free
    copy(put);
    put = put + 1 == slots ? 0 : put + 1;
    const LoraMat& w = P.mat[now.m];
    const int64_t o = (int64_t)(now.chunk - now.first) * kChunk + warp * kOuts + 8 * c;
    const uint8_t* at = ring + get * kSlot;
    if (now.kb == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float4 v[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        if (token[r] >= 0 && w.base) {
          const float4* from = reinterpret_cast<const float4*>(at + (g + 8 * r) * kXRow + warp * 128 + c * 32);
          v[0] = from[0], v[1] = from[1];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          y[2 * e][2 * r] = v[e].x, y[2 * e][2 * r + 1] = v[e].y;
          y[2 * e + 1][2 * r] = v[e].z, y[2 * e + 1][2 * r + 1] = v[e].w;
        }
      }
    }
    if (T.adapter >= 0) {
      const uint8_t* parts_at = smem + (now.m * kblocks + now.kb) * block_bytes<BF16>();
      uint32_t p[PARTS][2][4];
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 v = reinterpret_cast<const uint4*>(parts_at)[(k * 2 + e) * 32 + lane];
          p[k][e][0] = v.x, p[k][e][1] = v.y, p[k][e][2] = v.z, p[k][e][3] = v.w;
        }
      const float* scale = reinterpret_cast<const float*>(parts_at + PARTS * 2 * 32 * 16);
      const float back[2] = {scale[lane], scale[32 + lane]};
      uint4 b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        b[q] = *reinterpret_cast<const uint4*>(at + kTile * kXRow + (warp * kOuts + 8 * (g >> 1) + 2 * q + (g & 1)) * kBRow +
                                               16 * c);
      products<BF16, 4>(y, p, back, b, 4);
    }
    if (now.kb + 1 == kblocks && (T.adapter >= 0 || w.y != w.base)) {
      if ((w.rows & 3) == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (token[r] < 0) continue;
          float* dst = w.y + (int64_t)token[r] * w.rows + o;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (o + 4 * e < w.rows)
              reinterpret_cast<float4*>(dst)[e] =
                  make_float4(y[2 * e][2 * r], y[2 * e][2 * r + 1], y[2 * e + 1][2 * r], y[2 * e + 1][2 * r + 1]);
        }
      } else {
        // rows start anywhere: put together in this warp's part of the slot,
        // whose base it has used, and written 32 values of a token at a time
        // (a lane's eight values one by one are 4 bytes of every 32 to a
        // store: 112 us against 57 for 1266 tokens beside 1536 x (3910 + 7979))
        uint8_t* mine = ring + get * kSlot + warp * 128;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            reinterpret_cast<float4*>(mine + (g + 8 * r) * kXRow + c * 32)[e] =
                make_float4(y[2 * e][2 * r], y[2 * e][2 * r + 1], y[2 * e + 1][2 * r], y[2 * e + 1][2 * r + 1]);
        __syncwarp();
        const int rows = (int)w.rows, col = (int)o - 8 * c + lane;
        float* dst = w.y + col;
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
          const int to = __shfl_sync(~0u, token[t / 8], 4 * (t % 8));
          if (to >= 0 && col < rows)
            dst[(int64_t)to * rows] = *reinterpret_cast<const float*>(mine + t * kXRow + 4 * lane);
        }
      }
    }
    advance(now);
    get = get + 1 == slots ? 0 : get + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <bool BF16, int NT>
cudaError_t shrink(const LoraParams& p, unsigned tiles, int parts, cudaStream_t s) {
  auto kernel = lora_shrink_kernel<BF16, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, Shrink<NT>::kSmem, done);
  if (e != cudaSuccess) return e;
  const int groups = (p.n * p.rank / 8 + NT - 1) / NT;
  kernel<<<dim3(tiles, parts, groups), kThreads, Shrink<NT>::kSmem, s>>>(p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch(const LoraParams& p, cudaStream_t s) {
  const unsigned tiles = (unsigned)std::min<int64_t>(p.tokens, p.n_seg + p.tokens / kTile);
  const int parts = column_parts(p.tokens, p.cols);
  cudaError_t e;
  if (p.tokens <= 16) {
    lora_shrink_few_kernel<BF16><<<dim3(tiles, parts, p.n * p.rank / 8), kThreads, 0, s>>>(p);
    e = cudaGetLastError();
  } else if (p.n * p.rank <= 32) {
    // groups of 32 ranks | of 64, us, beside 2560 x 2560: 64 tokens, 8 to 32 ranks 7.5-8.6 | 8.3-9.4; 2048 tokens
    // 24.0-25.6 | 26.1-27.3; 40, 64, 3 x 16 ranks: 64 tokens 9.2-10.0 | 10.1-11.4, 512 15.0-19.5 | 15.3-19.8, 2048
    // 36.4-53.1 | 33.1-49.6
    e = shrink<BF16, 4>(p, tiles, parts, s);
  } else {
    e = shrink<BF16, 8>(p, tiles, parts, s);             // x is read once for 64 ranks
  }
  if (e != cudaSuccess) return e;
  unsigned chunks = 0;
  for (int m = 0; m < p.n; ++m) chunks += (unsigned)((p.mat[m].rows + kChunk - 1) / kChunk);
  int dev = 0;
  cudaGetDevice(&dev);
  // one wave of two CTAs per SM where the tiles allow
  const unsigned want = (unsigned)std::max(1, 2 * device_info(dev).sm_count / (int)std::min(tiles, 1u << 20));
  // three slots if two CTAs fit an SM with them, else two
  const int parts_bytes = rank_blocks(p.n, p.rank) * block_bytes<BF16>();
  const int slots = parts_bytes + 3 * kSlot <= 112 * 1024 ? 3 : 2, smem = parts_bytes + slots * kSlot;
  static std::atomic<uint64_t> done{0};
  e = allow_smem(lora_expand_kernel<BF16>, rank_blocks(kLoraMaxMats, 128) * block_bytes<BF16>() + 3 * kSlot, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles, std::min(chunks, want));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_expand_kernel<BF16>, p, parts, (int)chunks, slots);
}

}  // namespace

// Rows of h for any number of tokens up to this one.
size_t lora_workspace(int n, int rank, int64_t tokens) {
  const int64_t rows = std::min(kMaxParts * tokens, std::max(kSplitTokens, 2 * tokens));
  return sizeof(float) * (size_t)n * (size_t)rank * (size_t)rows;
}

cudaError_t launch_lora_add(const LoraParams& p, cudaStream_t s) {
  return p.bf16 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace q4k
