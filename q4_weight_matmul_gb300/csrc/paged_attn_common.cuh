// What the two attention kernels share: how the work over the paged cache is
// shared out among the CTAs, and how an item that several of them hold is
// put together.
//
// An item is one tile of up to ROWS query rows (token, head of the group) of
// one request and one key head; its units are the blocks of UNIT keys between
// the first key its first row sees and the last key its last row sees.  The
// units of all items in order (request, key head, row tile) are cut into
// equal contiguous ranges, one per CTA, so that long and short contexts,
// few requests and many, fill the GPU alike.  Lengths are read on the device:
// a captured launch follows them.  An item cut by range ends has a piece per
// CTA: every CTA stores its unnormalised sums with the maximum and sum of its
// softmax, and the last to arrive (a ticket per item) adds the pieces up in
// CTA order, so the result does not depend on who is last.
#pragma once

#include "q4k_internal.h"
#include "tc_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace q4k {
namespace attn {

constexpr int kMaxCtas = 160;           // of a launch
constexpr int kTicketBytes = 1024;      // leading workspace bytes: one counter per CTA

// Keys (or values) in shared memory: groups of 8 cells, per group the first
// 64 values of its cells, then the next 64; a cell's 64 values are 128 bytes,
// 128-byte swizzled.  The cache's tensor map has the same dimensions (values,
// cell of the group, 64s of values, group of the page, page and head), so one
// copy brings up to a whole page of a head.
template <int D>
struct Cells {
  static constexpr int kHalves = D / 64;
  static constexpr int kNext = 1024;                    // bytes to the next 64 values
  static constexpr int kGroup = kNext * kHalves;        // bytes of 8 cells
  static __device__ __forceinline__ uint32_t at(int cell, int half, int chunk) {
    return (uint32_t)((cell >> 3) * kGroup + half * kNext + (cell & 7) * 128 + ((chunk ^ (cell & 7)) << 4));
  }
};

// Copy cells of page `page` (num_pages or more: zeros) and key head `head`,
// from 8-cell group `group` of the page on.
__device__ __forceinline__ void load_cells(uint32_t dst, const void* map, int group, int page, int kv_heads, int head,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %2, %2, %3, %4}], [%5];"
      ::"r"(dst), "l"(map), "r"(0), "r"(group), "r"(page * kv_heads + head), "r"(tc::smem_u32(bar)) : "memory");
}

struct Shape {             // of one request
  int q0, n;               // first token, new tokens
  int64_t kv;              // keys
};

// The request's shape, cut to what the call's arrays hold; what was out of
// range is reported.
__device__ __forceinline__ Shape request(const AttnParams& P, int64_t r) {
  int a = P.cu_q[r], b = P.cu_q[r + 1];
  int64_t kv = P.kv_len[r];
  const int64_t most = P.max_pages * P.page_size;
  if (a < 0 || b < a || b > P.tokens || b - a > P.max_q || kv < 0 || kv > most) {
    atomicOr(P.err, kErrIndex);
    a = max(0, min(a, (int)P.tokens));
    b = max(a, min(b, (int)P.tokens));
    b = min(b, a + (int)P.max_q);
    kv = kv < 0 ? 0 : min(kv, most);
  }
  return {a, b - a, kv};
}

// The keys lo <= j < hi that some row of rows r0 .. r1-1 (of the request's
// n * group rows) sees.
__device__ __forceinline__ void key_range(const Shape& s, int group, int window, int r0, int r1, int64_t& lo,
                                          int64_t& hi) {
  const int64_t first = s.kv - s.n + r0 / group, last = s.kv - s.n + (r1 - 1) / group;
  hi = last + 1 > 0 ? last + 1 : 0;
  lo = window ? first - window + 1 : 0;
  if (lo < 0) lo = 0;
  if (lo > hi) lo = hi;
}

// Units of row tile m (0 .. tiles-1): at least one, so that a tile that sees
// no key is still written.
template <int ROWS, int UNIT>
__device__ __forceinline__ int tile_units(const Shape& s, int group, int window, int m, int64_t& lo, int64_t& hi) {
  const int rows = s.n * group;
  key_range(s, group, window, m * ROWS, min((m + 1) * ROWS, rows), lo, hi);
  const int64_t u = (hi + UNIT - 1) / UNIT - lo / UNIT;
  return u > 0 ? (int)u : 1;
}

template <int ROWS, int UNIT>
__device__ __forceinline__ int64_t request_units(const AttnParams& P, const Shape& s, int group) {
  if (s.n == 0) return 0;
  const int tiles = (s.n * group + ROWS - 1) / ROWS;
  int64_t sum = 0, lo, hi;
  for (int m = 0; m < tiles; ++m) sum += tile_units<ROWS, UNIT>(s, group, P.window, m, lo, hi);
  return sum;
}

// This CTA's share of the work.
struct Range {
  int64_t begin, end, total;
  int64_t req, req_base;      // the request that holds `begin`, the units before it
  int ctas;                   // CTAs that have work (the others have none)
};

// Collective over the block (THREADS threads, a multiple of 32).
template <int ROWS, int UNIT, int THREADS>
__device__ __forceinline__ Range share_out(const AttnParams& P, int group, int min_units, int64_t* scratch) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Range R{0, 0, 0, 0, 0, 0};
  // all units
  int64_t mine = 0;
  for (int64_t r = tid; r < P.n_req; r += THREADS)
    mine += P.kv_heads * request_units<ROWS, UNIT>(P, request(P, r), group);
  int64_t v = mine;
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) scratch[warp] = v;
  __syncthreads();
  for (int w = 0; w < W; ++w) R.total += scratch[w];
  const int64_t n = (R.total + min_units - 1) / min_units;
  R.ctas = (int)(n < gridDim.x ? n : gridDim.x);
  if (R.ctas < 1 || (int)blockIdx.x >= R.ctas) return R;      // the whole block
  R.begin = R.total * blockIdx.x / R.ctas;
  R.end = R.total * (blockIdx.x + 1) / R.ctas;
  // the request that holds the first unit
  int64_t base = 0;
  for (int64_t r0 = 0; r0 < P.n_req; r0 += THREADS) {
    const int64_t r = r0 + tid;
    // with one request per thread the first pass has the units already
    const int64_t own = P.n_req <= THREADS ? mine
                        : r < P.n_req ? P.kv_heads * request_units<ROWS, UNIT>(P, request(P, r), group) : 0;
    int64_t incl = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < W; ++w) {
      if (w < warp) incl += scratch[w];
      all += scratch[w];
    }
    const int64_t at = base + incl - own;
    if (own > 0 && R.begin >= at && R.begin < at + own) {
      scratch[W] = r;
      scratch[W + 1] = at;
    }
    base += all;
    if (R.begin < base) break;                                // the same for every thread
  }
  __syncthreads();
  R.req = scratch[W];
  R.req_base = scratch[W + 1];
  __syncthreads();
  return R;
}

__device__ __forceinline__ int owner(int64_t unit, const Range& R) {
  return (int)(((unit + 1) * R.ctas - 1) / R.total);
}

// The items of a CTA's range, one after another.
template <int ROWS, int UNIT>
struct Walk {
  Shape s;
  int64_t req;
  int head, tile, tiles;
  int64_t at;              // first unit of the item in the order of all
  int units;               // of the item
  int64_t lo, hi;          // its keys
  int u0, u1;              // the item's units that this CTA has

  __device__ __forceinline__ void load(const AttnParams& P, int64_t r, int group) {
    req = r;
    s = request(P, r);
    tiles = (s.n * group + ROWS - 1) / ROWS;
  }
  __device__ __forceinline__ void cut(const Range& R) {
    u0 = (int)(R.begin > at ? R.begin - at : 0);
    u1 = (int)(R.end < at + units ? R.end - at : units);
  }
  __device__ __forceinline__ void first(const AttnParams& P, const Range& R, int group) {
    load(P, R.req, group);
    const int64_t per_head = request_units<ROWS, UNIT>(P, s, group);
    head = (int)((R.begin - R.req_base) / per_head);
    at = R.req_base + head * per_head;
    for (tile = 0;; ++tile) {
      units = tile_units<ROWS, UNIT>(s, group, P.window, tile, lo, hi);
      if (R.begin < at + units) break;
      at += units;
    }
    cut(R);
  }
  // false: the range is done
  __device__ __forceinline__ bool next(const AttnParams& P, const Range& R, int group) {
    at += units;
    if (at >= R.end) return false;
    if (++tile == tiles) {
      tile = 0;
      if (++head == P.kv_heads) {
        head = 0;
        do load(P, req + 1, group);
        while (s.n == 0);                       // units remain, so a request with tokens follows
      }
    }
    units = tile_units<ROWS, UNIT>(s, group, P.window, tile, lo, hi);
    cut(R);
    return true;
  }
};

// Floats of one piece: per row the sums, then all maxima, then all sums of weights.
template <int ROWS, int D>
__host__ __device__ constexpr size_t piece_floats() { return (size_t)ROWS * (D + 2); }

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
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  else return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Store four consecutive outputs of a row.
template <bool BF16>
__device__ __forceinline__ void store4(void* out, bool f32, int64_t at, float4 v) {
  if (f32) *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack2<BF16>(v.x, v.y), pack2<BF16>(v.z, v.w));
}

__device__ __forceinline__ int64_t out_row(const AttnParams& P, const Shape& s, int head, int group, int row) {
  const int i = row / group;
  return (int64_t)(s.q0 + i) * P.heads + head * group + (row - i * group);
}

// Arrive with this CTA's piece of an item held by CTAs c0..c1; true in every
// thread of the last CTA.  `flag` is shared; SYNC is a barrier of the calling
// threads, `leader` one of them.
template <class SYNC>
__device__ __forceinline__ bool arrive(unsigned* ticket, int pieces, int* flag, bool leader, SYNC sync) {
  __threadfence();
  sync();
  if (leader) {
    const bool last = atomicAdd(ticket, 1u) == (unsigned)(pieces - 1);
    if (last) *ticket = 0u;                      // ready for the next call
    __threadfence();
    *flag = last;
  }
  sync();
  return *flag != 0;
}

// Add the pieces of CTAs c0..c1 up and write the item's rows: `n` threads,
// this one is `t`.  weights: kMaxCtas * ROWS shared floats.
template <int ROWS, int D, bool BF16, class SYNC>
__device__ __forceinline__ void combine(const AttnParams& P, const float* pieces, int c0, int c1, const Shape& s,
                                        int head, int group, int row0, int rows, float* weights, int t, int n,
                                        SYNC sync) {
  // piece of CTA c: slot 1 (the item starts in its range) for the first, slot 0 for the others
  auto piece = [&](int c) { return pieces + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * piece_floats<ROWS, D>(); };
  const int np = c1 - c0 + 1;
  for (int r = t; r < rows; r += n) {
    float m = -INFINITY;
    for (int c = c0; c <= c1; ++c) m = fmaxf(m, __ldcg(piece(c) + ROWS * D + r));
    float l = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const float mc = __ldcg(piece(c) + ROWS * D + r);
      const float w = mc == -INFINITY ? 0.f : exp2f(mc - m);
      l += w * __ldcg(piece(c) + ROWS * D + ROWS + r);
      weights[(c - c0) * ROWS + r] = w;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int c = 0; c < np; ++c) weights[c * ROWS + r] *= inv;
  }
  sync();
  for (int e = t; e < rows * (D / 4); e += n) {
    const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < np; ++c) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(piece(c0 + c) + r * D + d));
      const float w = weights[c * ROWS + r];
      a.x = fmaf(w, v.x, a.x), a.y = fmaf(w, v.y, a.y), a.z = fmaf(w, v.z, a.z), a.w = fmaf(w, v.w, a.w);
    }
    store4<BF16>(P.out, P.out_f32, out_row(P, s, head, group, row0 + r) * D + d, a);
  }
  sync();
}

// The same with one thread per row (row r, its output at out_at) and pieces
// laid out [D/4][ROWS][4], so that the threads of a warp read whole lines.
template <int ROWS, int D, bool BF16>
__device__ __forceinline__ void combine_rows(const AttnParams& P, const float* pieces, int c0, int c1, bool mine,
                                             int r, int64_t out_at) {
  if (!mine) return;
  auto piece = [&](int c) { return pieces + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * piece_floats<ROWS, D>(); };
  float m = -INFINITY, l = 0.f;
  for (int c = c0; c <= c1; ++c) m = fmaxf(m, __ldcg(piece(c) + ROWS * D + r));
  for (int c = c0; c <= c1; ++c) {
    const float mc = __ldcg(piece(c) + ROWS * D + r);
    if (mc != -INFINITY) l += exp2f(mc - m) * __ldcg(piece(c) + ROWS * D + ROWS + r);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
  for (int d = 0; d < D; d += 32) {
    float4 a[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) a[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int c = c0; c <= c1; ++c) {
      const float* from = piece(c) + (d / 4 * ROWS + r) * 4;
      float4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = __ldcg(reinterpret_cast<const float4*>(from + q * ROWS * 4));
      const float mc = __ldcg(piece(c) + ROWS * D + r), w = mc == -INFINITY ? 0.f : exp2f(mc - m) * inv;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        a[q].x = fmaf(w, v[q].x, a[q].x), a[q].y = fmaf(w, v[q].y, a[q].y);
        a[q].z = fmaf(w, v[q].z, a[q].z), a[q].w = fmaf(w, v[q].w, a[q].w);
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) store4<BF16>(P.out, P.out_f32, out_at + d + 4 * q, a[q]);
  }
}

}  // namespace attn
}  // namespace q4k
