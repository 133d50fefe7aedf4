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

#include "mma_sync.cuh"
#include "q4k_internal.h"
#include "tc_ptx.cuh"

namespace q4k {
namespace attn {

constexpr int kMaxCtas = 160;           // of a launch
// The workspace: a counter per CTA (few rows), a Split per CTA (many rows), the pieces.
constexpr int kTicketBytes = 1024, kSplitBytes = kMaxCtas * 32, kPieceBytes = kTicketBytes + kSplitBytes;

// The item that begins in a CTA's range and goes on past it.
struct Split {
  int last_cta;            // -1: there is none
  int q0, head, row0, rows;
  int unused[3];
};

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

// Whether some wait of the block has given up: one answer for the (converged)
// warp.  Lanes that read the flag at different times would part ways around
// the votes, elections and copies that the whole warp takes part in.
__device__ __forceinline__ bool given_up(volatile int* gave_up) { return __any_sync(0xffffffffu, *gave_up != 0); }

struct Shape {             // of one request
  int q0, n;               // first token, new tokens
  int kv;                  // keys
};

// The request's shape, cut to what the call's arrays hold; what was out of
// range is reported.
__device__ __forceinline__ Shape request(const AttnParams& P, int r) {
  int a = P.cu_q[r], b = P.cu_q[r + 1], kv = P.kv_len[r];
  const int most = (int)(P.max_pages * P.page_size);                  // below 2^31
  if (a < 0 || b < a || b > P.tokens || b - a > P.max_q || kv < 0 || kv > most) {
    atomicOr(P.err, kErrIndex);
    a = max(0, min(a, (int)P.tokens));
    b = max(a, min(b, (int)P.tokens));
    b = min(b, a + (int)P.max_q);
    kv = max(0, min(kv, most));
  }
  return {a, b - a, kv};
}

// The keys lo <= j < hi that some row of rows r0 .. r1-1 (of the request's
// n * group rows) sees.
__device__ __forceinline__ void key_range(const Shape& s, int group, int window, int r0, int r1, int& lo, int& hi) {
  const int first = s.kv - s.n + r0 / group, last = s.kv - s.n + (r1 - 1) / group;
  hi = max(last + 1, 0);
  lo = window && first >= window ? first - window + 1 : 0;
  lo = min(lo, hi);
}

// Units of row tile m (0 .. tiles-1): at least one, so that a tile that sees
// no key is still written.
template <int ROWS, int UNIT>
__device__ __forceinline__ int tile_units(const Shape& s, int group, int window, int m, int& lo, int& hi) {
  const int rows = s.n * group;
  key_range(s, group, window, m * ROWS, min((m + 1) * ROWS, rows), lo, hi);
  return max((int)(((unsigned)hi + UNIT - 1) / UNIT) - lo / UNIT, 1);
}

// Units of all row tiles of one key head.  The lanes of the (converged) warp
// share the tiles.
template <int ROWS, int UNIT>
__device__ __forceinline__ int64_t head_units(const AttnParams& P, const Shape& s, int group) {
  const int tiles = (s.n * group + ROWS - 1) / ROWS;
  int64_t sum = 0;
  int lo, hi;
  for (int m = threadIdx.x & 31; m < tiles; m += 32) sum += tile_units<ROWS, UNIT>(s, group, P.window, m, lo, hi);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// This CTA's share of the work.
struct Range {
  int64_t begin, end, total;
  int64_t share;              // units of a CTA; the first `longer` CTAs have one more
  int longer;
  int64_t req_base, per_head; // units before the request that holds `begin`, units of each of its heads
  int req;
  int ctas;                   // CTAs that have work (the others have none)
};

// a / b for a >= 0, b > 0: in 32 bits where they fit (a 64-bit division takes some hundred cycles).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

__device__ __forceinline__ void set_share(Range& R, int64_t total, int min_units) {
  const int64_t n = divide(total + min_units - 1, min_units);
  const int b = blockIdx.x;
  R.total = total;
  R.ctas = (int)(n < gridDim.x ? n : gridDim.x);
  if (b >= R.ctas) return;
  R.share = divide(total, R.ctas);
  R.longer = (int)(total - R.share * R.ctas);
  R.begin = R.share * b + min(b, R.longer);
  R.end = R.begin + R.share + (b < R.longer ? 1 : 0);
}

__device__ __forceinline__ int64_t scan_up(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// Collective over the block (THREADS threads, a multiple of 32); `scratch` is
// W + 3 words.  Requests are looked at one per lane where none has more than
// one row tile, else one per warp, whose lanes share its tiles.  Up to some
// number of requests every warp does that by itself, without a barrier of the
// block; beyond it the warps share the requests.  us of the whole call, every
// warp | shared, for n requests of one token over 64 keys: n = 1 5.3 | 7.0, 16
// 5.5 | 7.2, 32 10.0 | 10.5, 64 14.7 | 14.4, 128 21.6 | 20.0, 256 37.4 | 34.1,
// 1024 148 | 129; of 17 tokens: 1 12.6 | 15.0, 8 13.7 | 16.0, 32 14.8 | 16.0;
// of 512 tokens over 1024 keys: 4 59.5 | 59.2, 8 90.6 | 88.8, 32 276 | 265.
template <int ROWS, int UNIT, int THREADS>
__device__ __forceinline__ Range share_out(const AttnParams& P, int group, int min_units, int64_t* scratch) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_req = (int)P.n_req;
  const bool single = P.max_q * group <= ROWS;
  Range R{};
  auto units = [&](int r) -> int64_t {                  // single: of the lane's request; else of the warp's
    if (r >= n_req) return 0;
    const Shape s = request(P, r);
    int lo, hi;
    if (single) return s.n ? (int64_t)P.kv_heads * tile_units<ROWS, UNIT>(s, group, P.window, 0, lo, hi) : 0;
    return P.kv_heads * head_units<ROWS, UNIT>(P, s, group);
  };

  if (n_req <= (single ? 128 : 8)) {
    // lane r has request r's units (of the first 32)
    int64_t own = 0, all = 0;
    if (single) {
      own = units(lane);
      for (int r = lane + 32; r < n_req; r += 32) all += units(r);
    } else {
      for (int r = 0; r < n_req; ++r) {
        const int64_t u = units(r);
        if (lane == r) own = u;
      }
    }
    int64_t incl = scan_up(own), base = 0;
    if (n_req > 32) {
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    set_share(R, all + __shfl_sync(0xffffffffu, incl, 31), min_units);
    if ((int)blockIdx.x >= R.ctas) return R;
    for (int r0 = 0;;) {
      const unsigned past = __ballot_sync(0xffffffffu, R.begin < base + incl);
      if (past) {
        const int src = __ffs(past) - 1;
        R.req = r0 + src;
        R.req_base = base + __shfl_sync(0xffffffffu, incl - own, src);
        R.per_head = divide(__shfl_sync(0xffffffffu, own, src), P.kv_heads);
        return R;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
      r0 += 32;
      own = units(r0 + lane);
      incl = scan_up(own);
    }
  }

  const int step = single ? THREADS : W, index = single ? tid : warp;
  int64_t all = 0;
  for (int r = index; r < n_req; r += step) all += units(r);
  if (single)
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if (lane == 0) scratch[warp] = all;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) all += scratch[w];
  set_share(R, all, min_units);
  if ((int)blockIdx.x >= R.ctas) return R;              // the whole block
  int64_t base = 0;
  for (int r0 = 0; r0 < n_req; r0 += step) {
    const int64_t own = units(r0 + index);
    int64_t incl = single ? scan_up(own) : own;
    __syncthreads();
    if (lane == (single ? 31 : 0)) scratch[warp] = incl;
    __syncthreads();
    int64_t sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) incl += scratch[w];
      sum += scratch[w];
    }
    const int64_t at = base + incl - own;
    if ((single || lane == 0) && own > 0 && R.begin >= at && R.begin < at + own) {
      scratch[W] = r0 + index;
      scratch[W + 1] = at;
      scratch[W + 2] = own;
    }
    base += sum;
    if (R.begin < base) break;                          // the same for every thread
  }
  __syncthreads();
  R.req = (int)scratch[W];
  R.req_base = scratch[W + 1];
  R.per_head = divide(scratch[W + 2], P.kv_heads);
  return R;
}

__device__ __forceinline__ int owner(int64_t unit, const Range& R) {
  const int64_t past = unit - (R.share + 1) * R.longer;
  return (int)(past < 0 ? divide(unit, R.share + 1) : R.longer + divide(past, R.share));
}

// The items of a CTA's range, one after another.
template <int ROWS, int UNIT>
struct Walk {
  Shape s;
  int req, head, tile, tiles;
  int64_t at;              // first unit of the item in the order of all
  int units;               // of the item
  int lo, hi;              // its keys
  int u0, u1;              // the item's units that this CTA has

  __device__ __forceinline__ void load(const AttnParams& P, int r, int group) {
    req = r;
    s = request(P, r);
    tiles = (s.n * group + ROWS - 1) / ROWS;
  }
  __device__ __forceinline__ void cut(const Range& R) {
    u0 = (int)(R.begin > at ? R.begin - at : 0);
    u1 = (int)(R.end < at + units ? R.end - at : units);
  }
  // Converged warps: the lanes look for the tile together.
  __device__ __forceinline__ void first(const AttnParams& P, const Range& R, int group) {
    load(P, R.req, group);
    head = (int)divide(R.begin - R.req_base, R.per_head);
    at = R.req_base + head * R.per_head;
    const int lane = threadIdx.x & 31;
    tile = 0;
    for (int m0 = 0; tiles > 1; m0 += 32) {
      const int64_t own = m0 + lane < tiles ? tile_units<ROWS, UNIT>(s, group, P.window, m0 + lane, lo, hi) : 0;
      const int64_t incl = scan_up(own);
      const unsigned past = __ballot_sync(0xffffffffu, R.begin < at + incl);
      if (past) {
        const int src = __ffs(past) - 1;
        tile = m0 + src;
        at += __shfl_sync(0xffffffffu, incl - own, src);
        break;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    units = tile_units<ROWS, UNIT>(s, group, P.window, tile, lo, hi);
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
// threads, `leader` one of them: its fence covers the stores that the barrier
// put before it.
template <class SYNC>
__device__ __forceinline__ bool arrive(unsigned* ticket, int pieces, int* flag, bool leader, SYNC sync) {
  sync();
  if (leader) {
    __threadfence();
    const bool last = atomicAdd(ticket, 1u) == (unsigned)(pieces - 1);
    if (last) {
      *ticket = 0u;                              // ready for the next call
      __threadfence();
    }
    *flag = last;
  }
  sync();
  return *flag != 0;
}

// Add the pieces of CTAs c0..c1 up and write the item's rows: WARPS warps,
// this thread is `t` of them.  weights: kMaxCtas * ROWS shared floats.
template <int ROWS, int D, bool BF16, int WARPS, class SYNC>
__device__ __forceinline__ void combine(const AttnParams& P, const float* pieces, int c0, int c1, const Shape& s,
                                        int head, int group, int row0, int rows, float* weights, int t, SYNC sync) {
  // piece of CTA c: slot 1 (the item starts in its range) for the first, slot 0 for the others
  auto piece = [&](int c) { return pieces + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * piece_floats<ROWS, D>(); };
  const int np = c1 - c0 + 1, lane = t & 31;
  if (np <= 8) {
    // few pieces: a thread per row
    for (int r = t; r < rows; r += 32 * WARPS) {
      float m[8], l[8], top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = k < np ? __ldcg(piece(c0 + k) + ROWS * D + r) : -INFINITY;
        l[k] = k < np ? __ldcg(piece(c0 + k) + ROWS * D + ROWS + r) : 0.f;
        top = fmaxf(top, m[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = m[k] == -INFINITY ? 0.f : ex2(m[k] - top);
        sum += m[k] * l[k];
      }
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < np) weights[k * ROWS + r] = m[k] * inv;
    }
  } else
  // a warp per row: the lanes have its pieces' statistics
  for (int r = t >> 5; r < rows; r += WARPS) {
    constexpr int K = kMaxCtas / 32;
    float m[K], l[K], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = c0 + 32 * k + lane;
      m[k] = c <= c1 ? __ldcg(piece(c) + ROWS * D + r) : -INFINITY;
      l[k] = c <= c1 ? __ldcg(piece(c) + ROWS * D + ROWS + r) : 0.f;
      top = fmaxf(top, m[k]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      m[k] = m[k] == -INFINITY ? 0.f : exp2f(m[k] - top);
      sum += m[k] * l[k];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (32 * k + lane < np) weights[(32 * k + lane) * ROWS + r] = m[k] * inv;
  }
  sync();
  // two outputs' loads of up to eight pieces in flight
  constexpr int B = 8, E = 2;
  for (int e0 = t; e0 < rows * (D / 4); e0 += 32 * WARPS * E) {
    float4 a[E];
#pragma unroll
    for (int i = 0; i < E; ++i) a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < np; c += B) {
      float4 v[E][B];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int e = e0 + 32 * WARPS * i;
#pragma unroll
        for (int k = 0; k < B; ++k)
          if (c + k < np && e < rows * (D / 4)) v[i][k] = __ldcg(reinterpret_cast<const float4*>(piece(c0 + c + k)) + e);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int e = e0 + 32 * WARPS * i;
#pragma unroll
        for (int k = 0; k < B; ++k)
          if (c + k < np && e < rows * (D / 4)) {
            const float w = weights[(c + k) * ROWS + e / (D / 4)];
            a[i].x = fmaf(w, v[i][k].x, a[i].x), a[i].y = fmaf(w, v[i][k].y, a[i].y);
            a[i].z = fmaf(w, v[i][k].z, a[i].z), a[i].w = fmaf(w, v[i][k].w, a[i].w);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = e0 + 32 * WARPS * i, r = e / (D / 4);
      if (e < rows * (D / 4)) store4<BF16>(P.out, P.out_f32, out_row(P, s, head, group, row0 + r) * D + e % (D / 4) * 4, a[i]);
    }
  }
  sync();
}

}  // namespace attn
}  // namespace q4k
