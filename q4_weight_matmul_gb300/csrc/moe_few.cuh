// Products of the experts' matrices with few rows each (decode steps, short
// prompts): the weights stream through shared memory once per tile of 8 NT
// pairs of one expert, so HBM bounds them while an expert has one tile.
//
// y = sum_k w x over a superblock of 256 k, w = d sc q - dmin m (Q4_K) or
// d sc (q - 32) (Q6_K).  Everything that is not a power of two times a small
// integer stays out of the products:
//  - activations: x of a pair and superblock times a power of two that puts
//    the largest in [2^14, 2^15), as two binary16 parts (22 bits);
//  - Q4_K quants enter mma.sync m16n8k16 as binary16 subnormals: the bits of
//    q (or 16 q) in a half are the value q 2^-24, so widening a quant is one
//    AND for two of them, and the products are exact;
//  - a sub-block's (Q6_K: a group's) four (two) products start from zero, and
//    fp32 FMAs add d sc times their sum up; the min term is one product of
//    the eight m with the sub-blocks' sums of x, hi and lo;
//  - the power of two comes off once per superblock.
// Which k an instruction's operands hold is free, so a lane feeds the 4 or 8
// consecutive bytes that it loads without a transpose.
//
// A CTA's warps: 8 consumers, a producer that fills the ring (tensor copies of
// a stage's weights: kTileRows rows of one superblock, 256-value pieces of the
// pairs' activations), and kCvt warps that turn a stage's activations into
// operands in place, in the order in which the consumers' lanes read them.
// Consumers: 8 / KS warps take 32 rows each of every KS-th superblock (KS = 8
// where there are few rows of weights in all, so that every SM gets some), and
// add up their parts at an item's end.  An item is one tile of pairs times
// kOutRows outputs; CTAs take items in turn, tiles of one expert side by side
// so that they share the weights in L2.
//
// Waits are bounded; a warp agrees on a wait's outcome by a vote, and the
// producer waits for its copies before it leaves.  A warp that skips stages
// first waits until its stage has been issued (`issued`), since a parity alone
// could be that of the slot's phase before the last.
#pragma once

#include "mma_sync.cuh"
#include "moe.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

#include <algorithm>

namespace q4k {
namespace few {

enum Mode { kGateUp, kDownQ4, kDownQ6 };

constexpr int kConsumers = 8;
constexpr int kCvt = 3;                      // 12 warps in all: 168 registers a thread (13: 128)
constexpr int kThreads = 32 * (kConsumers + 1 + kCvt);
constexpr int kStep = 576;                   // bytes of an instruction's activations: 32 lanes x 16 bytes, 64 to spare
constexpr int kSums = 16 * kStep;            // the sub-blocks' sums of a tile of 8 pairs: 32 lanes x 8 bytes
constexpr int kInv = kSums + 256;            // the powers of two to take off: 8 floats
constexpr int kTileX = 9600;                 // bytes of a tile's activations (before: 8 rows of 1024)
constexpr int kMaxSmem = 232448 - 1024;

template <int MODE, int NT, int KS>
struct Cfg {
  static constexpr bool kUp = MODE == kGateUp, kQ6 = MODE == kDownQ6;
  static constexpr int kPairs = 8 * NT;
  static constexpr int kGroups = kConsumers / KS;
  static constexpr int kTileRows = 32 * kGroups;
  static constexpr int kOutRows = kUp ? kTileRows / 2 : kTileRows;
  static constexpr int kSb = kQ6 ? kQ6GpuBytes : kBlockBytes;
  static constexpr int kWeights = kTileRows * kSb;
  static constexpr int kScales = kQ6 ? kTileRows * 16 : 0;
  static constexpr int kSlot = kWeights + kScales + NT * kTileX;
  static constexpr int kPart = kGroups * (KS - 1) * 2 * NT * 4 * 32 * (int)sizeof(float);
  static constexpr int kFixed = 8192 + kPart;
  static constexpr int kSlots = (kMaxSmem - kFixed) / kSlot < 16 ? (kMaxSmem - kFixed) / kSlot : 16;
  static constexpr int kSmem = 1024 + kFixed + kSlots * kSlot;
  static_assert(kSlots >= 3 && kSlot % 128 == 0 && kWeights % 128 == 0);
};

struct Params {
  CUtensorMap w;              // rows of the experts' superblocks
  CUtensorMap w2;             // of the up matrices, or the rows' d (Q6_K)
  const float* x;
  const int32_t *order, *offsets;
  float* out;
  int* err;
  int64_t pairs, cols, blocks;   // blocks of kOutRows rows of a matrix
  int rows, nb, experts, top_k;
};

struct Head {                 // at the start of shared memory
  uint64_t full[16], ready[16], empty[16], part_full[8], part_empty[8];
  uint32_t mask[16];          // pairs of a stage that have activations
  uint32_t issued;            // stages whose copies are on their way
  int gave_up;
  int off[kMoeMaxExperts + 1], tiles[kMoeMaxExperts + 33];
};
static_assert(sizeof(Head) <= 8192);

__device__ __forceinline__ bool agreed(bool ok, volatile int* gave_up, int* err) {
  if (__all_sync(~0u, ok)) return true;
  if ((threadIdx.x & 31) == 0) {
    if (!*gave_up) atomicOr(err, 1);
    *gave_up = 1;
  }
  __syncwarp();
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* gave_up, int* err) {
  return agreed(tc::mbar_wait(bar, parity, gave_up), gave_up, err);
}
// Until stage n has been issued.
__device__ __forceinline__ bool warp_wait_issued(const uint32_t* issued, uint32_t n, volatile int* gave_up, int* err) {
  bool ok = true;
  const long long t0 = clock64();
  for (;;) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(tc::smem_u32(issued)) : "memory");
    if ((int32_t)(v - n) > 0) break;
    if (*gave_up || clock64() - t0 > tc::kTimeoutCycles) {
      ok = false;
      break;
    }
  }
  return agreed(ok, gave_up, err);
}

struct Item {
  int expert, first, n;       // pairs order[first] .. first + n - 1
  int64_t block;
};

// The table of tiles; one warp.  Offsets are cut to ascending values of 0..pairs.
__device__ inline void make_tiles(const Params& P, Head& H, int per_tile) {
  const int lane = threadIdx.x & 31, E = P.experts;
  int last = 0, run = 0;
  bool bad = false;
  for (int e0 = 0; e0 <= E; e0 += 32) {
    const int e = e0 + lane, raw = e <= E ? P.offsets[e] : 0;
    int v = raw < 0 ? 0 : raw > P.pairs ? (int)P.pairs : raw;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v = max(v, u);
    }
    v = max(v, last);
    if (e <= E) {
      bad |= v != raw;
      H.off[e] = v;
    }
    last = __shfl_sync(~0u, v, 31);
  }
  __syncwarp();
  for (int e0 = 0; e0 <= E; e0 += 32) {
    const int e = e0 + lane, n = e < E ? (H.off[e + 1] - H.off[e] + per_tile - 1) / per_tile : 0;
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += u;
    }
    H.tiles[e] = e <= E ? run + s - n : INT32_MAX;
    run += __shfl_sync(~0u, s, 31);
  }
  for (int e = (E / 32 + 1) * 32 + lane; e < kMoeMaxExperts + 33; e += 32) H.tiles[e] = INT32_MAX;
  if (bad && blockIdx.x == 0) atomicOr(P.err, kErrIndex);
}

// Item i; the whole warp.
__device__ __forceinline__ Item find_item(const Params& P, const Head& H, int64_t i, int per_tile) {
  const int lane = threadIdx.x & 31;
  const int64_t t = i / P.blocks;
  // the last expert whose first tile is t or before: among every 17th, then among those behind it
  const int a = __popc(__ballot_sync(~0u, lane * 17 <= P.experts && H.tiles[lane * 17] <= t)) - 1;
  const int b = __popc(__ballot_sync(~0u, lane < 17 && H.tiles[a * 17 + lane] <= t)) - 1;
  const int e = a * 17 + b;
  const int tiles = H.tiles[e + 1] - H.tiles[e];
  const int64_t in = i - H.tiles[e] * P.blocks;
  Item r;
  r.expert = e;
  r.block = in / tiles;
  const int k = (int)(in - r.block * tiles);
  r.first = H.off[e] + k * per_tile;
  r.n = min(per_tile, H.off[e + 1] - r.first);
  return r;
}

// ------------------------------------------------------------- activations
// A stage's pieces of 256 activations become operands in place; one warp.
// Two pairs at a time, 16 lanes each; a lane's four consecutive values are one
// lane's operand of one instruction: (0, 2), (1, 3), hi then lo.
template <bool Q6>
__device__ __forceinline__ void convert_tile(uint8_t* tile, uint32_t mask, int lane) {
  const int l = lane & 15, side = lane >> 4;
  float4 v[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int pair = 2 * r + side;
    const bool have = (mask >> pair) & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[r][j] = have ? *reinterpret_cast<const float4*>(tile + 1024 * pair + 16 * l + 256 * j) : make_float4(0, 0, 0, 0);
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int pair = 2 * r + side;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      top = fmaxf(top, fmaxf(fmaxf(fabsf(v[r][j].x), fabsf(v[r][j].y)), fmaxf(fabsf(v[r][j].z), fabsf(v[r][j].w))));
#pragma unroll
    for (int o = 1; o < 16; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    // 2^(141 - E) for the biased exponent E of the largest; 1/s stays a normal float
    const int E = (int)((__float_as_uint(top) >> 23) & 0xFFu), es = top == 0.0f ? 127 : min(253, max(1, 268 - E));
    const float s = __uint_as_float((uint32_t)es << 23);
    if (l == 0) reinterpret_cast<float*>(tile + kInv)[pair] = __uint_as_float((uint32_t)(254 - es) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = v[r][j].x * s, x1 = v[r][j].y * s, x2 = v[r][j].z * s, x3 = v[r][j].w * s;
      const uint32_t h02 = pack2<false>(x0, x2), h13 = pack2<false>(x1, x3);
      const float2 f02 = unpack2<false>(h02), f13 = unpack2<false>(h13);
      const uint32_t l02 = pack2<false>(x0 - f02.x, x2 - f02.y), l13 = pack2<false>(x1 - f13.x, x3 - f13.y);
      // Q4_K: sub-block 2 j + l / 8, bytes 4 (l % 8) ..: a lane's word l % 2 of the 8 bytes from 8 c on, c = l % 8 / 2
      // Q6_K: group 4 j + l / 4, lane c = l % 4
      const int step = Q6 ? 4 * j + (l >> 2) : 2 * (2 * j + (l >> 3)) + (l & 1), c = Q6 ? l & 3 : (l & 7) >> 1;
      *reinterpret_cast<uint4*>(tile + step * kStep + 16 * (4 * pair + c)) = make_uint4(h02, h13, l02, l13);
      if constexpr (!Q6) {
        const float2 e = unpack2<false>(l02), f = unpack2<false>(l13);
        float sum = ((f02.x + f02.y) + (f13.x + f13.y)) + ((e.x + e.y) + (f.x + f.y));
#pragma unroll
        for (int o = 1; o < 8; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
        if ((l & 7) == 0) {
          const int b = 2 * j + (l >> 3);                        // sub-block; its sum times 2^-6, below 2^14
          const __half hi = __float2half_rn(sum * 0.015625f);
          __half* at = reinterpret_cast<__half*>(tile + kSums + 8 * (4 * pair + (b >> 1))) + (b & 1);
          at[0] = hi;
          at[2] = __float2half_rn(sum * 0.015625f - __half2float(hi));
        }
      }
    }
  }
}

// ----------------------------------------------------------------- products
// 2^23 + byte i of w as a float, to become that byte times d by one exact FMA
__device__ __forceinline__ float magic(uint32_t w, int i) { return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + i)); }

__device__ __forceinline__ void add_scaled(float (&t)[4], const float (&a)[4], float low, float high) {
  t[0] = fmaf(low, a[0], t[0]), t[1] = fmaf(low, a[1], t[1]);
  t[2] = fmaf(high, a[2], t[2]), t[3] = fmaf(high, a[3], t[3]);
}

// Two tiles of 16 rows of Q4_K superblocks (`w`: this lane's first row of the
// first; the second `apart` bytes on) times the stage's activations.  A lane
// has rows r and r + 8 with r = 2 (g % 4) + g / 4, so that the 8-byte loads of
// a half-warp (rows 0, 2, 4, 6 x 32 bytes, 144 apart) touch every bank once.
template <int NT>
__device__ __forceinline__ void stage_q4(const uint8_t* w, int apart, const uint8_t* x, int lane, float (&total)[2][NT][4]) {
  const int c = lane & 3;
  uint32_t sc[2][2][2];
  float d[2][2], dmin[2][2];
  uint32_t m[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint4 h = *reinterpret_cast<const uint4*>(w + t * apart + 8 * r * kBlockBytes);
      const float2 dd = unpack2<false>(h.x);
      d[t][r] = dd.x * 16777216.0f, dmin[t][r] = dd.y * -1073741824.0f;       // 2^24; 2^24 and the sums' 2^6
      sc[t][r][0] = h.y & 0x3F3F3F3Fu;
      sc[t][r][1] = (h.w & 0x0F0F0F0Fu) | ((h.y >> 2) & 0x30303030u);
      const uint32_t mins = c < 2 ? h.z & 0x3F3F3F3Fu : ((h.w >> 4) & 0x0F0F0F0Fu) | ((h.z >> 2) & 0x30303030u);
      m[t][r] = __byte_perm(mins, 0, (c & 1) ? 0x4342 : 0x4140);              // m[2 c], m[2 c + 1] times 2^-24
    }
  float sum[2][NT][4] = {};
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    uint2 q[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        q[t][r] = *reinterpret_cast<const uint2*>(w + t * apart + 8 * r * kBlockBytes + 16 + 32 * ch + 8 * c);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int s = 2 * ch + half;
      const uint32_t bits = half ? 0x00F000F0u : 0x000F000Fu;
      uint4 b[2][NT];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          b[i][n] = *reinterpret_cast<const uint4*>(x + n * kTileX + (2 * s + i) * kStep + 16 * lane);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float acc[NT][4] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t u = i ? q[t][0].y : q[t][0].x, v = i ? q[t][1].y : q[t][1].x;
          const uint32_t a[4] = {u & bits, v & bits, (u >> 8) & bits, (v >> 8) & bits};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<false>(acc[n], a, b[i][n].x, b[i][n].y);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<false>(acc[n], a, b[i][n].z, b[i][n].w);
        }
        const float d0 = half ? d[t][0] * 0.0625f : d[t][0], d1 = half ? d[t][1] * 0.0625f : d[t][1];
        const float s0 = fmaf(magic(sc[t][0][s >> 2], s & 3), d0, -8388608.0f * d0),
                    s1 = fmaf(magic(sc[t][1][s >> 2], s & 3), d1, -8388608.0f * d1);
#pragma unroll
        for (int n = 0; n < NT; ++n) add_scaled(sum[t][n], acc[n], s0, s1);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint2 b = *reinterpret_cast<const uint2*>(x + n * kTileX + kSums + 8 * lane);
    const float2 inv = *reinterpret_cast<const float2*>(x + n * kTileX + kInv + 8 * c);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float acc[4] = {};
      const uint32_t a[4] = {m[t][0], m[t][1], m[t][0], m[t][1]};
      mma16816<false>(acc, a, b.x, b.y);
      add_scaled(sum[t][n], acc, dmin[t][0], dmin[t][1]);
      total[t][n][0] = fmaf(inv.x, sum[t][n][0], total[t][n][0]), total[t][n][1] = fmaf(inv.y, sum[t][n][1], total[t][n][1]);
      total[t][n][2] = fmaf(inv.x, sum[t][n][2], total[t][n][2]), total[t][n][3] = fmaf(inv.y, sum[t][n][3], total[t][n][3]);
    }
  }
}

// The same of Q6_K superblocks (GPU layout); `dr`: this lane's first row's
// scale of the superblock, rows 16 bytes apart.  q - 32 is made exactly: the
// nibble and the bit pair (upper bit inverted) under the exponent of 1024 with
// that bit turned back, minus 1056.  A lane has rows g and g + 8: 4-byte loads
// of 8 rows 208 bytes apart touch every bank once.
template <int NT>
__device__ __forceinline__ void stage_q6(const uint8_t* w, const uint8_t* dr, const uint8_t* x, int lane,
                                         float (&total)[2][NT][4]) {
  const int c = lane & 3;
  float d[2][2];
  uint4 sc[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      d[t][r] = __half2float(*reinterpret_cast<const __half*>(dr + (16 * t + 8 * r) * 16));
      sc[t][r] = *reinterpret_cast<const uint4*>(w + (16 * t + 8 * r) * kQ6GpuBytes);
    }
  float sum[2][NT][4] = {};
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t lo[2][2][2], hi[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* p = w + (16 * t + 8 * r) * kQ6GpuBytes + 16 + 48 * ch + 4 * c;
        lo[t][r][0] = *reinterpret_cast<const uint32_t*>(p);
        lo[t][r][1] = *reinterpret_cast<const uint32_t*>(p + 16);
        hi[t][r] = *reinterpret_cast<const uint32_t*>(p + 32);
      }
#pragma unroll
    for (int f = 0; f < 4; ++f) {                                // sub-block f / 2, group f % 2 of it
      uint4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        b[n] = *reinterpret_cast<const uint4*>(x + n * kTileX + (4 * ch + f) * kStep + 16 * lane);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t a[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t l = lo[t][r][f & 1] >> (4 * (f >> 1)), h = hi[t][r];
          const uint32_t h0 = f < 2 ? h << (4 - 2 * f) : h >> (2 * f - 4), h1 = h >> (4 + 2 * f);
          const uint32_t e0 = (l & 0x000F000Fu) ^ ((h0 & 0x00300030u) ^ 0x64206420u),
                         e1 = ((l >> 8) & 0x000F000Fu) ^ ((h1 & 0x00300030u) ^ 0x64206420u);
          const __half2 bias = __floats2half2_rn(-1056.0f, -1056.0f);
          const __half2 v0 = __hadd2(*reinterpret_cast<const __half2*>(&e0), bias),
                        v1 = __hadd2(*reinterpret_cast<const __half2*>(&e1), bias);
          a[r] = *reinterpret_cast<const uint32_t*>(&v0);
          a[2 + r] = *reinterpret_cast<const uint32_t*>(&v1);
        }
        const uint32_t w0 = reinterpret_cast<const uint32_t*>(&sc[t][0])[ch] ^ 0x80808080u,
                       w1 = reinterpret_cast<const uint32_t*>(&sc[t][1])[ch] ^ 0x80808080u;
        const float s0 = (magic(w0, f) - 8388736.0f) * d[t][0], s1 = (magic(w1, f) - 8388736.0f) * d[t][1];   // 2^23 + 128
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float acc[4] = {};
          mma16816<false>(acc, a, b[n].x, b[n].y);
          mma16816<false>(acc, a, b[n].z, b[n].w);
          add_scaled(sum[t][n], acc, s0, s1);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 inv = *reinterpret_cast<const float2*>(x + n * kTileX + kInv + 8 * c);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      total[t][n][0] = fmaf(inv.x, sum[t][n][0], total[t][n][0]), total[t][n][1] = fmaf(inv.y, sum[t][n][1], total[t][n][1]);
      total[t][n][2] = fmaf(inv.x, sum[t][n][2], total[t][n][2]), total[t][n][3] = fmaf(inv.y, sum[t][n][3], total[t][n][3]);
    }
  }
}

// -------------------------------------------------------------------- kernel
template <int MODE, int NT, int KS>
__global__ void __launch_bounds__(kThreads, 1) moe_few_kernel(const __grid_constant__ Params P) {
  using C = Cfg<MODE, NT, KS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  Head& H = *reinterpret_cast<Head*>(smem);
  float* part = reinterpret_cast<float*>(smem + 8192);
  uint8_t* ring = smem + C::kFixed;
  volatile int* gave_up = &H.gave_up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&H.full[i], 1);
      tc::mbar_init(&H.ready[i], 1);
      tc::mbar_init(&H.empty[i], C::kGroups);
    }
    for (int i = 0; i < C::kGroups; ++i) {
      tc::mbar_init(&H.part_full[i], KS - 1);
      tc::mbar_init(&H.part_empty[i], 1);
    }
    H.issued = 0;
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kConsumers) make_tiles(P, H, C::kPairs);
  __syncthreads();
  const int64_t items = H.tiles[P.experts] * P.blocks;
  const int nb = P.nb;

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    uint32_t n = 0;
    bool stop = false;
    for (int64_t i = blockIdx.x; i < items && !stop; i += gridDim.x) {
      const Item it = find_item(P, H, i, C::kPairs);
      int64_t row = -1;
      if (lane < it.n) {
        row = it.first + lane;
        if constexpr (C::kUp) {
          const int p = P.order[row];
          row = p >= 0 && p < P.pairs ? p / P.top_k : -1;
          if (row < 0) atomicOr(P.err, kErrIndex);
        }
      }
      __syncwarp();
      const uint32_t mask = __ballot_sync(~0u, row >= 0);
      const float* src = P.x + row * P.cols;
      const int w0 = (int)(it.expert * (int64_t)P.rows + it.block * C::kOutRows);
      for (int sb = 0; sb < nb; ++sb, ++n) {
        const uint32_t slot = n % C::kSlots;
        if (!warp_wait(&H.empty[slot], ((n / C::kSlots) & 1) ^ 1, gave_up, P.err)) {
          stop = true;
          break;
        }
        uint8_t* at = ring + slot * C::kSlot;
        tc::fence_proxy_async_smem();                            // the activations were rewritten in place
        if (lane == 0) {
          H.mask[slot] = mask;
          tc::mbar_arrive_expect_tx(&H.full[slot], C::kWeights + C::kScales + 1024 * __popc(mask));
          tc::tma_load_3d(at, &P.w, 0, w0, sb, &H.full[slot]);
          if constexpr (C::kUp) tc::tma_load_3d(at + C::kWeights / 2, &P.w2, 0, w0, sb, &H.full[slot]);
          if constexpr (C::kQ6) tc::tma_load_2d(at + C::kWeights, &P.w2, sb & ~7, w0, &H.full[slot]);
        }
        __syncwarp();
        if (row >= 0)
          tc::bulk_g2s(at + C::kWeights + C::kScales + (lane >> 3) * kTileX + (lane & 7) * 1024, src + sb * kQK, 1024,
                       &H.full[slot]);
        __syncwarp();
        if (lane == 0)
          asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(tc::smem_u32(&H.issued)), "r"(n + 1) : "memory");
      }
    }
    // its copies land before the CTA ends
    if (lane == 0)
      for (uint32_t j = n < C::kSlots ? 0 : n - C::kSlots; j < n; ++j)
        if (!tc::mbar_wait_sleep(&H.full[j % C::kSlots], (j / C::kSlots) & 1)) break;
  } else if (warp > kConsumers) {
    // ---------------------------------------------------------- activations
    const int64_t mine = items > blockIdx.x ? (items - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    const uint32_t stages = (uint32_t)(mine * nb);
    for (uint32_t n = warp - kConsumers - 1; n < stages; n += kCvt) {
      const uint32_t slot = n % C::kSlots;
      if (!warp_wait_issued(&H.issued, n, gave_up, P.err) ||
          !warp_wait(&H.full[slot], (n / C::kSlots) & 1, gave_up, P.err))
        break;
      const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&H.mask[slot]);
      uint8_t* at = ring + slot * C::kSlot + C::kWeights + C::kScales;
#pragma unroll 1
      for (int t = 0; t < NT; ++t) convert_tile<C::kQ6>(at + t * kTileX, (mask >> (8 * t)) & 0xFFu, lane);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&H.ready[slot]);
    }
  } else {
    // ------------------------------------------------------------- products
    const int group = warp % C::kGroups, share = warp / C::kGroups;
    const int g = lane >> 2, c = lane & 3;
    const int r0 = C::kQ6 ? g : 2 * (g & 3) + (g >> 2);
    // the warp's first row in a stage; gate and up: 16 rows of both halves
    const int base = C::kUp ? 16 * group : 32 * group;
    const int apart = (C::kUp ? C::kTileRows / 2 : 16) * C::kSb;
    uint32_t first = 0, turn = 0;
    bool stop = false;
    for (int64_t i = blockIdx.x; i < items && !stop; i += gridDim.x, first += nb, ++turn) {
      float total[2][NT][4] = {};
      for (int sb = share; sb < nb; sb += KS) {
        const uint32_t n = first + sb, slot = n % C::kSlots, parity = (n / C::kSlots) & 1;
        if (!warp_wait_issued(&H.issued, n, gave_up, P.err) || !warp_wait(&H.full[slot], parity, gave_up, P.err) ||
            !warp_wait(&H.ready[slot], parity, gave_up, P.err)) {
          stop = true;
          break;
        }
        const uint8_t* at = ring + slot * C::kSlot;
        const uint8_t* x = at + C::kWeights + C::kScales;
        if constexpr (C::kQ6)
          stage_q6<NT>(at + (base + r0) * C::kSb, at + C::kWeights + (base + r0) * 16 + 2 * (sb & 7), x, lane, total);
        else
          stage_q4<NT>(at + (base + r0) * C::kSb, apart, x, lane, total);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&H.empty[slot]);
      }
      if (stop) break;
      if constexpr (KS > 1) {
        constexpr int kValues = 2 * NT * 4;
        if (share > 0) {
          float* mine = part + (group * (KS - 1) + share - 1) * kValues * 32 + lane;
          if (!warp_wait(&H.part_empty[group], (turn & 1) ^ 1, gave_up, P.err)) break;
#pragma unroll
          for (int j = 0; j < kValues; ++j) mine[32 * j] = total[j / (4 * NT)][(j / 4) % NT][j % 4];
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&H.part_full[group]);
          continue;
        }
        if (!warp_wait(&H.part_full[group], turn & 1, gave_up, P.err)) break;
        for (int s = 0; s < KS - 1; ++s) {
          const float* other = part + (group * (KS - 1) + s) * kValues * 32 + lane;
#pragma unroll
          for (int j = 0; j < kValues; ++j) total[j / (4 * NT)][(j / 4) % NT][j % 4] += other[32 * j];
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&H.part_empty[group]);
      }
      const Item it = find_item(P, H, i, C::kPairs);
#pragma unroll
      for (int t = 0; t < (C::kUp ? 1 : 2); ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t row = it.block * C::kOutRows + base + 16 * t + r0 + 8 * (j >> 1);
            const int col = 8 * n + 2 * c + (j & 1);
            if (row < P.rows && col < it.n) {
              float v = total[t][n][j];
              if constexpr (C::kUp) v = v / (1.0f + expf(-v)) * total[1][n][j];
              P.out[(int64_t)(it.first + col) * P.rows + row] = v;
            }
          }
    }
  }
}

template <int MODE, int NT, int KS>
cudaError_t launch(const MoeProduct& p, float* out, cudaStream_t s) {
  using C = Cfg<MODE, NT, KS>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(moe_few_kernel<MODE, NT, KS>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  Params P{};
  const int64_t rows = p.rows * p.plan.experts, nb = p.cols / kQK;
  const int64_t pitch = C::kQ6 ? q6k_gpu_row_bytes(nb) : nb * kBlockBytes;
  const uint64_t dims[3] = {(uint64_t)C::kSb, (uint64_t)rows, (uint64_t)nb};
  const uint64_t strides[2] = {(uint64_t)pitch, (uint64_t)C::kSb};
  const uint32_t box[3] = {(uint32_t)C::kSb, (uint32_t)(C::kUp ? C::kTileRows / 2 : C::kTileRows), 1};
  if (!encode_tmap_u8_3d(&P.w, p.w, dims, strides, box)) return cudaErrorInvalidValue;
  if (C::kUp && !encode_tmap_u8_3d(&P.w2, p.up, dims, strides, box)) return cudaErrorInvalidValue;
  if (C::kQ6 && !encode_tmap_2d(&P.w2, CU_TENSOR_MAP_DATA_TYPE_UINT16, p.w + nb * kQ6GpuBytes, (uint64_t)nb,
                                (uint64_t)rows, (uint64_t)pitch, 8, C::kTileRows, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  P.x = p.x, P.order = p.plan.order, P.offsets = p.plan.offsets, P.out = out, P.err = p.err;
  P.pairs = p.plan.tokens * p.plan.top_k, P.cols = p.cols, P.blocks = (p.rows + C::kOutRows - 1) / C::kOutRows;
  P.rows = (int)p.rows, P.nb = (int)nb, P.experts = p.plan.experts, P.top_k = p.plan.top_k;
  int dev = 0;
  cudaGetDevice(&dev);
  const int64_t most = std::min(P.pairs, P.pairs / C::kPairs + P.experts) * P.blocks;
  moe_few_kernel<MODE, NT, KS><<<(unsigned)std::min<int64_t>(most, device_info(dev).sm_count), kThreads, C::kSmem, s>>>(P);
  return cudaGetLastError();
}

// The variant for a product of `rows` outputs.
template <int MODE>
cudaError_t launch_mode(const MoeProduct& p, float* out, cudaStream_t s) {
  const int64_t pairs = p.plan.tokens * p.plan.top_k, used = std::min<int64_t>(pairs, p.plan.experts);
  if (pairs <= 8 * used) {
    // a block of rows for each of four groups of warps, unless that leaves SMs without one
    if (used * ((p.rows + 63) / 64) >= 2 * 152) return launch<MODE, 1, 2>(p, out, s);
    return launch<MODE, 1, 8>(p, out, s);
  }
  if (pairs <= 16 * used) return launch<MODE, 2, 2>(p, out, s);
  return launch<MODE, 4, 2>(p, out, s);
}

}  // namespace few
}  // namespace q4k
