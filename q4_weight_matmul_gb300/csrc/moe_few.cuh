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
//    4 q (or 64 q) in a half are the value q 2^-22, so widening two quants is
//    a shift for two masks, and the products are exact.  (Sums lose what lies
//    below the largest product's exponent, taken as that of a normal number:
//    with q 2^-24, one shift less, the relative error of h was 1.9e-6, now 4e-7);
//  - a sub-block's (Q6_K: a group's) four (two) products start from zero, and
//    fp32 FMAs add d sc times their sum up; the min term is one product of
//    the eight m with the sub-blocks' sums of x, hi and lo;
//  - the power of two comes off once per superblock.
// Which k an instruction's operands hold is free, so a lane feeds the 4 or 8
// consecutive bytes that it loads without a transpose.
//
// The activations' operands depend on neither the rows nor the matrix, so a
// first launch makes them once, in the order in which the lanes read them, and
// the products copy them beside the weights (made in every CTA by warps of its
// own they held the products up: 64 users x 8 of 128 experts 107 us).
//
// A CTA's warps: 12 consumers, three that copy weights into the ring (a stage:
// kTileRows rows of one superblock; 16 bytes a lane, since tensor copies of
// 144-byte rows take longer than memory: 64 users 79 us) and one that draws
// the items and copies the pairs' operands.  Consumers: four
// groups of 32 rows; the three warps of a group take every third superblock
// and add up their parts at an item's end.  An item is one tile of pairs times
// kOutRows outputs.  CTAs draw items from a counter, experts with many pairs
// first, so that the last to end are short; tiles of one expert lie side by
// side and share the weights in L2.
//
// Measured: one token, 8 of 128 experts of 2048 x 768, gate and up 9.7 us, down
// Q6_K 10.6; 64 tokens 68 us (3.3 TB/s), down 46; 12 tokens, 2 of 8 experts of
// 4096 x 12288, 97 us (4.7 TB/s), of which the stream of the weights alone takes
// 70.  Nothing in it is full: with 64 tokens (2048 columns) instructions issue in
// 48 % of the cycles, the pipe of shifts and masks works in 38 % (down Q6_K 47),
// the tensor pipe in 25 %, shared memory in 32 %, and HBM gives half its rate.
// Bound: latency and hand-over.  The largest share of the warps' time is waits
// for memory and barriers (3.4 of some 7 warps a scheduler has); an item of 2048
// columns is eight stages for three warps, and ends with a chain of three
// hand-overs of sums.  One token: the latency of two launches.
//
// Waits are bounded; a warp agrees on a wait's outcome by a vote, and who
// copies waits for its copies before it leaves.
#pragma once

#include "mma_sync.cuh"
#include "moe.cuh"
#include "tc_ptx.cuh"

#include <algorithm>

namespace q4k {
namespace few {

enum Mode { kGateUp, kDownQ4, kDownQ6 };

constexpr int kGroups = 4, kShares = 3;      // consumer warps: four groups of 32 rows, each shared by three
constexpr int kConsumers = kGroups * kShares;
constexpr int kCopiers = 3, kLead = kConsumers + kCopiers;     // warps that copy weights; the one that leads
constexpr int kThreads = 32 * (kLead + 1);
constexpr int kTileRows = 32 * kGroups;
constexpr int kMaxSmem = 232448 - 1024, kHeadBytes = 8064;
// The operands of 8 pairs and a superblock: 16 instructions x 32 lanes x 16
// bytes (of up to four pairs: x 8), the sub-blocks' sums of x (32 lanes x 8
// bytes), the powers of two to take off (8 floats).
constexpr int kTileX = 16 * 512 + 256 + 32, kHalfX = 16 * 256 + 256 + 32;
constexpr int kQueue = 4;                    // items on their way from the producer to the consumers

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
// An arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

template <int MODE, int NT>
struct Cfg {
  static constexpr bool kUp = MODE == kGateUp, kQ6 = MODE == kDownQ6;
  static constexpr int kPairs = 8 * NT;
  static constexpr int kOutRows = kUp ? kTileRows / 2 : kTileRows;
  static constexpr int kSb = kQ6 ? kQ6GpuBytes : kBlockBytes;
  static constexpr int kWeights = kTileRows * kSb;
  static constexpr int kScales = kQ6 ? kTileRows * 4 : 0;            // the rows' d of two superblocks
  static constexpr int kSlot = (kWeights + kScales + NT * kTileX + 127) / 128 * 128;
  static constexpr int kValues = 2 * NT * 4;                        // sums of a lane
  static constexpr int kFixed = kHeadBytes + kGroups * kValues * 32 * (int)sizeof(float);
  // Where a slot serves one share alone, a warp sees every phase of the slots
  // it waits for.  Elsewhere it waits first until its stage has been issued: a
  // parity alone could be that of the slot's phase before the last.
  static constexpr int kRoom = (kMaxSmem - kFixed) / kSlot;
  static constexpr int kSlots = kRoom >= 2 * kShares ? kRoom / kShares * kShares : kRoom;
  static constexpr bool kOwnSlots = kSlots % kShares == 0;
  static constexpr int kSmem = 1024 + kFixed + kSlots * kSlot;
  static_assert(kSlots >= 3 && kSlots <= 12 && kWeights % 128 == 0 && kFixed % 128 == 0);
};

struct Params {
  const uint8_t *w, *up;      // the experts' matrices, rows of `pitch` bytes
  const uint8_t* x;           // operands [eighths of tiles][nb][kTileX]
  const int32_t* offsets;
  int32_t* counter;
  float* out;
  int* err;
  int64_t pairs, pitch;
  uint32_t blocks;            // of kOutRows rows of a matrix
  int rows, nb, experts;
};

struct SplitParams {
  const float* x;
  const int32_t *order, *offsets;
  uint8_t* out;
  int32_t* counter;
  int* err;
  int64_t pairs, cols;
  int nb, experts, top_k;     // top_k 0: x has a row for every pair
};

// Until stage n has been issued.
template <long long kTimeoutCycles = tc::kTimeoutCycles>
__device__ __forceinline__ bool warp_wait_issued(const uint32_t* issued, uint32_t n, volatile int* gave_up, int* err) {
  bool ok = true;
  const long long t0 = clock64();
  for (;;) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(tc::smem_u32(issued)) : "memory");
    if ((int32_t)(v - n) > 0) break;
    if (*gave_up || clock64() - t0 > kTimeoutCycles) {
      ok = false;
      break;
    }
    __nanosleep(40);
  }
  return agreed(ok, gave_up, err);
}

// Which pairs each expert has, and the tiles of up to `per_tile` of them that
// they make: experts in `perm`'s order (those with more than 8 pairs, with
// more than 4, the rest), position i's tiles from first[i] on.
struct Tiles {
  int off[kMoeMaxExperts + 1], eighth[kMoeMaxExperts];   // an expert's first pair, its first group of 8 pairs
  int first[kMoeMaxExperts + 33];
  uint16_t perm[kMoeMaxExperts];
  int warps[16];
};
struct Head {                 // at the start of shared memory
  uint64_t full[12], empty[12], part[kGroups][kShares], item_full[kQueue], item_empty[kQueue];
  int4 item[kQueue];          // expert, block, first pair, pairs; no pairs: the end
  uint32_t issued;            // stages whose copies are on their way
  int gave_up;
  Tiles tiles;
};
static_assert(sizeof(Head) <= kHeadBytes);

struct Item {
  int expert, block;
  int first, n;               // pairs order[first] .. first + n - 1
};

// The tables; a whole block, each thread for kMoeMaxExperts / THREADS
// experts.  Offsets are cut to ascending values of 0..pairs.  Returns the
// number of tiles.
template <int THREADS, int PER_TILE>
__device__ __forceinline__ int make_tiles(Tiles& T, const int32_t* offsets, int E, int pairs, int* err) {
  constexpr int J = kMoeMaxExperts / THREADS;
  const int e0 = threadIdx.x * J;
  int raw[J + 1], v[J + 1], all;
#pragma unroll
  for (int j = 0; j <= J; ++j) raw[j] = e0 + j <= E ? offsets[e0 + j] : INT32_MAX;
  for (int i = threadIdx.x; i < kMoeMaxExperts + 33; i += THREADS) T.first[i] = INT32_MAX;
  int top = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) top = max(top, min(raw[j], pairs));             // beyond E: pairs, past every expert
  int last = scan_block<THREADS, true>(top, T.warps, all);
  bool bad = e0 == 0 && raw[0] != 0;                                          // pairs before the first expert's
  int classes = 0, eighths = 0;                                               // three counts of ten bits
#pragma unroll
  for (int j = 0; j <= J; ++j) {
    last = v[j] = max(last, min(raw[j], pairs));
    bad |= e0 + j <= E && v[j] != raw[j];
    if (j > 0 && e0 + j <= E) {
      const int n = v[j] - v[j - 1];
      eighths += (n + 7) / 8;
      classes += n > 8 ? 1 : n > 4 ? 1 << 10 : 1 << 20;
    }
  }
  int count;
  int at = scan_block<THREADS, false>(classes, T.warps, count);
  eighths = scan_block<THREADS, false>(eighths, T.warps, all);
  int p0 = at & 1023, p1 = (count & 1023) + (at >> 10 & 1023), p2 = (count & 1023) + (count >> 10 & 1023) + (at >> 20);
#pragma unroll
  for (int j = 0; j <= J; ++j) {
    if (e0 + j <= E && (j < J || e0 + j == kMoeMaxExperts)) T.off[e0 + j] = v[j];
    if (j < J && e0 + j < E) {
      const int n = v[j + 1] - v[j];
      T.eighth[e0 + j] = eighths;
      eighths += (n + 7) / 8;
      T.perm[n > 8 ? p0++ : n > 4 ? p1++ : p2++] = (uint16_t)(e0 + j);
    }
  }
  if (bad && blockIdx.x == 0) atomicOr(err, kErrIndex);
  __syncthreads();
  int tiles[J], sum = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    tiles[j] = 0;
    if (e0 + j < E) {
      const int e = T.perm[e0 + j];
      tiles[j] = (T.off[e + 1] - T.off[e] + PER_TILE - 1) / PER_TILE;
    }
    sum += tiles[j];
  }
  int first = scan_block<THREADS, false>(sum, T.warps, all);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (e0 + j <= E) T.first[e0 + j] = first;
    first += tiles[j];
  }
  if (E == kMoeMaxExperts && threadIdx.x == 0) T.first[E] = all;
  __syncthreads();
  return all;
}

// Item i of items of `blocks` blocks a tile; the whole warp.
__device__ __forceinline__ Item find_item(const Tiles& T, uint32_t i, uint32_t blocks, int per_tile) {
  const int lane = threadIdx.x & 31;
  const int t = (int)(i / blocks);
  // the last position whose first tile is t or before: among every 17th, then among those behind it
  const int a = __popc(__ballot_sync(~0u, T.first[lane * 17] <= t)) - 1;
  const int b = __popc(__ballot_sync(~0u, lane < 17 && T.first[a * 17 + lane] <= t)) - 1;
  const int k = a * 17 + b;
  const uint32_t tiles = T.first[k + 1] - T.first[k], in = i - T.first[k] * blocks;
  Item r;
  r.expert = T.perm[k];
  r.block = (int)(in / tiles);
  r.first = T.off[r.expert] + (int)(in - r.block * tiles) * per_tile;
  r.n = min(per_tile, T.off[r.expert + 1] - r.first);
  return r;
}

// ------------------------------------------------------------- activations
// The operands of 8 pairs and a superblock; one warp.  Two pairs at a time, 16
// lanes each; a lane's four consecutive values are one lane's operand of one
// instruction: (0, 2), (1, 3), hi then lo.  With up to four pairs (HALF) the
// hi parts are the columns 0..3 and the lo parts the columns 4..7 of one
// product.  `row`: lane i's pair's activations, NULL for zeros.  The columns
// behind the n pairs stay as they are: no result is stored from them.
template <bool Q6, bool HALF>
__device__ __forceinline__ void make_operands(uint8_t* tile, const float* row, int n, int lane) {
  const int l = lane & 15, side = lane >> 4;
  constexpr int kRounds = HALF ? 2 : 4, kSums = HALF ? 16 * 256 : 16 * 512, kInv = kSums + 256;
  float4 v[kRounds][4];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const float* from = reinterpret_cast<const float*>(__shfl_sync(~0u, (unsigned long long)row, 2 * r + side));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[r][j] = from ? reinterpret_cast<const float4*>(from)[l + 16 * j] : make_float4(0, 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (2 * r >= n) break;
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
    if (l < (HALF ? 2 : 1)) reinterpret_cast<float*>(tile + kInv)[pair + 4 * l] = __uint_as_float((uint32_t)(254 - es) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = v[r][j].x * s, x1 = v[r][j].y * s, x2 = v[r][j].z * s, x3 = v[r][j].w * s;
      const uint32_t h02 = pack2<false>(x0, x2), h13 = pack2<false>(x1, x3);
      const float2 f02 = unpack2<false>(h02), f13 = unpack2<false>(h13);
      const uint32_t l02 = pack2<false>(x0 - f02.x, x2 - f02.y), l13 = pack2<false>(x1 - f13.x, x3 - f13.y);
      // Q4_K: sub-block 2 j + l / 8, bytes 4 (l % 8) ..: a lane's word l % 2 of the 8 bytes from 8 c on, c = l % 8 / 2
      // Q6_K: group 4 j + l / 4, lane c = l % 4
      const int step = Q6 ? 4 * j + (l >> 2) : 2 * (2 * j + (l >> 3)) + (l & 1), c = Q6 ? l & 3 : (l & 7) >> 1;
      if constexpr (HALF) {
        *reinterpret_cast<uint2*>(tile + step * 256 + 8 * (4 * pair + c)) = make_uint2(h02, h13);
        *reinterpret_cast<uint2*>(tile + step * 256 + 8 * (4 * pair + 16 + c)) = make_uint2(l02, l13);
      } else {
        *reinterpret_cast<uint4*>(tile + step * 512 + 16 * (4 * pair + c)) = make_uint4(h02, h13, l02, l13);
      }
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
  if constexpr (HALF && !Q6)
    if (side) *reinterpret_cast<uint2*>(tile + kSums + 128 + 8 * l) = make_uint2(0, 0);   // columns 4..7
}

constexpr int kSplitWarps = 4;

// A CTA for each group of 8 pairs, its warps for the superblocks.
template <bool Q6>
__global__ void __launch_bounds__(32 * kSplitWarps) moe_few_split_kernel(const SplitParams P, int per_tile) {
  __shared__ Tiles T;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 32) *P.counter = 0;
  if ((int)blockIdx.x >= make_tiles<32 * kSplitWarps, 8>(T, P.offsets, P.experts, (int)P.pairs, P.err)) return;
  const Item it = find_item(T, blockIdx.x, 1, 8);
  const int k = (it.first - T.off[it.expert]) / per_tile;                    // the tile that the group is part of
  const bool half = min(per_tile, T.off[it.expert + 1] - T.off[it.expert] - k * per_tile) <= 4;
  const float* row = nullptr;
  if (lane < it.n) {
    int64_t r = it.first + lane;
    if (P.top_k) {
      const int p = P.order[r];
      r = p >= 0 && p < P.pairs ? p / P.top_k : -1;
      if (r < 0 && warp == 0) atomicOr(P.err, kErrIndex);
    }
    if (r >= 0) row = P.x + r * P.cols;
  }
  const int64_t eighth = T.eighth[it.expert] + (it.first - T.off[it.expert]) / 8;
  for (int sb = blockIdx.y * kSplitWarps + warp; sb < P.nb; sb += gridDim.y * kSplitWarps) {
    uint8_t* tile = P.out + (eighth * P.nb + sb) * kTileX;
    const float* at = row ? row + sb * kQK : nullptr;
    if (half) make_operands<Q6, true>(tile, at, it.n, lane);
    else make_operands<Q6, false>(tile, at, it.n, lane);
  }
}

// ----------------------------------------------------------------- products
// 2^23 + byte i of w as a float, to become that byte times d by one exact FMA
__device__ __forceinline__ float magic(uint32_t w, int i) { return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + i)); }

// A lane's activations of one instruction: hi in x, y, lo in z, w (HALF: x, y alone).
template <bool HALF>
__device__ __forceinline__ uint4 operand(const uint8_t* x, int step, int lane) {
  if constexpr (HALF) {
    const uint2 v = *reinterpret_cast<const uint2*>(x + step * 256 + 8 * lane);
    return make_uint4(v.x, v.y, 0, 0);
  } else {
    return *reinterpret_cast<const uint4*>(x + step * 512 + 16 * lane);
  }
}

__device__ __forceinline__ void add_scaled(float (&t)[4], const float (&a)[4], float low, float high) {
  t[0] = fmaf(low, a[0], t[0]), t[1] = fmaf(low, a[1], t[1]);
  t[2] = fmaf(high, a[2], t[2]), t[3] = fmaf(high, a[3], t[3]);
}

// Two tiles of 16 rows of Q4_K superblocks (`w`: this lane's first row of the
// first; the second `apart` bytes on) times the stage's activations.  A lane
// has rows r and r + 8 with r = 2 (g % 4) + g / 4, so that the 8-byte loads of
// a half-warp (rows 0, 2, 4, 6 x 32 bytes, 144 apart) touch every bank once.
template <int NT, bool HALF>
__device__ __forceinline__ void stage_q4(const uint8_t* w, int apart, const uint8_t* x, int lane, float (&total)[2][NT][4]) {
  constexpr int kSums = HALF ? 16 * 256 : 16 * 512;
  const int c = lane & 3;
  // a 4 that the compiler does not know: products go to another pipe than the shifts and masks that it would make of them
  // (64 tokens' gate and up 69.4 -> 68.2 us; the same of >> 6, the high half of a product, is slower)
  uint32_t four;
  asm volatile("mov.u32 %0, 4;" : "=r"(four));
  uint32_t sc[2][2][2];
  float d[2][2], dmin[2][2];
  uint32_t m[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint4 h = *reinterpret_cast<const uint4*>(w + t * apart + 8 * r * kBlockBytes);
      const float2 dd = unpack2<false>(h.x);
      d[t][r] = dd.x * 4194304.0f, dmin[t][r] = dd.y * -67108864.0f;          // 2^22; 2^20 and the sums' 2^6
      sc[t][r][0] = h.y & 0x3F3F3F3Fu;
      sc[t][r][1] = (h.w & 0x0F0F0F0Fu) | ((h.y >> 2) & 0x30303030u);
      const uint32_t mins = c < 2 ? h.z & 0x3F3F3F3Fu : ((h.w >> 4) & 0x0F0F0F0Fu) | ((h.z >> 2) & 0x30303030u);
      m[t][r] = __byte_perm(mins, 0, (c & 1) ? 0x4342 : 0x4140) << 4;         // m[2 c], m[2 c + 1] times 2^-20
    }
  float sum[2][NT][4] = {};
  // A chunk of 64 k has four sums in the making (two sub-blocks, two tiles of
  // rows): taken in turn, none waits for its product before.
  constexpr int kTogether = NT == 1 ? 2 : 1;                   // sub-blocks at a time
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    uint2 q[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        q[t][r] = *reinterpret_cast<const uint2*>(w + t * apart + 8 * r * kBlockBytes + 16 + 32 * ch + 8 * c);
#pragma unroll
    for (int first = 0; first < 2; first += kTogether) {
      float acc[kTogether][2][NT][4] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 b[kTogether][NT];
#pragma unroll
        for (int h = 0; h < kTogether; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n) b[h][n] = operand<HALF>(x + n * kTileX, 2 * (2 * ch + first + h) + i, lane);
        uint32_t a[kTogether][2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t u = i ? q[t][0].y : q[t][0].x, v = i ? q[t][1].y : q[t][1].x;
#pragma unroll
          for (int h = 0; h < kTogether; ++h) {
            const uint32_t bits = first + h ? 0x03C003C0u : 0x003C003Cu;
            a[h][t][0] = u * four & bits, a[h][t][1] = v * four & bits, a[h][t][2] = u >> 6 & bits, a[h][t][3] = v >> 6 & bits;
          }
        }
#pragma unroll
        for (int h = 0; h < kTogether; ++h)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<false>(acc[h][t][n], a[h][t], b[h][n].x, b[h][n].y);
        if constexpr (!HALF)
#pragma unroll
          for (int h = 0; h < kTogether; ++h)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<false>(acc[h][t][n], a[h][t], b[h][n].z, b[h][n].w);
      }
#pragma unroll
      for (int h = 0; h < kTogether; ++h) {
        const int s = 2 * ch + first + h;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float d0 = s & 1 ? d[t][0] * 0.0625f : d[t][0], d1 = s & 1 ? d[t][1] * 0.0625f : d[t][1];
          const float s0 = fmaf(magic(sc[t][0][s >> 2], s & 3), d0, -8388608.0f * d0),
                      s1 = fmaf(magic(sc[t][1][s >> 2], s & 3), d1, -8388608.0f * d1);
#pragma unroll
          for (int n = 0; n < NT; ++n) add_scaled(sum[t][n], acc[h][t][n], s0, s1);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint2 b = *reinterpret_cast<const uint2*>(x + n * kTileX + kSums + 8 * lane);
    const float2 inv = *reinterpret_cast<const float2*>(x + n * kTileX + kSums + 256 + 8 * c);
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
// scale of the superblock, rows 4 bytes apart.  q - 32 is made exactly: the
// nibble and the bit pair (upper bit inverted) under the exponent of 1024 with
// that bit turned back, minus 1056.  A lane has rows g and g + 8: 4-byte loads
// of 8 rows 208 bytes apart touch every bank once.
template <int NT, bool HALF>
__device__ __forceinline__ void stage_q6(const uint8_t* w, const uint8_t* dr, const uint8_t* x, int lane,
                                         float (&total)[2][NT][4]) {
  constexpr int kSums = HALF ? 16 * 256 : 16 * 512;
  const int c = lane & 3;
  float d[2][2];
  uint4 sc[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      d[t][r] = __half2float(*reinterpret_cast<const __half*>(dr + (16 * t + 8 * r) * 4));
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
        b[n] = operand<HALF>(x + n * kTileX, 4 * ch + f, lane);
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
          if constexpr (!HALF) mma16816<false>(acc, a, b[n].z, b[n].w);
          add_scaled(sum[t][n], acc, s0, s1);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 inv = *reinterpret_cast<const float2*>(x + n * kTileX + kSums + 256 + 8 * c);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      total[t][n][0] = fmaf(inv.x, sum[t][n][0], total[t][n][0]), total[t][n][1] = fmaf(inv.y, sum[t][n][1], total[t][n][1]);
      total[t][n][2] = fmaf(inv.x, sum[t][n][2], total[t][n][2]), total[t][n][3] = fmaf(inv.y, sum[t][n][3], total[t][n][3]);
    }
  }
}

// -------------------------------------------------------------------- kernel
// A consumer warp's part of an item of up to 8 N pairs: its superblocks, the
// sums of its group's warps put together, the results stored.  False: a wait
// gave up.
template <class C, int N, bool HALF>
__device__ __forceinline__ bool consume(const Params& P, Head& H, float* part, const uint8_t* ring, const Item& it,
                                        uint32_t first, uint32_t turn) {
  volatile int* gave_up = &H.gave_up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp % kGroups;
  // The stages' shares go on from item to item, so that a slot stays one share's.  `rank`: which superblocks of this item
  // (every third) they are; the sums are put together by rank, the same way wherever the item comes.
  const int share = warp / kGroups, rank = (share + kShares - first % kShares) % kShares;
  const int c = lane & 3, r0 = C::kQ6 ? lane >> 2 : 2 * ((lane >> 2) & 3) + (lane >> 4);
  // the warp's first row in a stage; gate and up: 16 rows of both halves
  const int base = C::kUp ? 16 * group : 32 * group;
  float total[2][N][4] = {};
  for (uint32_t n = first + rank; n < first + P.nb; n += kShares) {
    const uint32_t slot = n % C::kSlots, sb = n - first;
    if (!C::kOwnSlots && !warp_wait_issued(&H.issued, n, gave_up, P.err)) return false;
    if (!warp_wait(&H.full[slot], (n / C::kSlots) & 1, gave_up, P.err)) return false;
    const uint8_t* at = ring + slot * C::kSlot;
    const uint8_t* x = at + C::kWeights + C::kScales;
    if constexpr (C::kQ6)
      stage_q6<N, HALF>(at + (base + r0) * C::kSb, at + C::kWeights + (base + r0) * 4 + 2 * (sb & 1), x, lane, total);
    else
      stage_q4<N, HALF>(at + (base + r0) * C::kSb, (C::kUp ? kTileRows / 2 : 16) * C::kSb, x, lane, total);
    warp_release(&H.empty[slot]);
  }
  // the ranks' sums, one after the other through the group's place: rank 2, 1, 0, when that of the item before is done
  constexpr int kSums = 8 * N;
  float* place = part + group * C::kValues * 32 + lane;
  if (!warp_wait(&H.part[group][0], (turn & 1) ^ 1, gave_up, P.err)) return false;
  if (rank < kShares - 1) {
    if (!warp_wait(&H.part[group][rank + 1], turn & 1, gave_up, P.err)) return false;
#pragma unroll
    for (int j = 0; j < kSums; ++j) total[j / (4 * N)][(j / 4) % N][j % 4] += place[32 * j];
  }
  if (rank > 0) {
#pragma unroll
    for (int j = 0; j < kSums; ++j) place[32 * j] = total[j / (4 * N)][(j / 4) % N][j % 4];
  }
  warp_release(&H.part[group][rank]);
  if (rank > 0) return true;
  if constexpr (HALF) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) total[t][0][j] += __shfl_xor_sync(~0u, total[t][0][j], 2);     // lo to hi
  }
#pragma unroll
  for (int t = 0; t < (C::kUp ? 1 : 2); ++t)
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = it.block * C::kOutRows + base + 16 * t + r0 + 8 * (j >> 1);
        const int col = 8 * n + 2 * c + (j & 1);
        if (row < P.rows && col < it.n) {
          float v = total[t][n][j];
          if constexpr (C::kUp) v = silu(v) * total[1][n][j];
          P.out[(int64_t)(it.first + col) * P.rows + row] = v;
        }
      }
  return true;
}

template <int MODE, int NT>
__global__ void __launch_bounds__(kThreads, 1) moe_few_kernel(const __grid_constant__ Params P) {
  using C = Cfg<MODE, NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  Head& H = *reinterpret_cast<Head*>(smem);
  float* part = reinterpret_cast<float*>(smem + kHeadBytes);
  uint8_t* ring = smem + C::kFixed;
  volatile int* gave_up = &H.gave_up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nb = P.nb;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&H.full[i], 32 * kCopiers + 1);
      tc::mbar_init(&H.empty[i], kGroups);
    }
    for (int i = 0; i < kGroups * kShares; ++i) tc::mbar_init(&H.part[0][i], 1);
    for (int i = 0; i < kQueue; ++i) {
      tc::mbar_init(&H.item_full[i], 1);
      tc::mbar_init(&H.item_empty[i], kConsumers + kCopiers);
    }
    H.issued = 0;
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const uint32_t items = make_tiles<kThreads, C::kPairs>(H.tiles, P.offsets, P.experts, (int)P.pairs, P.err) * P.blocks;

  if (warp == kLead) {
    // ------------------------------------------------- items, and the operands
    uint32_t n = 0, i = blockIdx.x;
    int ticket = 0;
    bool stop = false;
    for (uint32_t turn = 0; !stop; ++turn) {
      const Item it = i < items ? find_item(H.tiles, i, P.blocks, C::kPairs) : Item{0, 0, 0, 0};
      const uint32_t q = turn % kQueue;
      if (!warp_wait(&H.item_empty[q], ((turn / kQueue) & 1) ^ 1, gave_up, P.err)) break;
      if (lane == 0) {
        H.item[q] = make_int4(it.expert, it.block, it.first, it.n);
        tc::mbar_arrive(&H.item_full[q]);
      }
      __syncwarp();
      if (turn == 0) asm volatile("griddepcontrol.wait;" ::: "memory");       // the operands; the weights need no wait
      if (it.n == 0) break;
      const int eighths = (it.n + 7) / 8;
      const uint32_t bytes = it.n <= 4 ? kHalfX : kTileX;
      const uint8_t* x = P.x + (int64_t)(H.tiles.eighth[it.expert] + (it.first - H.tiles.off[it.expert]) / 8) * nb * kTileX;
      if (lane == 0) ticket = (int)gridDim.x + atomicAdd(P.counter, 1);
      for (int sb = 0; sb < nb; ++sb, ++n) {
        const uint32_t slot = n % C::kSlots;
        if (!warp_wait(&H.empty[slot], ((n / C::kSlots) & 1) ^ 1, gave_up, P.err)) {
          stop = true;
          break;
        }
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(&H.full[slot], eighths * bytes);
          uint8_t* at = ring + slot * C::kSlot + C::kWeights + C::kScales;
          for (int k = 0; k < eighths; ++k)
            tc::bulk_g2s(at + k * kTileX, x + ((int64_t)k * nb + sb) * kTileX, bytes, &H.full[slot]);
          if constexpr (!C::kOwnSlots)
            asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(tc::smem_u32(&H.issued)), "r"(n + 1) : "memory");
        }
        __syncwarp();
      }
      i = __shfl_sync(~0u, ticket, 0);
    }
    // its copies land before the CTA ends
    if (lane == 0)
      for (uint32_t j = n < C::kSlots ? 0 : n - C::kSlots; j < n; ++j)
        if (!tc::mbar_wait_sleep(&H.full[j % C::kSlots], (j / C::kSlots) & 1)) break;
  } else if (warp >= kConsumers) {
    // -------------------------------------------------------------- weights
    const int tid = threadIdx.x - 32 * kConsumers;
    constexpr int kPieces = C::kSb / 16, kMatrixRows = C::kOutRows, kEach = kMatrixRows * kPieces / (32 * kCopiers),
                  kRest = kMatrixRows * kPieces % (32 * kCopiers);
    int row[kEach + (kRest > 0)], col[kEach + (kRest > 0)];
#pragma unroll
    for (int j = 0; j < kEach + (kRest > 0); ++j) {
      const int q = tid + 32 * kCopiers * j;
      row[j] = q / kPieces, col[j] = 16 * (q % kPieces);
    }
    const int last = P.experts * P.rows - 1;
    uint32_t n = 0;
    bool stop = false;
    for (uint32_t turn = 0; !stop; ++turn) {
      const uint32_t q = turn % kQueue;
      if (!warp_wait(&H.item_full[q], (turn / kQueue) & 1, gave_up, P.err)) break;
      const int4 it = H.item[q];
      warp_release(&H.item_empty[q]);
      if (it.w == 0) break;
      const int w0 = it.x * P.rows + it.y * C::kOutRows;
      uint32_t off[kEach + (kRest > 0)];                         // (128 rows are less than 2^32 bytes)
#pragma unroll
      for (int j = 0; j < kEach + (kRest > 0); ++j) off[j] = (uint32_t)(min(row[j], last - w0) * P.pitch) + col[j];
      const uint8_t *from = P.w + w0 * P.pitch, *from2 = C::kUp ? P.up + w0 * P.pitch : nullptr;
      for (int sb = 0; sb < nb; ++sb, ++n) {
        const uint32_t slot = n % C::kSlots;
        if (!warp_wait(&H.empty[slot], ((n / C::kSlots) & 1) ^ 1, gave_up, P.err)) {
          stop = true;
          break;
        }
        const uint32_t at = tc::smem_u32(ring + slot * C::kSlot) + 16 * tid;
#pragma unroll
        for (int j = 0; j < kEach + (kRest > 0); ++j) {
          if (j == kEach && tid >= kRest) break;
          copy16(at + 16 * 32 * kCopiers * j, from + off[j]);
          if constexpr (C::kUp) copy16(at + C::kWeights / 2 + 16 * 32 * kCopiers * j, from2 + off[j]);
        }
        if constexpr (C::kQ6)
          for (int r = tid; r < kTileRows; r += 32 * kCopiers)
            copy4(tc::smem_u32(ring + slot * C::kSlot + C::kWeights) + 4 * r,
                  P.w + (int64_t)min(w0 + r, last) * P.pitch + (int64_t)kQ6GpuBytes * nb + 2 * (sb & ~1));
        copies_arrive(&H.full[slot]);
        from += C::kSb;
        if constexpr (C::kUp) from2 += C::kSb;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------------------- products
    uint32_t first = 0;
    for (uint32_t turn = 0;; ++turn, first += nb) {
      const uint32_t q = turn % kQueue;
      if (!warp_wait(&H.item_full[q], (turn / kQueue) & 1, gave_up, P.err)) break;
      const int4 v = H.item[q];
      warp_release(&H.item_empty[q]);
      const Item it{v.x, v.y, v.z, v.w};
      bool ok;
      if (it.n == 0) break;
      if (it.n <= 4) ok = consume<C, 1, true>(P, H, part, ring, it, first, turn);
      else if (NT == 1 || it.n <= 8) ok = consume<C, 1, false>(P, H, part, ring, it, first, turn);
      else ok = consume<C, NT, false>(P, H, part, ring, it, first, turn);
      if (!ok) break;
    }
  }
}

inline int64_t most_eighths(int64_t pairs, int experts) { return std::min(pairs, pairs / 8 + experts); }

template <int MODE, int NT>
cudaError_t launch(const MoeProduct& p, void* work, float* out, cudaStream_t s) {
  using C = Cfg<MODE, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(moe_few_kernel<MODE, NT>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  Params P{};
  const int64_t nb = p.cols / kQK, pairs = p.plan.tokens * p.plan.top_k;
  const int64_t pitch = C::kQ6 ? q6k_gpu_row_bytes(nb) : nb * kBlockBytes;
  P.counter = static_cast<int32_t*>(work), P.x = static_cast<uint8_t*>(work) + 128;
  P.w = p.w, P.up = p.up, P.pitch = pitch;
  P.offsets = p.plan.offsets, P.out = out, P.err = p.err, P.pairs = pairs;
  P.blocks = (uint32_t)((p.rows + C::kOutRows - 1) / C::kOutRows);
  P.rows = (int)p.rows, P.nb = (int)nb, P.experts = p.plan.experts;
  const int64_t most = std::min(pairs, pairs / C::kPairs + P.experts) * P.blocks;
  if (most * nb >= (int64_t(1) << 31)) return cudaErrorNotSupported;           // 32-bit counters of items and stages
  SplitParams S{p.x, p.plan.order, p.plan.offsets, static_cast<uint8_t*>(work) + 128, P.counter, p.err, pairs, p.cols,
                (int)nb, p.plan.experts, C::kUp ? p.plan.top_k : 0};
  const int64_t eighths = most_eighths(pairs, p.plan.experts);
  // few groups of pairs: a warp for each superblock
  const unsigned parts = (unsigned)std::max<int64_t>(1, std::min<int64_t>((nb + kSplitWarps - 1) / kSplitWarps, 4 * 152 / eighths));
  moe_few_split_kernel<C::kQ6><<<dim3((unsigned)eighths, parts), 32 * kSplitWarps, 0, s>>>(S, C::kPairs);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  int dev = 0;
  cudaGetDevice(&dev);
  return launch_after(moe_few_kernel<MODE, NT>, dim3((unsigned)std::min<int64_t>(most, device_info(dev).sm_count)), kThreads,
                      C::kSmem, s, P);
}

// Tiles of 16 pairs as soon as some expert can have more than 8.
template <int MODE>
cudaError_t launch_mode(const MoeProduct& p, void* work, float* out, cudaStream_t s) {
  return p.plan.tokens <= 8 ? launch<MODE, 1>(p, work, out, s) : launch<MODE, 2>(p, work, out, s);
}

}  // namespace few
}  // namespace q4k
