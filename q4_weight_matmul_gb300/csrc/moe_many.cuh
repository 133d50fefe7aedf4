// Products of the experts' matrices with many rows each (prompts), on the
// tensor cores (tcgen05): 128 or 256 weight rows times up to 112 pairs of one
// expert, fp32 sums of exact 16-bit products as in moe_few.cuh.
//
// Measured: 4096 tokens, 4 of 32 experts of 2560 x 1536: gate and up 408 us
// (2 x 258 GFLOP with both parts: 1.26 PFLOP/s; 434 us after a quarter of a
// second, when the power limit has taken the clock from 2070 to some 1850 MHz),
// down 299 us; 513 tokens, 6 of 60 experts of 2560 x 1280: 131 us, down Q6_K
// 110 us.  Bound: the making of a step's A and the issue of its products, see
// below.  The launches alone (they overlap by some us): gate and up of 4096
// tokens layout 4, split 46 (it moves 168 MB), products 373; down layout 4,
// split 36, products 213, putting together 45.
//
// Four launches.  (1) One CTA lays the pairs out in tiles: an expert's n pairs
// become ceil(n / 112) tiles (or ceil(n / 32): see kMoeSmallTiles) of equal
// size, a multiple of 16.  (2) Each pair's activations, times a power of two
// that puts the row's largest in [2^14, 2^15), become two binary16 parts,
// stored tile by tile as the products read them (64 k of hi, then of lo, in the
// 128-byte-swizzled layout), with the sums of every 32 of them (hi and lo,
// times 2^-5).  (3) The products.  (4) For down: the weighted rows of a token
// are added up (moe_product.cu).
//
// The weights are the products' A and lie in tensor memory: a converter thread
// owns a weight row, which is a lane there, and writes sc q - c as binary16, exact.
// So shared memory feeds the tensor core with B alone (with both operands
// there, 128 columns an instruction would take all of its bandwidth).  The min
// term dmin m sums(x) is part of the same sum: with r = dmin / d the sum over a
// superblock is d (sum (sc q - c) x - sum (r m - c) sums(x)), r m - c as two
// binary16 parts (22 bits) beside the sums' parts, so a superblock takes one
// FMA per row and column in the epilogue.  c, some 8 sc, is there because a sum
// loses bits by its size: without it the quants' and the mins' parts, which
// nearly cancel, are each several times as large as their difference (relative
// error of h 1.95e-6 in place of 1.26e-6, for 2 to 5 % of the time).  Where
// |r| > 16, all of it is taken 2^-e times, e = floor(log2 |r|) - 3, so that r m
// fits binary16; sc q 2^-e stays exact up to e = 20, and beyond (dmin > 2^24 d)
// d counts as 0.
// Q6_K: sc (q - 32) needs up to 13 bits: hi = binary16 of it and lo = the rest
// (-1, 0, 1), two tiles that meet the hi and lo, and the hi parts of x.
//
// A CTA's warps: 0 copies activations, 2 draws items (a tile of pairs times a
// block of rows; large tiles first) and copies weights, 1 and 3 issue the
// products, one for each tile of rows (a burst of eight waits and starts for
// some 400 cycles, which the other's products cover), then two groups of four
// convert (with one, 700 cycles a tile held the products up, 547 us for 4096
// tokens; four for tiles of 32 pairs), and eight run the epilogue (totals in
// registers).  With 128 pairs an expert the tensor pipe works in half of the
// cycles and instructions issue in 53 %; with 16 (tiles of 32) 21 % and 65 %.  Every wait is bounded, and its loop short and inline: with ten
// instructions more in each, the roles' loops did not fit the instruction
// caches together (459 us).
#pragma once

#include "mma_sync.cuh"
#include "mmq_cvt.cuh"
#include "moe.cuh"
#include "tmap.h"

#include <algorithm>

namespace q4k {
namespace many {

enum Mode { kGateUp, kDownQ4, kDownQ6 };

constexpr int kRows = 128;                    // weight rows of a product
constexpr int kStages = 4;                    // of 64 k of the activations, hi and lo
constexpr int kUnits = 3, kQueue = 4;

constexpr uint32_t kProduct = (1u << 4) | ((uint32_t)(kRows >> 4) << 24);      // f16 operands, f32 sums, 128 rows

struct Tile {                 // pairs first .. first + n - 1 of an expert; their padded rows from `row` on
  int expert, first, n, row;
};
struct Control {
  int tiles, counter, pad[30];
};

// COLS: the most pairs of a tile.  A step of the products is 64 k (or twice
// that) of both A tiles (Q6_K: of both parts), the last of a superblock with
// its min term.  Tensor memory: three sums in turn, the A tiles of two steps in
// turn, those of the min terms.
//  - 112: a step's products take longer than making its A.  (With 128 columns a
//    sum the min terms' only place is among the steps', where they hold the
//    next step up: 482 us for 4096 tokens.)
//  - 32: the other way round, so there are twice the converters, steps of 128 k
//    (a step costs the warps that issue products some 800 cycles), and the
//    activations' hi and lo parts are columns of one product beside each other.
template <int MODE, int COLS>
struct Cfg {
  static constexpr bool kUp = MODE == kGateUp, kQ6 = MODE == kDownQ6;
  static constexpr bool kBeside = COLS == 32;
  static constexpr int kCols = COLS, kUnitCols = kBeside ? 2 * COLS : COLS;
  static constexpr int kHalves = kBeside ? 2 : 1, kPerBlock = 4 / kHalves;           // 64 k of a step, steps of a superblock
  static constexpr int kMins = kBeside ? 2 : 1;              // places of min terms
  static constexpr uint32_t kAColumn = kUnits * kUnitCols, kMinColumn = kAColumn + 128 * kHalves;
  static constexpr int kConverters = kBeside ? 16 : 8, kEpilogue = kBeside ? 4 : 8;  // warps
  static constexpr int kThreads = 32 * (4 + kConverters + kEpilogue);
  static constexpr int kStageBytes = 2 * COLS * 128 * kHalves, kSumBytes = COLS * 128;         // (the sums of four superblocks)
  static constexpr int kSb = kQ6 ? kQ6GpuBytes : kBlockBytes;
  static constexpr int kRaw = kBeside ? (kQ6 ? 5 : 8) : (kQ6 ? 3 : 4);               // weight tiles (128 rows of a superblock) in flight
  static constexpr int kIssuers = kQ6 ? 1 : 2;               // warps that issue products
  static constexpr int kTilesM = kQ6 ? 1 : 2;                // of 128 rows each
  static constexpr int kOutRows = MODE == kDownQ4 ? 2 * kRows : kRows;
  // The tensor core drops what is below its sum's last place at every product,
  // towards zero, so a superblock's sum comes out too small: by half a place a
  // product in the mean.  A sum of n products that grows steadily has lost some
  // 0.3 n 2^-24 of itself at its end: with n = 34 (tiles of 32 pairs: 18) 10
  // (5.5), and so it was measured for normal activations, rows of any length
  // and both formats.  Its scale puts that mean back: the relative error of h
  // 1.26e-6 -> 5.2e-7 (6.2e-7 -> 3.6e-7), of down 2.5e-7 and 7.3e-7 -> 1.4e-7
  // and 4e-7.  It is a mean: sums that lose less come out too large, by 6e-7 of
  // themselves at most, where all but one term is zero (rows with one value in
  // 32: down 2.7e-7 -> 4.0e-7; positive values: Q4_K 0.5e-7 -> 5.9e-7, Q6_K
  // 1.1e-6 -> 4.9e-7).
  static constexpr float kBack = 1.0f + (kBeside ? 6 : 10) * 5.9604644775390625e-8f;
  // registers of the three kinds of warps; at launch 768 x 80 and 640 x 96
  static constexpr int kFewRegs = 32, kConvRegs = kBeside ? 72 : 64, kEpiRegs = 160;
  static_assert(32 * (4 * kFewRegs + kConverters * kConvRegs + kEpilogue * kEpiRegs) == kThreads * (kBeside ? 80 : 96));
  static_assert(kMinColumn + 32 * kMins <= 512);
};

struct Params {
  CUtensorMap w, up;          // rows of the experts' superblocks
  const Control* control;
  const Tile* tiles;
  const float* inv;
  const uint8_t *x, *sums, *scales;    // scales: the rows' d (Q6_K), rows of `pitch` bytes
  float* out;
  int* counter;
  int* err;
  int64_t pitch;
  int rows, nb, blocks;
};

template <int MODE, int COLS>
struct __align__(1024) Smem {
  using C = Cfg<MODE, COLS>;
  uint8_t x[kStages][C::kStageBytes];
  uint8_t sums[2][C::kSumBytes];
  uint8_t raw[C::kRaw][kRows * C::kSb];
  float scale[2][2][kRows];
  uint64_t xfull[kStages], sfull[2], sempty[2], rfull[C::kRaw], rempty[C::kRaw], afull[2], mfull[C::kMins], done[4],
      tfull[kUnits], tempty[kUnits], dfull[2], dempty[2], qfull[kQueue], qempty[kQueue], drain[2];
  Tile item[kQueue];
  int block[kQueue];
  uint32_t tmem;
  int gave_up;
};
static_assert(sizeof(Smem<kGateUp, 112>) + 1024 <= 232448 && sizeof(Smem<kDownQ6, 112>) + 1024 <= 232448);
static_assert(sizeof(Smem<kGateUp, 32>) + 1024 <= 232448 && sizeof(Smem<kDownQ6, 32>) + 1024 <= 232448);

// One lane of a converged warp; what it issues takes its operands from uniform
// registers.
__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// D[tmem] (+)= A[tmem] B[smem]^T
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t what, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(what), "r"(add) : "memory");
}
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// ---------------------------------------------------------------- the tiles
// One CTA, a thread per expert.  Tiles of equal size lie in any order: each
// result is the same wherever its tile comes.
struct LayoutParams {
  const int32_t* offsets;
  Control* control;
  Tile* tiles;
  int* err;
  int pairs, experts;
};

template <int kCols>
__global__ void __launch_bounds__(kMoeMaxExperts) moe_many_layout_kernel(const LayoutParams P) {
  __shared__ int warps[16], count[kCols / 16 + 1], start[kCols / 16 + 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int e = threadIdx.x, E = P.experts;
  if (e <= kCols / 16) count[e] = 0;
  const int raw0 = e <= E ? P.offsets[e] : INT32_MAX, raw1 = e < E ? P.offsets[e + 1] : INT32_MAX;
  int all;
  const int before = scan_block<kMoeMaxExperts, true>(min(raw0, P.pairs), warps, all);
  const int first = max(max(before, 0), min(raw0, P.pairs)), last = max(first, min(raw1, P.pairs));
  if (e < E && (first != raw0 || last != raw1 || (e == 0 && raw0 != 0))) atomicOr(P.err, kErrIndex);   // (no pairs before the first expert's)
  const int n = e < E ? last - first : 0, tiles = (n + kCols - 1) / kCols;
  const int each = tiles ? ((n + tiles - 1) / tiles + 15) / 16 * 16 : 16;
  const int used = (n + each - 1) / each;                     // (rounding up can save one)
  int row = scan_block<kMoeMaxExperts, false>(used ? (used - 1) * each + (n - (used - 1) * each + 15) / 16 * 16 : 0, warps, all);
  for (int k = 0; k < used; ++k) atomicAdd(&count[(min(each, n - k * each) + 15) / 16], 1);
  __syncthreads();
  if (e == 0) {
    int run = 0;
    for (int c = kCols / 16; c > 0; --c) start[c] = run, run += count[c];
    P.control->tiles = run;
    P.control->counter = 0;
  }
  __syncthreads();
  for (int k = 0; k < used; ++k) {
    const int m = min(each, n - k * each);
    P.tiles[atomicAdd(&start[(m + 15) / 16], 1)] = Tile{e, first + k * each, m, row + k * each};
  }
}

// ----------------------------------------------------------- activations
struct SplitParams {
  const float* x;
  const int32_t* order;
  const Control* control;
  const Tile* tiles;
  uint8_t *out, *sums;
  float* inv;
  int* err;
  int64_t pairs, cols;
  int nb, top_k;              // top_k 0: x has a row for every pair
};

// A CTA for 8 pairs of a tile, a warp each; a lane has 8 neighbouring values
// of a superblock.  PERMUTE: the values of 4 in the order 0, 2, 1, 3, in which
// Q4_K quants leave their bytes without a transpose.
template <bool PERMUTE>
__global__ void __launch_bounds__(256) moe_many_split_kernel(const SplitParams P) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x >= P.control->tiles) return;
  const Tile T = P.tiles[blockIdx.x];
  const int i = 8 * blockIdx.y + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= T.n) return;
  const int padded = (T.n + 15) / 16 * 16;
  int64_t r = T.first + i;
  if (P.top_k) {
    const int p = P.order[r];
    r = p >= 0 && p < P.pairs ? p / P.top_k : -1;
    if (r < 0 && lane == 0) atomicOr(P.err, kErrIndex);
  }
  const float4* from = reinterpret_cast<const float4*>(P.x + max(r, (int64_t)0) * P.cols);
  float top = 0.0f;
  if (r >= 0) {
#pragma unroll 4
    for (int k = lane; k < P.cols / 4; k += 32) {
      const float4 v = from[k];
      top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  const int E = (int)((__float_as_uint(top) >> 23) & 0xFFu), es = top == 0.0f ? 127 : min(253, max(1, 268 - E));
  const float s = __uint_as_float((uint32_t)es << 23);
  if (lane == 0) P.inv[T.row + i] = __uint_as_float((uint32_t)(254 - es) << 23);
  uint8_t* out = P.out + (int64_t)T.row * P.cols * 4 + i * 128 + (((lane & 7) ^ (i & 7)) << 4);
  __half* sums = reinterpret_cast<__half*>(P.sums + (int64_t)T.row * ((P.nb + 3) / 4) * 128 + i * 128);
  for (int sb = 0; sb < P.nb; ++sb) {
    float4 a = make_float4(0, 0, 0, 0), b = a;
    if (r >= 0) a = from[64 * sb + 2 * lane], b = from[64 * sb + 2 * lane + 1];
    const float v[8] = {a.x * s, (PERMUTE ? a.z : a.y) * s, (PERMUTE ? a.y : a.z) * s, a.w * s,
                        b.x * s, (PERMUTE ? b.z : b.y) * s, (PERMUTE ? b.y : b.z) * s, b.w * s};
    uint32_t hi[4], lo[4];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      hi[k] = pack2<false>(v[2 * k], v[2 * k + 1]);
      const float2 h = unpack2<false>(hi[k]);
      lo[k] = pack2<false>(v[2 * k] - h.x, v[2 * k + 1] - h.y);
      const float2 l = unpack2<false>(lo[k]);
      sum += (h.x + h.y) + (l.x + l.y);
    }
    uint8_t* at = out + (int64_t)(4 * sb + (lane >> 3)) * 2 * padded * 128;
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + padded * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if constexpr (PERMUTE) {                                   // Q4_K: the sub-blocks' sums
      sum += __shfl_xor_sync(~0u, sum, 1);
      sum += __shfl_xor_sync(~0u, sum, 2);
      if ((lane & 3) == 0) {
        const float x = sum * 0.03125f;
        const __half h = __float2half_rn(x);
        // 16-byte chunk 2 (sb % 4) has the hi parts, the next one the lo parts
        const int c = 2 * (sb & 3), k = lane >> 2;
        __half* to = sums + (int64_t)(sb >> 2) * padded * 64;
        to[((c ^ (i & 7)) << 3) + k] = h;
        to[(((c + 1) ^ (i & 7)) << 3) + k] = __float2half_rn(x - __half2float(h));
      }
    }
  }
}

// ------------------------------------------------------------- converters
// 32 weights of a Q4_K row (the low or high nibbles of 32 quant bytes) times
// their scale s, less a middle c (see middles), pairs (0, 2), (1, 3) of every four.
template <bool HIGH>
__device__ __forceinline__ void convert_q4(const uint4& q0, const uint4& q1, uint32_t s, uint32_t (&a)[16]) {
  // (1024 + q) s - (1024 s + c), (1024 + 16 q) s / 16 - (64 s + c): one exact FMA each
  const uint32_t m = HIGH ? cvt::mul_h2(s, 0x2C002C00u) : s, b = cvt::mul_h2(s, HIGH ? 0xD480D480u : 0xE408E408u);
  const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = w[i] >> 8;
    asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, %4, 0x64006400, 0xEA;\n\tfma.rn.f16x2 %0, t, %2, %3;\n\t}"
        : "=r"(a[2 * i]) : "r"(w[i]), "r"(m), "r"(b), "n"(HIGH ? 0x00F000F0 : 0x000F000F));
    asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, %4, 0x64006400, 0xEA;\n\tfma.rn.f16x2 %0, t, %2, %3;\n\t}"
        : "=r"(a[2 * i + 1]) : "r"(u), "r"(m), "r"(b), "n"(HIGH ? 0x00F000F0 : 0x000F000F));
  }
}

// What a Q4_K row's header says about a superblock.
struct Header {
  uint32_t sc[2], m[2];       // 6-bit scales and mins
  uint32_t down;              // 2^-e twice, or 0 where d counts as 0
  float scale, r;             // what a sum is to be multiplied with; r m 2^-e as part of it: r times -2^5
};
__device__ __forceinline__ Header header_of(const uint4& h) {
  Header H;
  cvt::header_sc_m(h, H.sc[0], H.sc[1], H.m[0], H.m[1]);
  const float2 d = unpack2<false>(h.x);                        // d, dmin
  H.r = __fdividef(-32.0f * d.y, d.x);                         // (within 2^-22)
  H.scale = d.x;
  H.down = 0x3C003C00u;
  // (a d or dmin that is NaN gives a ratio that is: the first stays in the scale, the second in r, and so in the sum)
  if (fabsf(H.r) > 512.0f && d.y != 0.0f) {                    // |r| > 16, or d = 0
    const int e = (int)(__float_as_uint(H.r) >> 23 & 0xFF) - 127 - 8;
    if (d.x == 0.0f || e > 20) {
      H.down = 0, H.r = -512.0f, H.scale = d.y * 0.0625f;
    } else {
      H.r = __uint_as_float(__float_as_uint(H.r) - ((uint32_t)e << 23));
      H.scale = __uint_as_float(__float_as_uint(d.x) + ((uint32_t)e << 23));
      const __half2 t = __float2half2_rn(__uint_as_float((uint32_t)(127 - e) << 23));
      H.down = *reinterpret_cast<const uint32_t*>(&t);
    }
  } else if (d.y == 0.0f) {
    H.r = 0.0f;                                                // (d may be 0 too)
  }
  return H;
}

// -c of sub-blocks 2 i and 2 i + 1: 8 s, as binary16 holds 1032 s (and 72 s,
// which is exact).
__device__ __forceinline__ float2 middles(const Header& H, int i) {
  const uint32_t bytes = __byte_perm(H.sc[i >> 1], 0x64646464u, i & 1 ? 0x4342 : 0x4140), bias = 0xE400E400u;
  const __half2 s = __hmul2(__hadd2(*reinterpret_cast<const __half2*>(&bytes), *reinterpret_cast<const __half2*>(&bias)),
                            *reinterpret_cast<const __half2*>(&H.down));
  const __half2 b = __hmul2(s, __floats2half2_rn(-1032.0f, -72.0f));
  return __half22float2(__hfma2(s, __floats2half2_rn(1024.0f, 64.0f), b));
}

// The two binary16 parts of r m - c for the eight mins: [hi | hi], [lo | lo].
__device__ __forceinline__ void convert_min(const Header& H, uint32_t (&a)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = H.m[i >> 1] >> (16 * (i & 1));
    const float2 c = middles(H, i);
    const float v0 = H.r * (float)(w & 0xFFu) - 32.0f * c.x, v1 = H.r * (float)(w >> 8 & 0xFFu) - 32.0f * c.y;
    a[i] = a[4 + i] = pack2<false>(v0, v1);
    const float2 h = unpack2<false>(a[i]);
    a[8 + i] = a[12 + i] = pack2<false>(v0 - h.x, v1 - h.y);
  }
}

// Sub-block S (32 weights) of a Q6_K row's chunk (32 bytes of low nibbles, 16
// of bit pairs; `scales` of its groups) as the parts of sc (q - 32), in order.
__device__ __forceinline__ void convert_q6(const uint4& l0, const uint4& l1, const uint4& h, uint32_t scales, int S,
                                           uint32_t (&hi)[16], uint32_t (&lo)[16]) {
  const uint32_t lw[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w}, hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int g = 0; g < 2; ++g) {                                // the sub-block's groups of 16
    const float sf = (float)(int8_t)(scales >> (16 * S + 8 * g));
    const __half2 sc = __float2half2_rn(sf), bias = __float2half2_rn(-1056.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bytes of q with the top bit inverted, then two at a time under the exponent of 1024
      const uint32_t v = ((lw[4 * g + i] >> (4 * S)) & 0x0F0F0F0Fu) | (((hw[i] >> (4 * S + 2 * g)) & 0x03030303u) << 4);
      const uint32_t p0 = __byte_perm(v, 0, 0x4140) ^ 0x64206420u, p1 = __byte_perm(v, 0, 0x4342) ^ 0x64206420u;
      const __half2 q0 = __hadd2(*reinterpret_cast<const __half2*>(&p0), bias),
                    q1 = __hadd2(*reinterpret_cast<const __half2*>(&p1), bias);
      const __half2 h0 = __hmul2(q0, sc), h1 = __hmul2(q1, sc);
      const __half2 r0 = __hfma2(q0, sc, __hneg2(h0)), r1 = __hfma2(q1, sc, __hneg2(h1));
      hi[8 * g + 2 * i] = *reinterpret_cast<const uint32_t*>(&h0), hi[8 * g + 2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h1);
      lo[8 * g + 2 * i] = *reinterpret_cast<const uint32_t*>(&r0), lo[8 * g + 2 * i + 1] = *reinterpret_cast<const uint32_t*>(&r1);
    }
  }
}

// ------------------------------------------------------------------ products
template <int MODE, int COLS>
__global__ void __launch_bounds__(Cfg<MODE, COLS>::kThreads, 1) moe_many_kernel(const __grid_constant__ Params P) {
  using C = Cfg<MODE, COLS>;
  constexpr int kConverters = C::kConverters, kEpilogue = C::kEpilogue;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<MODE, COLS>& S = *reinterpret_cast<Smem<MODE, COLS>*>(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
  volatile int* gave_up = &S.gave_up;
  int* err = P.err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nb = P.nb;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) tc::mbar_init(&S.xfull[i], 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(&S.done[i], C::kIssuers);
    for (int i = 0; i < C::kRaw; ++i) tc::mbar_init(&S.rfull[i], 1), tc::mbar_init(&S.rempty[i], C::kQ6 ? kConverters : kConverters / 2);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&S.sfull[i], 1), tc::mbar_init(&S.sempty[i], C::kIssuers);
      tc::mbar_init(&S.dfull[i], C::kQ6 ? 4 : 8), tc::mbar_init(&S.dempty[i], kEpilogue);
    }
    for (int i = 0; i < 2; ++i) tc::mbar_init(&S.afull[i], kConverters);
    for (int i = 0; i < C::kMins; ++i) tc::mbar_init(&S.mfull[i], 8);
    for (int i = 0; i < kUnits; ++i) tc::mbar_init(&S.tfull[i], 1), tc::mbar_init(&S.tempty[i], kEpilogue);
    for (int i = 0; i < kQueue; ++i) tc::mbar_init(&S.qfull[i], 1), tc::mbar_init(&S.qempty[i], 1 + C::kIssuers + kConverters + kEpilogue);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&S.drain[i], 1);
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    tc::tmem_alloc(&S.tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // Whoever has all 512 columns has them from 0 on; the address as a constant
  // keeps the products' operands in uniform registers.
  constexpr uint32_t tmem = 0;
  if (threadIdx.x == 0 && S.tmem != tmem) {
    *gave_up = 1;
    atomicOr(err, 1);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The next item of a warp; false: there is none, or a wait gave up.
  uint32_t turn = 0;
  Tile T;
  int block = 0;
  auto next_item = [&]() -> bool {
    const uint32_t q = turn % kQueue;
    if (!warp_wait(&S.qfull[q], (turn / kQueue) & 1, gave_up, err)) return false;
    T = S.item[q], block = S.block[q];
    warp_release(&S.qempty[q]);
    ++turn;
    return T.n > 0;
  };

  // Until step `k` is done with its operands.  (Four barriers: a step four later waits for this one's operands, or for
  // the place of a min term that this one's superblock had.)
  auto step_done = [&](uint32_t k) { return warp_wait(&S.done[k % 4], (k / 4) & 1, gave_up, err); };

  if (warp < 4) {
    registers_down<C::kFewRegs>();
    if (warp == 0) {
      // ------------------------------------------------------ activations
      uint32_t j = 0, g = 0;                                   // stages, groups of sums issued
      bool stop = false;
      while (!stop && next_item()) {
        const uint32_t padded = (T.n + 15) / 16 * 16;
        const uint8_t* x = P.x + (int64_t)T.row * nb * 1024;
        const uint8_t* sums = P.sums + (int64_t)T.row * ((nb + 3) / 4) * 128;
        for (int c = 0; c < 4 * nb; c += C::kHalves, ++j) {
          if (!C::kQ6 && c % 16 == 0) {
            stop = !warp_wait(&S.sempty[g & 1], ((g >> 1) & 1) ^ 1, gave_up, err);
            if (stop) break;
            if (elect()) {
              tc::mbar_arrive_expect_tx(&S.sfull[g & 1], padded * 128);
              tc::bulk_g2s(S.sums[g & 1], sums + (int64_t)(c / 16) * padded * 128, padded * 128, &S.sfull[g & 1]);
            }
            __syncwarp();
            ++g;
          }
          const uint32_t slot = j % kStages;
          stop = j >= kStages && !step_done(j - kStages);
          if (stop) break;
          if (elect()) {
            const uint32_t bytes = C::kHalves * 2 * padded * 128;
            tc::mbar_arrive_expect_tx(&S.xfull[slot], bytes);
            tc::bulk_g2s(S.x[slot], x + (int64_t)c * 2 * padded * 128, bytes, &S.xfull[slot]);
          }
          __syncwarp();
        }
      }
      if (lane == 0) {                                         // its copies land before the CTA ends
        for (uint32_t i = j < kStages ? 0 : j - kStages; i < j; ++i)
          if (!tc::mbar_wait_sleep(&S.xfull[i % kStages], (i / kStages) & 1)) break;
        for (uint32_t i = g < 2 ? 0 : g - 2; i < g; ++i)
          if (!tc::mbar_wait_sleep(&S.sfull[i & 1], (i >> 1) & 1)) break;
      }
    } else if (warp == 2) {
      // ----------------------------------------------- items, and their weights
      const int items = P.control->tiles * P.blocks;
      int i = blockIdx.x;
      uint32_t n = 0;
      bool stop = false;
      for (uint32_t t = 0; !stop; ++t) {
        const uint32_t q = t % kQueue;
        const bool have = i < items;
        Tile tile{0, 0, 0, 0};
        int ticket = 0;
        if (have) {
          tile = P.tiles[i / P.blocks], block = i % P.blocks;
          if (lane == 0) ticket = (int)gridDim.x + atomicAdd(P.counter, 1);
        }
        if (!warp_wait(&S.qempty[q], ((t / kQueue) & 1) ^ 1, gave_up, err)) break;
        if (lane == 0) {
          S.item[q] = tile, S.block[q] = block;
          tc::mbar_arrive(&S.qfull[q]);
        }
        __syncwarp();
        if (!have) break;
        const int w0 = tile.expert * P.rows + block * C::kOutRows;
        for (int r = 0; r < C::kTilesM * nb; ++r, ++n) {
          const int sb = r / C::kTilesM, mt = r % C::kTilesM;
          const uint32_t slot = n % C::kRaw;
          stop = !warp_wait(&S.rempty[slot], ((n / C::kRaw) & 1) ^ 1, gave_up, err);
          if (stop) break;
          if (elect()) {
            tc::mbar_arrive_expect_tx(&S.rfull[slot], kRows * C::kSb);
            tc::tma_load_3d(S.raw[slot], C::kUp && mt ? &P.up : &P.w, 0, C::kUp ? w0 : w0 + kRows * mt, sb, &S.rfull[slot]);
          }
          __syncwarp();
        }
        i = __shfl_sync(~0u, ticket, 0);
      }
      if (lane == 0)
        for (uint32_t r = n < C::kRaw ? 0 : n - C::kRaw; r < n; ++r)
          if (!tc::mbar_wait_sleep(&S.rfull[r % C::kRaw], (r / C::kRaw) & 1)) break;
    } else if (warp == 1 || !C::kQ6) {
      // --------------------------------------------------------- products
      const uint32_t mt = C::kQ6 || warp == 1 ? 0 : 1;          // of this tile of rows (Q6_K: both parts)
      uint32_t k = 0, g = 0, u = mt, b = 0;                    // steps, groups of sums of x, sums, superblocks
      bool stop = false;
      while (!stop && next_item()) {
        // (from a vote, so that it is uniform to the compiler)
        const uint32_t padded = 16 * __popc(__ballot_sync(~0u, 16 * lane < T.n)), narrow = kProduct | (padded >> 3) << 17,
                       what = C::kBeside ? kProduct | (padded >> 2) << 17 : narrow;
        for (int sb = 0; sb < nb && !stop; ++sb, ++b, u += C::kTilesM) {
          const uint32_t d = tmem + C::kUnitCols * (u % kUnits);
          const bool last = (sb & 3) == 3 || sb == nb - 1;
          stop = !warp_wait(&S.tempty[u % kUnits], ((u / kUnits) & 1) ^ 1, gave_up, err);
#pragma unroll 1
          for (int c = 0; c < C::kPerBlock; ++c, ++k) {
            const uint32_t x = tc::smem_u32(S.x[k % kStages]), a = tmem + C::kAColumn + 64 * C::kHalves * (k & 1) + 32 * mt;
            const uint32_t sums = tc::smem_u32(S.sums[g & 1]) + 32 * (sb & 3);
            stop = stop || !warp_wait(&S.xfull[k % kStages], (k / kStages) & 1, &S.afull[k & 1], (k >> 1) & 1, gave_up, err);
            if (!C::kQ6 && c == C::kPerBlock - 1)
              stop = stop || !warp_wait(&S.sfull[g & 1], (g >> 1) & 1, &S.mfull[b % C::kMins], (b / C::kMins) & 1, gave_up, err);
            if (stop) break;
            tc::fence_after_sync();
            if (elect()) {
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h) {
                const uint64_t hi = tc::desc_sw128(x + h * 2 * padded * 128), lo = hi + padded * 8;   // (of 16 bytes)
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {                  // 16 k: 32 bytes of a row
                  mma_ts(d, a + 64 * h + 8 * i, hi + 2 * i, what, c | h | i ? 1 : 0);
                  if constexpr (!C::kBeside) mma_ts(d, a + 64 * h + 8 * i, lo + 2 * i, what, 1);
                  if constexpr (C::kQ6) mma_ts(d, a + 64 * h + 32 + 8 * i, hi + 2 * i, narrow, 1);
                }
              }
              if (!C::kQ6 && c == C::kPerBlock - 1) {
                const uint32_t m = tmem + C::kMinColumn + 32 * (b % C::kMins) + 16 * mt;
                mma_ts(d, m, tc::desc_sw128(sums), narrow, 1);
                mma_ts(d, m + 8, tc::desc_sw128(sums), narrow, 1);
                if (last) tc::mma_commit(&S.sempty[g & 1]);
              }
              tc::mma_commit(&S.done[k % 4]);
              if (c == C::kPerBlock - 1) tc::mma_commit(&S.tfull[u % kUnits]);
            }
            __syncwarp();
          }
          g += !C::kQ6 && last;
        }
      }
      if (elect()) tc::mma_commit(&S.drain[mt]);               // every product is done before tensor memory goes
      __syncwarp();
      if (!tc::mbar_wait_sleep(&S.drain[mt], 0)) atomicOr(err, 1);
    }
  } else if (warp < 4 + kConverters) {
    // --------------------------------------------------------------- converters
    registers_down<C::kConvRegs>();
    // group: of the tiles of rows (Q6_K: sub-blocks of 64 k); turn_of: of a step's 64 k, where it has them twice
    const int quarter = warp & 3, group = (warp - 4) >> 2 & 1, row = 32 * quarter + lane;
    constexpr int kTurns = C::kHalves;
    const int turn_of = kTurns == 1 ? 0 : (warp - 4) >> 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16) + C::kAColumn;
    uint32_t n = 0, b = 0;                                     // raw tiles, superblocks
    // step k's A tiles may be written; they have been
    auto begin_step = [&](uint32_t k) {
      const bool ok = k < 2 || step_done(k - 2);
      tc::fence_after_sync();
      return ok;
    };
    auto end_step = [&](uint64_t* bar) {
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    auto scale_of = [&](int mt, float v) -> bool {             // of a superblock's sum, for the epilogue
      if (!warp_wait(&S.dempty[b & 1], ((b >> 1) & 1) ^ 1, gave_up, err)) return false;
      S.scale[b & 1][mt][row] = v;
      warp_release(&S.dfull[b & 1]);
      return true;
    };
    bool stop = false;
    while (!stop && next_item()) {
      if constexpr (C::kQ6) {
        // a group makes the operands of one sub-block of every 64 k: half of the hi tile and of the lo tile
        const __half* scales = reinterpret_cast<const __half*>(
            P.scales + (T.expert * (int64_t)P.rows + min(block * C::kOutRows + row, P.rows - 1)) * P.pitch);
        for (int sb = 0; sb < nb && !stop; ++sb, ++n, ++b) {
          const uint32_t slot = n % C::kRaw;
          const float d = __half2float(scales[sb]);
          stop = !warp_wait(&S.rfull[slot], (n / C::kRaw) & 1, gave_up, err) || (group + turn_of == 0 && !scale_of(0, d * C::kBack));
          if (stop) break;
          const uint8_t* w = S.raw[slot] + row * C::kSb;
#pragma unroll 1
          for (int c = turn_of; c < 4; c += kTurns) {
            const uint4* p = reinterpret_cast<const uint4*>(w + 16 + 48 * c);
            const uint4 l0 = p[0], l1 = p[1], h = p[2];
            const uint32_t sc = *reinterpret_cast<const uint32_t*>(w + 4 * c), k = C::kPerBlock * b + c / C::kHalves,
                           at = lanes + 64 * (C::kHalves * (k & 1) + turn_of) + 16 * group;
            if (c >= 4 - kTurns) warp_release(&S.rempty[slot]);
            uint32_t hi[16], lo[16];
            convert_q6(l0, l1, h, sc, group, hi, lo);
            stop = !begin_step(k);
            if (stop) break;
            tc::tmem_st16(at, hi);
            tc::tmem_st16(at + 32, lo);
            end_step(&S.afull[k & 1]);
          }
        }
      } else {
        // a group has one of the two tiles of rows
        for (int sb = 0; sb < nb && !stop; ++sb, n += 2, ++b) {
          const uint32_t slot = (n + group) % C::kRaw;
          stop = !warp_wait(&S.rfull[slot], ((n + group) / C::kRaw) & 1, gave_up, err);
          if (stop) break;
          const uint8_t* w = S.raw[slot] + row * C::kSb;
          const Header H = header_of(*reinterpret_cast<const uint4*>(w));
#pragma unroll 1
          for (int c = turn_of; c < 4; c += kTurns) {
            const uint4* p = reinterpret_cast<const uint4*>(w + 16 + 32 * c);
            const uint4 q0 = p[0], q1 = p[1];
            if (c >= 4 - kTurns) warp_release(&S.rempty[slot]);
            const uint32_t s = c < 2 ? H.sc[0] : H.sc[1], k = C::kPerBlock * b + c / C::kHalves,
                           at = lanes + 64 * (C::kHalves * (k & 1) + turn_of) + 32 * group;
            uint32_t v[16], w2[16];
            convert_q4<false>(q0, q1, cvt::mul_h2(cvt::byte_h2(s, 2 * (c & 1)), H.down), v);
            convert_q4<true>(q0, q1, cvt::mul_h2(cvt::byte_h2(s, 2 * (c & 1) + 1), H.down), w2);
            stop = !begin_step(k);
            if (stop) break;
            tc::tmem_st16(at, v);
            tc::tmem_st16(at + 16, w2);
            end_step(&S.afull[k & 1]);
            if (turn_of == 0 && c == (kTurns == 1 ? 1 : 0)) {
              // the superblock whose min term had this place before is done (one turn: as begin_step has seen)
              convert_min(H, v);
              if constexpr (kTurns > 1) {
                stop = b >= C::kMins && !step_done(C::kPerBlock * (b - C::kMins + 1) - 1);
                if (stop) break;
                tc::fence_after_sync();
              }
              tc::tmem_st16(lanes + (C::kMinColumn - C::kAColumn) + 32 * (b % C::kMins) + 16 * group, v);
              stop = !scale_of(group, H.scale * C::kBack);
              if (stop) break;
              end_step(&S.mfull[b % C::kMins]);
            }
          }
        }
      }
    }
  } else {
    // ----------------------------------------------------------------- epilogue
    registers_up<C::kEpiRegs>();
    const int quarter = warp & 3, row = 32 * quarter + lane, half = (warp - 4 - kConverters) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    uint32_t u = 0, b = 0;                                     // sums, superblocks
    bool stop = false;
    while (!stop && next_item()) {
      // 16 columns at a time, half of them each
      const int sixteens = (T.n + 15) / 16, first = half ? (sixteens + 1) / 2 : 0,
                mine = kEpilogue == 4 ? sixteens : half ? sixteens / 2 : (sixteens + 1) / 2;
      // the powers of two to take off: column 32 i + lane of the warp's in inv[i]
      float inv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) inv[i] = 32 * i + lane < 16 * mine ? P.inv[T.row + 16 * first + 32 * i + lane] : 0.0f;
      constexpr int kMine = kEpilogue == 4 ? C::kCols / 16 : 4;
      uint64_t total[C::kTilesM][kMine][8];
#pragma unroll
      for (int mt = 0; mt < C::kTilesM; ++mt)
#pragma unroll
        for (int k = 0; k < kMine; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) total[mt][k][i] = 0;
      for (int sb = 0; sb < nb && !stop; ++sb, ++b) {
        stop = !warp_wait(&S.dfull[b & 1], (b >> 1) & 1, gave_up, err);
        if (stop) break;
#pragma unroll
        for (int mt = 0; mt < C::kTilesM; ++mt, ++u) {
          const uint32_t t = u % kUnits;
          stop = !warp_wait(&S.tfull[t], (u / kUnits) & 1, gave_up, err);
          if (stop) break;
          tc::fence_after_sync();
          const float d = S.scale[b & 1][mt][row];
          const uint64_t d2 = pair_of(d, d);
          const uint32_t at = lanes + C::kUnitCols * t + 16 * first;
#pragma unroll
          for (int k = 0; k < kMine; ++k) {
            if (k < mine) {
              uint32_t v[16], lo[16];
              tc::tmem_ld16(at + 16 * k, v);
              if constexpr (C::kBeside) tc::tmem_ld16(at + 16 * (sixteens + k), lo);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                total[mt][k][i] = fma2(d2, pair_of(v[2 * i], v[2 * i + 1]), total[mt][k][i]);
                if constexpr (C::kBeside) total[mt][k][i] = fma2(d2, pair_of(lo[2 * i], lo[2 * i + 1]), total[mt][k][i]);
              }
            }
          }
          tc::fence_before_sync();
          warp_release(&S.tempty[t]);
          if (mt == C::kTilesM - 1 && lane == 0) tc::mbar_arrive(&S.dempty[b & 1]);
        }
      }
      if (stop) break;
#pragma unroll
      for (int mt = 0; mt < (C::kUp ? 1 : C::kTilesM); ++mt) {
        const int r = block * C::kOutRows + kRows * mt + row;
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          if (k >= mine) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int col = 16 * (first + k) + 2 * i;
            const float i0 = __shfl_sync(~0u, inv[k >> 1], (16 * k + 2 * i) & 31),
                        i1 = __shfl_sync(~0u, inv[k >> 1], (16 * k + 2 * i + 1) & 31);
            float2 v = halves(total[mt][k][i]);
            v.x *= i0, v.y *= i1;
            if constexpr (C::kUp) {
              const float2 w = halves(total[1][k][i]);
              v.x = silu(v.x) * (w.x * i0), v.y = silu(v.y) * (w.y * i1);
            }
            if (r < P.rows) {
              float* out = P.out + (int64_t)(T.first + col) * P.rows + r;
              if (col < T.n) out[0] = v.x;
              if (col + 1 < T.n) out[P.rows] = v.y;
            }
          }
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(S.tmem, 512);
  }
}

// -------------------------------------------------------------------- launches
inline int64_t most_tiles(int64_t pairs, int experts, int cols) { return std::min(pairs, pairs / cols + experts); }
inline int64_t most_rows(int64_t pairs, int experts, int cols) { return (pairs + 15 * most_tiles(pairs, experts, cols) + 15) / 16 * 16; }

struct Places {               // in the workspace
  size_t tiles, inv, x, sums, end;
};
inline Places places(int64_t pairs, int experts, int64_t cols, int tile) {
  const auto up = [](size_t v) { return (v + 1023) / 1024 * 1024; };
  const size_t rows = (size_t)most_rows(pairs, experts, tile);
  Places p{};
  p.tiles = sizeof(Control);
  p.inv = up(p.tiles + sizeof(Tile) * (size_t)most_tiles(pairs, experts, tile));
  p.x = up(p.inv + sizeof(float) * rows);
  p.sums = p.x + rows * (size_t)cols * 4;
  p.end = p.sums + rows * (size_t)((cols / kQK + 3) / 4) * 128;
  return p;
}

template <int MODE, int COLS>
cudaError_t launch(const MoeProduct& p, void* work, float* out, cudaStream_t s) {
  using C = Cfg<MODE, COLS>;
  static std::atomic<uint64_t> done{0};
  constexpr int kSmem = (int)sizeof(Smem<MODE, COLS>) + 1024;
  cudaError_t e = allow_smem(moe_many_kernel<MODE, COLS>, kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t pairs = p.plan.tokens * p.plan.top_k, nb = p.cols / kQK, all = p.rows * p.plan.experts;
  const int64_t pitch = C::kQ6 ? q6k_gpu_row_bytes(nb) : nb * kBlockBytes, blocks = (p.rows + C::kOutRows - 1) / C::kOutRows;
  const int64_t tiles = most_tiles(pairs, p.plan.experts, COLS);
  if (tiles * blocks * nb * 16 >= (int64_t(1) << 31)) return cudaErrorNotSupported;        // 32-bit counters
  uint8_t* at = static_cast<uint8_t*>(work);
  const Places w = places(pairs, p.plan.experts, p.cols, COLS);
  Control* control = reinterpret_cast<Control*>(at);
  Tile* list = reinterpret_cast<Tile*>(at + w.tiles);
  float* inv = reinterpret_cast<float*>(at + w.inv);
  Params P{};
  const uint64_t dims[3] = {(uint64_t)C::kSb, (uint64_t)all, (uint64_t)nb}, strides[2] = {(uint64_t)pitch, (uint64_t)C::kSb};
  const uint32_t box[3] = {(uint32_t)C::kSb, kRows, 1};
  if (!encode_tmap_u8_3d(&P.w, p.w, dims, strides, box)) return cudaErrorInvalidValue;
  if (C::kUp && !encode_tmap_u8_3d(&P.up, p.up, dims, strides, box)) return cudaErrorInvalidValue;
  P.control = control, P.tiles = list, P.inv = inv, P.x = at + w.x, P.sums = at + w.sums;
  P.scales = p.w + nb * kQ6GpuBytes, P.out = out, P.counter = &control->counter, P.err = p.err, P.pitch = pitch;
  P.rows = (int)p.rows, P.nb = (int)nb, P.blocks = (int)blocks;
  const LayoutParams A{p.plan.offsets, control, list, p.err, (int)pairs, p.plan.experts};
  moe_many_layout_kernel<COLS><<<1, kMoeMaxExperts, 0, s>>>(A);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const SplitParams B{p.x, p.plan.order, control, list, at + w.x, at + w.sums, inv, p.err, pairs, p.cols, (int)nb,
                      C::kUp ? p.plan.top_k : 0};
  if ((e = launch_after(moe_many_split_kernel<!C::kQ6>, dim3((unsigned)tiles, COLS / 8), 256, 0, s, B)) != cudaSuccess) return e;
  int dev = 0;
  cudaGetDevice(&dev);
  return launch_after(moe_many_kernel<MODE, COLS>, dim3((unsigned)std::min<int64_t>(tiles * blocks, device_info(dev).sm_count)), C::kThreads,
                      kSmem, s, P);
}

}  // namespace many
}  // namespace q4k
