// Attention over the paged cache for few query rows per key head: decoding,
// draft verification, and any call that wants fp32 results.
//
// Every key and value is read once per row tile and meets at most a few dozen
// rows, so HBM bounds it: 4 D bytes a key against 4 D operations a key and
// row.  One CTA per SM takes its share of the keys (paged_attn_common.cuh).
// A producer warp streams slots of 32 keys and their values (tensor copies of
// whole pages or page parts, 128-byte swizzled) into a ring; eight consumer
// warps take the slots in turn, each with its own running maximum, sum and
// output of the softmax, and put them together once per item.  So no warp
// ever waits for another while keys stream.
//
// Products run on mma.sync m16n8k16 (fp32 accumulate).  The weights P keep
// fp32's precision through 16-bit operands: P = hi + lo (binary16, 22 bits)
// or hi + mid + lo (bfloat16, 24 bits), scaled by 2^14 so that weights down
// to 2^-14 of the largest keep all their bits in binary16's normal range.  A
// slot's products start from zero and are added to O in fp32 registers: the
// tensor core's own running sum truncates, and over thousands of steps that
// would show in the 1e-6s.
//
// Up to 8 rows (Rows8) are the N of the products, with 16 keys or 16 values
// as M: S^T = K Q^T, O^T += V^T P^T, half of the products that rows as M
// would take.  Up to 4 of them stand twice, in columns 0-3 and 4-7, and the
// one P V product has hi in the first and lo in the second.  More rows
// (Rows16) are the M: S = Q K^T, O += P V, 16 to a warp.
//
// Measured (8 key heads of 128, groups of 4, fp32 results): 64 requests of up
// to 8192 keys 200 us, 6.4 TB/s (96 % of the copy rate; 218 us while the
// producer read the shared give-up flag before every copy instead of once a
// slot); 131072 keys of one request 86 us; 1021 keys 8.9 us, of which the
// launch 2, the share of the work 1.5, the first copy 1, a slot 1, putting
// warps and pieces together 3.  The variants for 16, 32 and 64 rows spill some
// 300 bytes a thread (the share of the work and the walk over it, in 64-bit
// numbers; the producer's 40 registers), those for up to 8 none; what that
// costs has not been measured.
#pragma once

#include "mma_sync.cuh"
#include "paged_attn_common.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>

namespace q4k {
namespace attn {

constexpr int kUnit = 32;               // keys of a slot
constexpr float kLift = 14.0f;          // weights are held times 2^14

template <int D>
struct FewLayout {
  static constexpr int kTile = kUnit * D * 2;              // keys (or values) of a slot
  static constexpr int kSlot = 2 * kTile;
};

// KIND 0: up to 4 rows, 1: up to 8, else 16 rows in each of WR = KIND / 16
// warps that share a slot (16, 32, 64).
template <int D, int KIND>
struct FewConfig {
  static constexpr int kWR = KIND < 16 ? 1 : KIND / 16;
  static constexpr int kRows = KIND == 0 ? 4 : KIND == 1 ? 8 : KIND;
  // Consumer warps.  Up to 8 rows a slot is little work: four warps keep up, and leave room for three slots each
  // (eight with one each read 5.4 TB/s of 64 x 8192 keys where four read 5.6).
  static constexpr int kWarps = KIND < 16 ? 4 : 8;
  static constexpr int kThreads = 32 * (kWarps + 4);       // and the producer's warpgroup, of which one warp works
  static constexpr int kGroups = kWarps / kWR;             // slots consumed at once
  // bytes where the groups' outputs meet, and later the pieces' weights
  static constexpr int kOutputs = kGroups * kRows * D * 4, kWeights = kMaxCtas * kRows * 4;
  static constexpr int kSum = kOutputs > kWeights ? kOutputs : kWeights;
  static constexpr int kSmemMax = 227 * 1024;
  static constexpr int kFixed = 4096;                      // barriers, statistics, base alignment
  static constexpr int kRing = (kSmemMax - kSum - kFixed) / FewLayout<D>::kSlot;
  // a multiple of the groups: a slot is always the same warps', who so never wait for a phase of it
  // before the one before that has passed (a parity would not tell the two apart)
  static constexpr int kSlots = (kRing > 24 ? 24 : kRing) / kGroups * kGroups;
  static constexpr int kSmem = kSlots * FewLayout<D>::kSlot + kSum + kFixed;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The item as a warp sees it.
struct Item {
  const uint16_t* q;
  int64_t key0;                // position 0 of the item's keys
  int lo, hi;                  // positions that some row of the tile sees
  int row0, rows, group, head;
  Shape s;
  int window;
  float to_log2;

  __device__ __forceinline__ const uint16_t* q_row(const AttnParams& P, int row, int dim) const {
    return q + out_row(P, s, head, group, row0 + row) * dim;
  }
  // the positions lo .. hi-1 that row `row` of the tile sees
  __device__ __forceinline__ void bounds(int row, bool has, int& from, int& to) const {
    const int64_t pos = s.kv - s.n + (row0 + row) / group;
    const int64_t first = window ? pos - window + 1 : 0;
    to = has && pos + 1 > key0 ? (int)(pos + 1 - key0) : 0;
    from = first > key0 ? (int)(first - key0) : 0;
  }
};

// Which values of the 16 keys from position `at` on some row sees, as masks of
// a V operand's registers (pairs of keys 2 c, 2 c + 1, and 8 more).
__device__ __forceinline__ void keep_masks(uint32_t (&keep)[2], int at, int c, const Item& it) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int j = at + 8 * e + 2 * c;
    keep[e] = (j >= it.lo && j < it.hi ? 0xffffu : 0u) | (j + 1 >= it.lo && j + 1 < it.hi ? 0xffff0000u : 0u);
  }
}

// A new maximum for a row: what to subtract from its scores (a row that has
// seen nothing yet keeps weights of zero) and the factor of its sums.
__device__ __forceinline__ void raise(float& m, float top, float& sub, float& f) {
  sub = top == -INFINITY ? 0.f : top - kLift;
  f = m == -INFINITY ? 0.f : ex2(m - top);
  m = top;
}

// Up to 8 rows as the N of the products; lane (g, c) = (lane / 4, lane % 4)
// has the scores of keys g and g + 8 and rows 2 c, 2 c + 1, and of O^T values
// g and g + 8 of every 16.  TWICE: up to 4 rows, in columns 0-3 and again in
// 4-7.
template <int D, bool BF16, bool TWICE>
struct Rows8 {
  static constexpr int PARTS = BF16 ? 3 : 2, PRODUCTS = TWICE ? 1 + (PARTS > 2) : PARTS;
  uint32_t q[D / 16][2];
  float o[D / 16][4];
  float m[2], l[2];
  int lo[2], hi[2], lo_all, hi_all;

  __device__ __forceinline__ static int row(int column) { return TWICE ? column & 3 : column; }

  __device__ __forceinline__ bool begin(const AttnParams& P, const Item& it, int lane) {
    const int g = lane >> 2, c = lane & 3, r = row(g);
    const bool has = r < it.rows;
    const uint16_t* from = it.q_row(P, has ? r : 0, D) + 2 * c;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) q[k][e] = has ? *reinterpret_cast<const uint32_t*>(from + 16 * k + 8 * e) : 0u;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = -INFINITY, l[e] = 0.f;
      it.bounds(row(2 * c + e), row(2 * c + e) < it.rows, lo[e], hi[e]);
    }
    int x;
    it.bounds(0, true, x, hi_all);
    it.bounds(it.rows - 1, true, lo_all, x);
    return true;
  }

  // the slot of the keys from position `at` on; ks, vs: its keys and values
  __device__ __forceinline__ void slot(const Item& it, uint32_t ks, uint32_t vs, int at, int lane) {
    const int g = lane >> 2, c = lane & 3;
    // two sums each, of the even and the odd k steps, for shorter chains
    float s[2][2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][0][e] = s[t][1][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; k += 2) {
      uint32_t a[2][2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          ldsm4(a[i][t], ks + Cells<D>::at(16 * t + (lane & 15), (k + i) >> 2, 2 * ((k + i) & 3) + (lane >> 4)));
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) mma16816<BF16>(s[t][i], a[i][t], q[k + i][0], q[k + i][1]);
    }
    float top[2] = {m[0], m[1]};
    const bool inside = at >= lo_all && hi_all - at >= kUnit;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = (s[t][0][e] + s[t][1][e]) * it.to_log2;
        if (!inside) {
          const int p = at + 16 * t + g + 8 * (e >> 1);
          if (p < lo[e & 1] || p >= hi[e & 1]) v = -INFINITY;
        }
        s[t][0][e] = v;
        top[e & 1] = fmaxf(top[e & 1], v);
      }
    float sub[2], f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], x));
      raise(m[e], top[e], sub[e], f[e]);
      l[e] *= f[e];
    }
    // weights of (key, row pair), split and turned into operands of (row, key pair)
    uint32_t p[PRODUCTS][2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = ex2(s[t][0][2 * h] - sub[0]), y = ex2(s[t][0][2 * h + 1] - sub[1]);
        l[0] += x, l[1] += y;
        uint32_t part[PARTS + 1];
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
          part[i] = pack2<BF16>(x, y);
          const float2 r = unpack2<BF16>(part[i]);
          x -= r.x, y -= r.y;
        }
        part[PARTS] = 0u;
#pragma unroll
        for (int i = 0; i < PRODUCTS; ++i)
          p[i][t][h] = transpose8x8(!TWICE ? part[i] : c < 2 ? part[2 * i] : part[2 * i + 1]);
      }
    const bool edge = at < it.lo || it.hi - at < kUnit;
    uint32_t keep[2][2];
    if (edge) {
      keep_masks(keep[0], at, c, it);
      keep_masks(keep[1], at + 16, c, it);
    }
#pragma unroll
    for (int n = 0; n < D / 16; n += 4) {
      uint32_t a[4][2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          ldsm4t(a[i][t], vs + Cells<D>::at(16 * t + (lane & 7) + 8 * (lane >> 4), (n + i) >> 2,
                                            2 * ((n + i) & 3) + ((lane >> 3) & 1)));
          if (edge) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[i][t][e] &= keep[t][e >> 1];
          }
        }
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < PRODUCTS; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) mma16816<BF16>(acc[i], a[i][t], p[j][t][0], p[j][t][1]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n + i][e] = fmaf(o[n + i][e], f[e & 1], acc[i][e]);
    }
  }

  // this group's statistics and outputs [row], [row][D]
  __device__ __forceinline__ void end(float* stat_m, float* stat_l, float* sum, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
    if (TWICE) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += __shfl_xor_sync(0xffffffffu, o[i][e], 2);
      if (c >= 2) return;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (g == 0) stat_m[2 * c + e] = m[e], stat_l[2 * c + e] = l[e];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        sum[(2 * c + e) * D + 16 * i + g] = o[i][e];
        sum[(2 * c + e) * D + 16 * i + g + 8] = o[i][2 + e];
      }
    }
  }
};

// 16 rows, from row `my0` of the tile on, as the M of the products; lane
// (g, c) has rows g and g + 8, keys or values 2 c, 2 c + 1 of every 8.
template <int D, bool BF16>
struct Rows16 {
  static constexpr int PARTS = BF16 ? 3 : 2;
  uint32_t q[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];
  int lo[2], hi[2], lo_all, hi_all, my0;

  // false: the tile has no such rows
  __device__ __forceinline__ bool begin(const AttnParams& P, const Item& it, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = my0 + g + 8 * r;
      const bool has = row < it.rows;
      const uint16_t* from = it.q_row(P, has ? row : 0, D) + 2 * c;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][r] = has ? *reinterpret_cast<const uint32_t*>(from + 16 * k) : 0u;
        q[k][2 + r] = has ? *reinterpret_cast<const uint32_t*>(from + 16 * k + 8) : 0u;
      }
      m[r] = -INFINITY, l[r] = 0.f;
      it.bounds(row, has, lo[r], hi[r]);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    if (my0 >= it.rows) return false;
    int x;
    it.bounds(my0, true, x, hi_all);
    it.bounds(min(my0 + 15, it.rows - 1), true, lo_all, x);
    return true;
  }

  __device__ __forceinline__ void slot(const Item& it, uint32_t ks, uint32_t vs, int at, int lane) {
    const int c = lane & 3;
    float s[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {              // 32 values: chunks 4k .. 4k+3
      uint32_t b[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) ldsm4(b[t], ks + Cells<D>::at(8 * t + (lane & 7), k >> 1, 4 * (k & 1) + (lane >> 3)));
#pragma unroll
      for (int t = 0; t < 4; ++t) mma16816<BF16>(s[t], q[2 * k], b[t][0], b[t][1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) mma16816<BF16>(s[t], q[2 * k + 1], b[t][2], b[t][3]);
    }
    const bool inside = at >= lo_all && hi_all - at >= kUnit;
    float top[2] = {m[0], m[1]}, sub[2], f[2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[t][e] *= it.to_log2;
        if (!inside) {
          const int p = at + 8 * t + 2 * c + (e & 1);
          if (p < lo[e >> 1] || p >= hi[e >> 1]) s[t][e] = -INFINITY;
        }
        top[e >> 1] = fmaxf(top[e >> 1], s[t][e]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      raise(m[r], top[r], sub[r], f[r]);
      l[r] *= f[r];
    }
    // weights, their sums, and their 16-bit parts as A operands of two k steps of 16 keys
    uint32_t p[PARTS][2][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = ex2(s[t][2 * r] - sub[r]), y = ex2(s[t][2 * r + 1] - sub[r]);
        l[r] += x + y;
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
          const uint32_t h = pack2<BF16>(x, y);
          const float2 v = unpack2<BF16>(h);
          x -= v.x, y -= v.y;
          p[i][t >> 1][(t & 1) * 2 + r] = h;
        }
      }
    const bool edge = at < it.lo || it.hi - at < kUnit;
    uint32_t keep[2][2];
    if (edge) {
      keep_masks(keep[0], at, c, it);
      keep_masks(keep[1], at + 16, c, it);
    }
#pragma unroll
    for (int n = 0; n < D / 32; ++n) {              // 32 values: four tiles of 8
      uint32_t b[2][2][4];   // [16 values][16 keys]: (keys 0-7, values 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ldsm4t(b[j][k], vs + Cells<D>::at(16 * k + (lane & 15), n >> 1, 4 * (n & 1) + 2 * j + (lane >> 4)));
          if (edge) {
#pragma unroll
            for (int e = 0; e < 4; ++e) b[j][k][e] &= keep[k][e & 1];
          }
        }
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma16816<BF16>(acc[j], p[i][k], b[j >> 1][k][2 * (j & 1)], b[j >> 1][k][2 * (j & 1) + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * n + i][e] = fmaf(o[4 * n + i][e], f[e >> 1], acc[i][e]);
    }
  }

  __device__ __forceinline__ void end(float* stat_m, float* stat_l, float* sum, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = my0 + g + 8 * r;
      if (c == 0) stat_m[row] = m[r], stat_l[row] = l[r];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(sum + (size_t)row * D + 8 * i + 2 * c) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
    }
  }
};

template <int D, bool BF16, int KIND>
struct RowsOf {
  using type = Rows16<D, BF16>;
};
template <int D, bool BF16>
struct RowsOf<D, BF16, 0> {
  using type = Rows8<D, BF16, true>;
};
template <int D, bool BF16>
struct RowsOf<D, BF16, 1> {
  using type = Rows8<D, BF16, false>;
};

struct FewParams {
  AttnParams a;
  int page_shift, box;           // box: keys of one copy, min(page size, 32)
  int min_units;
};

template <int D, bool BF16, int KIND>
__global__ void __launch_bounds__((FewConfig<D, KIND>::kThreads), 1)
paged_attn_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ FewParams F) {
  using L = FewLayout<D>;
  using C = FewConfig<D, KIND>;
  constexpr int ROWS = C::kRows, WR = C::kWR;
  extern __shared__ uint8_t raw[];
  const AttnParams& P = F.a;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = tc::smem_u32(base);
  float* sum = reinterpret_cast<float*>(base + C::kSlots * L::kSlot);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + C::kSlots * L::kSlot + C::kSum);
  uint64_t* empty = full + C::kSlots;
  int64_t* scratch = reinterpret_cast<int64_t*>(empty + C::kSlots);   // 16 words
  float* stat_m = reinterpret_cast<float*>(scratch + 16);             // [group][row]
  float* stat_l = stat_m + 128;
  volatile int* gave_up = reinterpret_cast<volatile int*>(stat_l + 128);
  int* last = const_cast<int*>(gave_up) + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = P.heads / P.kv_heads;
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], WR);
    }
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const Range R = share_out<ROWS, kUnit, C::kThreads>(P, group, F.min_units, scratch);
  if ((int)blockIdx.x >= R.ctas) return;
  __syncthreads();                                   // the barriers are there
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!tc::mbar_wait(bar, parity, gave_up) && !*gave_up) {
      *gave_up = 1;
      atomicOr(P.err, 1);
    }
  };

  Walk<ROWS, kUnit> w;
  w.first(P, R, group);
  uint32_t issued = 0;                               // slots before this item, the same count in every warp

  // KIND >= 16: 384 threads x 168 registers at launch = 256 x 232 + 128 x 40
  if (warp >= C::kWarps) {
    // ---------------------------------------------------------- producer
    if constexpr (KIND >= 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp > C::kWarps) return;
    const int pages_slot = F.box < kUnit ? kUnit / F.box : 1;
    const int none = P.num_pages > 0 ? (int)P.num_pages : 1;    // a page past the end reads as zeros
    bool stop = false;                               // a wait of the block gave up: no more copies
    do {
      const int64_t key0 = (w.lo / kUnit) * kUnit;
      const int32_t* table = P.page_table + (int64_t)w.req * P.max_pages;
      int64_t cached = -1;                           // page index that lane 0's entry is for
      int entry = none;
      for (int u = w.u0; u < w.u1; ++u, ++issued) {  // `issued`: slots that got their copies
        const int slot = issued % C::kSlots;
        const int64_t key = key0 + (int64_t)u * kUnit;
        const int64_t p0 = key >> F.page_shift;
        if (cached < 0 || p0 + pages_slot > cached + 32) {
          cached = p0;
          const int64_t p = p0 + lane, from = p << F.page_shift;
          entry = none;
          if (from < w.hi && from + P.page_size > w.lo) {        // a page that some row of the tile needs
            entry = table[p];
            if (entry < 0 || entry >= P.num_pages) {
              atomicOr(P.err, kErrIndex);
              entry = none;
            }
          }
        }
        if (issued >= C::kSlots) wait(&empty[slot], (issued / C::kSlots - 1) & 1);
        if ((stop = given_up(gave_up))) break;
        if (lane == 0) tc::mbar_arrive_expect_tx(&full[slot], L::kSlot);
        for (int i = 0; i < pages_slot; ++i) {
          const int page = __shfl_sync(0xffffffffu, entry, (int)(p0 + i - cached));
          const int cell = (int)(key & (P.page_size - 1));
          if (lane == 0) {
            const uint32_t dst = ring + slot * L::kSlot + i * F.box * D * 2;
            const int from = F.box < kUnit ? 0 : cell >> 3;
            load_cells(dst, &kmap, from, page, P.kv_heads, w.head, &full[slot]);
            load_cells(dst + L::kTile, &vmap, from, page, P.kv_heads, w.head, &full[slot]);
          }
        }
      }
    } while (!stop && w.next(P, R, group));
    // copies end before the block does, whoever gives up and when: the last ones to each slot
    if (lane == 0) {
      for (uint32_t j = issued < C::kSlots ? 0 : issued - C::kSlots; j < issued; ++j)
        if (!tc::mbar_wait_sleep(&full[j % C::kSlots], (j / C::kSlots) & 1)) break;
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  if constexpr (KIND >= 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
  constexpr int kThreads = 32 * C::kWarps;
  auto sync = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  const uint32_t grp = warp / WR;
  float* pieces = reinterpret_cast<float*>(static_cast<uint8_t*>(P.workspace) + kPieceBytes);
  typename RowsOf<D, BF16, KIND>::type part;
  if constexpr (KIND >= 16) part.my0 = warp % WR * 16;

  do {
    const int row0 = w.tile * ROWS, rows = min(ROWS, w.s.n * group - row0);
    const int64_t key0 = (w.lo / kUnit) * kUnit;
    const Item it{static_cast<const uint16_t*>(P.q), key0, (int)(w.lo - key0), (int)(w.hi - key0), row0, rows, group,
                  w.head, w.s, P.window, P.scale * 1.4426950408889634f};
    const bool active = part.begin(P, it, lane);
    for (int u = w.u0; u < w.u1; ++u, ++issued) {
      if (issued % C::kGroups != grp) continue;
      const int slot = issued % C::kSlots;
      wait(&full[slot], (issued / C::kSlots) & 1);
      if (active) part.slot(it, ring + slot * L::kSlot, ring + slot * L::kSlot + L::kTile, u * kUnit, lane);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[slot]);
    }
    // the groups' statistics and outputs meet: sum[group][row][D]
    part.end(stat_m + grp * ROWS, stat_l + grp * ROWS, sum + (size_t)grp * ROWS * D, lane);
    sync();
    const bool whole = w.u0 == 0 && w.u1 == w.units;
    float* mine = pieces + ((size_t)blockIdx.x * 2 + (w.u0 == 0 ? 1 : 0)) * piece_floats<ROWS, D>();
    for (int e = tid; e < rows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < C::kGroups; ++i) m = fmaxf(m, stat_m[i * ROWS + r]);
      float l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < C::kGroups; ++i) {
        const float mi = stat_m[i * ROWS + r];
        if (mi == -INFINITY) continue;
        const float f = exp2f(mi - m);
        const float4 v = *reinterpret_cast<const float4*>(sum + (size_t)(i * ROWS + r) * D + d);
        l = fmaf(f, stat_l[i * ROWS + r], l);
        a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        store4<BF16>(P.out, P.out_f32, out_row(P, w.s, w.head, group, row0 + r) * D + d,
                     make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
      } else {
        __stcg(reinterpret_cast<float4*>(mine + r * D + d), a);
        if (d == 0) {
          __stcg(mine + ROWS * D + r, m);
          __stcg(mine + ROWS * D + ROWS + r, l);
        }
      }
    }
    if (whole) {
      sync();                                           // before the next item writes the shared sums
    } else {
      const int c0 = owner(w.at, R), c1 = owner(w.at + w.units - 1, R);
      if (arrive(static_cast<unsigned*>(P.workspace) + c0, c1 - c0 + 1, last, tid == 0, sync))
        combine<ROWS, D, BF16, C::kWarps>(P, pieces, c0, c1, w.s, w.head, group, row0, rows, sum, tid, sync);
    }
  } while (w.next(P, R, group));
}

// Launch the variant; defined in one translation unit per head size and type.
template <int D, bool BF16>
cudaError_t launch_few(const CUtensorMap& kmap, const CUtensorMap& vmap, const FewParams& f, int kind, int ctas,
                       cudaStream_t s);

template <int D, bool BF16, int KIND>
cudaError_t launch_few_variant(const CUtensorMap& kmap, const CUtensorMap& vmap, const FewParams& f, int ctas,
                               cudaStream_t s) {
  auto kernel = paged_attn_few_kernel<D, BF16, KIND>;
  constexpr int smem = FewConfig<D, KIND>::kSmem;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, FewConfig<D, KIND>::kThreads, smem, s>>>(kmap, vmap, f);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace q4k
