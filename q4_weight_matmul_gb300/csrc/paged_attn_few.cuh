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
// Products run on mma.sync m16n8k16 (fp32 accumulate): S = Q K^T with the 16
// rows of a warp as M, then O += P V.  The weights P keep fp32's precision
// through 16-bit operands: P = hi + lo (binary16, 22 bits) or hi + mid + lo
// (bfloat16, 24 bits), scaled by 2^14 so that weights down to 2^-14 of the
// largest keep all their bits in binary16's normal range.  With at most 8
// rows to a tile (PACK) hi and lo share one product: hi in rows 0-7, lo in
// rows 8-15, their results added.  A slot's products start from zero and
// are added to O in fp32 registers: the tensor core's own running sum
// truncates, and over thousands of steps that would show in the 1e-6s.
#pragma once

#include "mma_sync.cuh"
#include "paged_attn_common.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>

namespace q4k {
namespace attn {

constexpr int kUnit = 32;               // keys of a slot
constexpr int kConsumers = 8;           // consumer warps
constexpr int kFewThreads = 32 * (kConsumers + 4);   // the producer's warpgroup: one warp works
constexpr float kLift = 14.0f;          // weights are held times 2^14

template <int D>
struct FewLayout {
  static constexpr int kTile = kUnit * D * 2;              // keys (or values) of a slot
  static constexpr int kSlot = 2 * kTile;
};

// WR: warps that share a slot, 16 rows each (1, 2, 4); PACK: at most 8 rows, WR 1.
template <int D, int WR, bool PACK>
struct FewConfig {
  static constexpr int kRows = PACK ? 8 : 16 * WR;
  static constexpr int kGroups = kConsumers / WR;          // slots consumed at once
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

struct FewParams {
  AttnParams a;
  int page_shift, box;           // box: keys of one copy, min(page size, 32)
  int min_units;
};

template <int D, bool BF16, int WR, bool PACK>
__global__ void __launch_bounds__(kFewThreads, 1)
paged_attn_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ FewParams F) {
  using L = FewLayout<D>;
  using C = FewConfig<D, WR, PACK>;
  constexpr int ROWS = C::kRows;
  constexpr int PARTS = BF16 ? 3 : 2;               // 16-bit parts of a weight
  extern __shared__ uint8_t raw[];
  const AttnParams& P = F.a;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = tc::smem_u32(base);
  float* sum = reinterpret_cast<float*>(base + C::kSlots * L::kSlot);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + C::kSlots * L::kSlot + C::kSum);
  uint64_t* empty = full + C::kSlots;
  int64_t* scratch = reinterpret_cast<int64_t*>(empty + C::kSlots);   // 16 words
  float* stat_m = reinterpret_cast<float*>(scratch + 16);             // [group][row]
  float* stat_l = stat_m + kConsumers * 16;
  volatile int* gave_up = reinterpret_cast<volatile int*>(stat_l + kConsumers * 16);
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
  const Range R = share_out<ROWS, kUnit, kFewThreads>(P, group, F.min_units, scratch);
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

  // 384 threads x 168 registers at launch = 256 x 208 + 128 x 88
  if (warp >= kConsumers) {
    // ---------------------------------------------------------- producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp > kConsumers) return;
    const int pages_slot = F.box < kUnit ? kUnit / F.box : 1;
    const int none = P.num_pages > 0 ? (int)P.num_pages : 1;    // a page past the end reads as zeros
    do {
      const int64_t key0 = (w.lo / kUnit) * kUnit;
      const int32_t* table = P.page_table + (int64_t)w.req * P.max_pages;
      int64_t cached = -1;                           // page index that lane 0's entry is for
      int entry = none;
      for (int u = w.u0; u < w.u1; ++u, ++issued) {
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
        if (lane == 0 && !*gave_up) tc::mbar_arrive_expect_tx(&full[slot], L::kSlot);
        for (int i = 0; i < pages_slot; ++i) {
          const int page = __shfl_sync(0xffffffffu, entry, (int)(p0 + i - cached));
          const int cell = (int)(key & (P.page_size - 1));
          if (lane == 0 && !*gave_up) {
            const uint32_t dst = ring + slot * L::kSlot + i * F.box * D * 2;
            const int from = F.box < kUnit ? 0 : cell >> 3;
            load_cells(dst, &kmap, from, page, P.kv_heads, w.head, &full[slot]);
            load_cells(dst + L::kTile, &vmap, from, page, P.kv_heads, w.head, &full[slot]);
          }
        }
      }
    } while (w.next(P, R, group));
    // after a wait gave up, the copies still in flight end before the block does
    if (lane == 0 && *gave_up) {
      for (uint32_t j = issued < C::kSlots ? 0 : issued - C::kSlots; j < issued; ++j)
        if (!tc::mbar_wait_sleep(&full[j % C::kSlots], (j / C::kSlots) & 1)) break;
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  constexpr int kThreads = 32 * kConsumers;
  auto sync = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  const uint32_t grp = warp / WR;
  const int wr = warp % WR;
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const float to_log2 = P.scale * 1.4426950408889634f;
  float* pieces = reinterpret_cast<float*>(static_cast<uint8_t*>(P.workspace) + kTicketBytes);

  do {
    const int rows_all = w.s.n * group, row0 = w.tile * ROWS;
    const int rows = min(ROWS, rows_all - row0);
    const int my0 = wr * 16;                          // first of this warp's rows within the tile
    const bool active = my0 < rows;
    // Q fragments: rows g and g + 8 (PACK: row g only)
    uint32_t q[D / 16][4];
    const int ra = my0 + g, rb = my0 + g + 8;
    const bool has_a = ra < rows, has_b = !PACK && rb < rows;
    {
      const uint16_t* qa = static_cast<const uint16_t*>(P.q);
      const uint16_t* pa = qa + (has_a ? out_row(P, w.s, w.head, group, row0 + ra) * D : 0);
      const uint16_t* pb = qa + (has_b ? out_row(P, w.s, w.head, group, row0 + rb) * D : 0);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][0] = has_a ? *reinterpret_cast<const uint32_t*>(pa + 16 * k + c2) : 0u;
        q[k][1] = has_b ? *reinterpret_cast<const uint32_t*>(pb + 16 * k + c2) : 0u;
        q[k][2] = has_a ? *reinterpret_cast<const uint32_t*>(pa + 16 * k + 8 + c2) : 0u;
        q[k][3] = has_b ? *reinterpret_cast<const uint32_t*>(pb + 16 * k + 8 + c2) : 0u;
      }
    }
    // the keys each row sees, as positions within the item: [lo_x, hi_x)
    const int64_t key0 = (w.lo / kUnit) * kUnit;
    auto bounds = [&](int row, bool has, int& lo, int& hi) {
      const int64_t pos = w.s.kv - w.s.n + (row0 + row) / group;
      const int64_t from = P.window ? pos - P.window + 1 : 0;
      hi = has && pos + 1 > key0 ? (int)(pos + 1 - key0) : 0;
      lo = from > key0 ? (int)(from - key0) : 0;
    };
    int lo_a, hi_a, lo_b, hi_b;
    bounds(ra, has_a, lo_a, hi_a);
    bounds(rb, has_b, lo_b, hi_b);
    // positions that every row of the warp sees need no mask
    int lo_all = 0, hi_all = 0;
    if (active) {
      int x;
      bounds(my0, true, x, hi_all);
      bounds(min(my0 + 15, rows - 1), true, lo_all, x);
    }
    const int lo_item = (int)(w.lo - key0), hi_item = (int)(w.hi - key0);

    constexpr int NT = D / 8;
    float o[NT][PACK ? 2 : 4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < (PACK ? 2 : 4); ++e) o[i][e] = 0.f;
    float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;

    for (int u = w.u0; u < w.u1; ++u, ++issued) {
      if (issued % C::kGroups != grp) continue;
      const int slot = issued % C::kSlots;
      wait(&full[slot], (issued / C::kSlots) & 1);
      if (active) {
        const uint32_t ks = ring + slot * L::kSlot, vs = ks + L::kTile;
        // S: 4 tiles of 8 keys
        float s[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
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
        // scores in units of log 2, masked where a row does not see the key
        const int at = u * kUnit;
        const bool inside = at >= lo_all && at + kUnit <= hi_all;
        float top_a = m_a, top_b = m_b;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[t][e] *= to_log2;
            if (!inside) {
              const int p = at + 8 * t + c2 + (e & 1);
              const bool seen = e < 2 ? (p >= lo_a && p < hi_a) : (p >= lo_b && p < hi_b);
              if (!seen) s[t][e] = -INFINITY;
            }
          }
          top_a = fmaxf(top_a, fmaxf(s[t][0], s[t][1]));
          top_b = fmaxf(top_b, fmaxf(s[t][2], s[t][3]));
        }
        top_a = fmaxf(top_a, __shfl_xor_sync(0xffffffffu, top_a, 1));
        top_a = fmaxf(top_a, __shfl_xor_sync(0xffffffffu, top_a, 2));
        if (!PACK) {
          top_b = fmaxf(top_b, __shfl_xor_sync(0xffffffffu, top_b, 1));
          top_b = fmaxf(top_b, __shfl_xor_sync(0xffffffffu, top_b, 2));
        }
        // a row that has seen nothing yet keeps weights of zero
        const float sub_a = top_a == -INFINITY ? 0.f : top_a - kLift, sub_b = top_b == -INFINITY ? 0.f : top_b - kLift;
        const float f_a = m_a == -INFINITY ? 0.f : exp2f(m_a - top_a);
        const float f_b = m_b == -INFINITY ? 0.f : exp2f(m_b - top_b);
        m_a = top_a, m_b = top_b;
        // weights, their sums, and their 16-bit parts as A fragments of two k steps of 16 keys
        uint32_t p[PARTS][2][4];
        float add_a = 0.f, add_b = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float e0 = exp2f(s[t][0] - sub_a), e1 = exp2f(s[t][1] - sub_a);
          float e2 = 0.f, e3 = 0.f;
          add_a += e0 + e1;
          if (!PACK) {
            e2 = exp2f(s[t][2] - sub_b), e3 = exp2f(s[t][3] - sub_b);
            add_b += e2 + e3;
          }
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            const uint32_t h = pack2<BF16>(e0, e1);
            const float2 f = unpack2<BF16>(h);
            e0 -= f.x, e1 -= f.y;
            p[i][t >> 1][(t & 1) * 2] = h;
            if (!PACK) {
              const uint32_t h2 = pack2<BF16>(e2, e3);
              const float2 f2 = unpack2<BF16>(h2);
              e2 -= f2.x, e3 -= f2.y;
              p[i][t >> 1][(t & 1) * 2 + 1] = h2;
            }
          }
        }
        l_a = l_a * f_a + add_a;
        l_b = l_b * f_b + add_b;
        // values that no row of the tile sees may be anything: they become zeros
        uint32_t keep[2][2];
        const bool edge = at < lo_item || at + kUnit > hi_item;
        if (edge) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = at + 16 * k + 8 * e + c2;
              keep[k][e] = (j >= lo_item && j < hi_item ? 0xffffu : 0u) |
                           (j + 1 >= lo_item && j + 1 < hi_item ? 0xffff0000u : 0u);
            }
        }
        // O += P V, 32 values (four tiles of 8) at a time
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
          float acc[4][4];
          uint32_t b[2][2][4];   // [16 values][16 keys]: (keys 0-7, values 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              ldsm4t(b[j][k], vs + Cells<D>::at(16 * k + (lane & 15), n >> 1, 4 * (n & 1) + 2 * j + (lane >> 4)));
          if (edge) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) b[j][k][e] &= keep[k][e & 1];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            constexpr int STEP = PACK ? 2 : 1;
#pragma unroll
            for (int i = 0; i < PARTS; i += STEP) {
              uint32_t a[4];
              if constexpr (PACK) {
                const int lo = i + 1 < PARTS ? i + 1 : i;
                a[0] = p[i][k][0], a[2] = p[i][k][2];
                a[1] = i + 1 < PARTS ? p[lo][k][0] : 0u, a[3] = i + 1 < PARTS ? p[lo][k][2] : 0u;
              } else {
                a[0] = p[i][k][0], a[1] = p[i][k][1], a[2] = p[i][k][2], a[3] = p[i][k][3];
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) mma16816<BF16>(acc[j], a, b[j >> 1][k][2 * (j & 1)], b[j >> 1][k][2 * (j & 1) + 1]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float(&x)[PACK ? 2 : 4] = o[4 * n + i];
            if constexpr (PACK) {
              x[0] = fmaf(x[0], f_a, acc[i][0] + acc[i][2]);
              x[1] = fmaf(x[1], f_a, acc[i][1] + acc[i][3]);
            } else {
              x[0] = fmaf(x[0], f_a, acc[i][0]), x[1] = fmaf(x[1], f_a, acc[i][1]);
              x[2] = fmaf(x[2], f_b, acc[i][2]), x[3] = fmaf(x[3], f_b, acc[i][3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[slot]);
    }

    // ---- the groups' statistics and outputs meet: sum[group][row][D]
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
    if ((lane & 3) == 0) {
      stat_m[grp * ROWS + my0 + g] = m_a;
      stat_l[grp * ROWS + my0 + g] = l_a;
      if (!PACK) {
        stat_m[grp * ROWS + my0 + g + 8] = m_b;
        stat_l[grp * ROWS + my0 + g + 8] = l_b;
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float* at = sum + (size_t)(grp * ROWS + my0 + g) * D + 8 * i + c2;
      *reinterpret_cast<float2*>(at) = make_float2(o[i][0], o[i][1]);
      if constexpr (!PACK) *reinterpret_cast<float2*>(at + 8 * D) = make_float2(o[i][2], o[i][3]);
    }
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
        combine<ROWS, D, BF16, kConsumers>(P, pieces, c0, c1, w.s, w.head, group, row0, rows, sum, tid, sync);
    }
  } while (w.next(P, R, group));
}

// Launch the variant; defined in one translation unit per head size and type.
template <int D, bool BF16>
cudaError_t launch_few(const CUtensorMap& kmap, const CUtensorMap& vmap, const FewParams& f, int variant, int ctas,
                       cudaStream_t s);

template <int D, bool BF16, int WR, bool PACK>
cudaError_t launch_few_variant(const CUtensorMap& kmap, const CUtensorMap& vmap, const FewParams& f, int ctas,
                               cudaStream_t s) {
  auto kernel = paged_attn_few_kernel<D, BF16, WR, PACK>;
  constexpr int smem = FewConfig<D, WR, PACK>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kFewThreads, smem, s>>>(kmap, vmap, f);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace q4k
