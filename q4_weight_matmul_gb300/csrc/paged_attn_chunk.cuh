// Attention over the paged cache for many query rows per key head: chunks of
// prompts, with 16-bit results.
//
// 4 D operations per row and key on the tensor cores against an exponential
// and a handful of fp32 operations, so the tensor pipe bounds it, closely
// followed by the softmax.  One CTA per SM takes its share of the (row tile,
// 64 keys) units (paged_attn_common.cuh).  A row tile is 256 rows in two
// halves of 128, each with its own four softmax warps, one thread per row.
//
//   warp 8   streams key and value tiles (64 x D, tensor copies of pages or
//            page parts, 128-byte swizzled) into a ring of ten
//   warps 9, 10     issue a half's S = Q K^T (both operands from shared
//            memory, S in tensor memory)
//   warps 12, 13    issue a half's O += P V (P from tensor memory, V read with
//            its keys as the K dimension, O in tensor memory)
//   warps 0-3, 4-7   load Q, turn S into P = exp2(S c - m) in place, rescale
//            O when a row's maximum grows, write the results
//
// Each half has two S tiles: while its softmax works on one, the products of
// the next are made in the other, so neither waits for the other's latency
// (tiles of 128 keys with one S per half spent half of the time in that
// chain: 4400 cycles per 128 keys against 2048 of tensor work).  64 keys is
// what tensor memory has room for: 2 (halves) x (2 x 64 + D) columns of 512.
// Each kind of product of each half has a warp of its own, whose waits hold
// up nothing else (one warp for both kinds of a half took 1830 cycles per 64
// keys, one polling for both halves 3800; the tensor work is 1280).
//
// P is rounded to the cache's type for the second product (16 bits: 2^-11 or
// 2^-8 of each weight, as the result itself is); its sum is taken in fp32
// before that.  m is a row's maximum as of its last rescale: O is rescaled
// only when the maximum has grown by more than 2^6 since, so almost never
// after a row's first tiles, and P, lifted by 2^8, stays below binary16's
// largest value and above its subnormals down to 2^-22 of the largest weight.
//
// The tensor core's running sum O truncates at every product, some 2^-23 of
// itself a time and always the same way (the mean of 2^28 keys' values came out
// 1.2 % low; 131072 keys cost as much as binary16's rounding).  So after 256
// units (1024 products: 2^-13) O is added to sums in the workspace, in fp32,
// and starts again from zero.
//
// Measured (8 key heads of 128, groups of 4): chunks of 2048 and 1705 tokens
// over 16384 and 16086 keys, pages of 16: 667 us at the full clock, 1410
// TFLOP/s (74 % of the bf16 rate); back to back 711-735 us, as the GPU's power
// cap takes the clock from 2070 to some 1830 MHz after a tenth of a second.
// 512 tokens over 4096 keys 49 us.
//
// What bounds it: 667 us are 1850 cycles per 64 keys of 256 rows.  The products
// take 1024 of them at the tensor pipe's full rate (its counter says 58 %
// active, the issue slots' 41 %) and 1280 as far as S = Q K^T with 64 keys to
// an instruction is fed by shared memory at two thirds of that; the softmax
// runs beside them (two weights to a packed operation and three values to a
// maximum: 717 -> 701 us).  Where the other 570 cycles go is not known: waits
// between the roles, or the kernel's spills (384 bytes a thread, of the share
// of the work and the walk over it).
#pragma once

#include "paged_attn_common.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>

namespace q4k {
namespace attn {

constexpr int kChunkRows = 256;
constexpr int kChunkKeys = 64;
constexpr int kChunkThreads = 512;
constexpr float kChunkLift = 8.0f, kChunkGrow = 6.0f;
constexpr int kChunkFold = 256;         // units after which O starts again from zero

template <int D>
struct ChunkLayout {
  static constexpr int kTile = kChunkKeys * D * 2;          // keys (or values) of a unit
  static constexpr int kQHalf = 128 * 128;                  // 64 values of 128 rows of Q
  static constexpr int kQTile = kQHalf * (D / 64);
  static constexpr int kRing = 10;
  static constexpr int kQ = 2 * kQTile;
  static constexpr int kSmem = kQ + kRing * kTile + 512 + 1024;     // barriers; base alignment
};

struct ChunkParams {
  AttnParams a;
  int page_shift, box;          // box: keys of one copy, min(page size, 64)
  int min_units;
};

// D[tmem] (+)= A[tmem] B[smem]: A's rows are lanes, two 16-bit values a column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// Shared-memory operand descriptors, 128-byte swizzled: the address (in units
// of 16 bytes, as all below), the distance to the next 64 values where the K
// dimension is the slow one in memory (V), the distance of 8-row groups.
__device__ __forceinline__ uint64_t desc(uint32_t addr16, uint32_t next, uint32_t group) {
  const uint32_t low = addr16 | (next >> 4) << 16, high = (group >> 4) | (1u << 14) | (2u << 29);
  return ((uint64_t)high << 32) | low;
}

// One lane of the (converged) warp.  With this and warp-wide votes in the
// conditions around it, the operands of the tensor instructions stay in
// uniform registers; under `lane == 0` each instruction's operands were moved
// there one by one, and issuing them took longer than running them.
__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}
// Two fp32 values as one operand, their product-sum and sum.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// o += g times the four sums at `at`, where g is not 0; `store`: kept there again.
__device__ __forceinline__ void add_held(float* at, uint32_t* o, float g, bool store) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(o[e]);
  if (g != 0.f) {
    const float4 was = __ldcg(reinterpret_cast<const float4*>(at));
    v[0] = fmaf(g, was.x, v[0]), v[1] = fmaf(g, was.y, v[1]), v[2] = fmaf(g, was.z, v[2]), v[3] = fmaf(g, was.w, v[3]);
  }
  if (store) __stcg(reinterpret_cast<float4*>(at), make_float4(v[0], v[1], v[2], v[3]));
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(v[e]);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kChunkThreads, 1)
paged_attn_chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ ChunkParams F) {
  using L = ChunkLayout<D>;
  using C = Cells<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const AttnParams& P = F.a;
  const uint32_t q_smem = tc::smem_u32(smem), ring = q_smem + L::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kQ + L::kRing * L::kTile);
  uint64_t* empty = full + L::kRing;
  uint64_t* q_full = empty + L::kRing;               // [2]
  uint64_t* s_full = q_full + 2;                     // [half * 2 + S tile], as the next two
  uint64_t* p_full = s_full + 4;
  uint64_t* pv_done = p_full + 4;
  uint64_t* drained = pv_done + 4;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tmem_at + 1);
  int64_t* scratch = reinterpret_cast<int64_t*>(smem + L::kQ + L::kRing * L::kTile + 320);   // 19 words

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = P.heads / P.kv_heads;
  if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) tc::mbar_init(&q_full[i], 4);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&p_full[i], 4);
      tc::mbar_init(&pv_done[i], 1);
    }
    tc::mbar_init(drained, 4);
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Split* split = reinterpret_cast<Split*>(static_cast<uint8_t*>(P.workspace) + kTicketBytes) + blockIdx.x;
  if (tid == 0) split->last_cta = -1;                // until this thread finds one
  const Range R = share_out<kChunkRows, kChunkKeys, kChunkThreads>(P, group, F.min_units, scratch);
  if ((int)blockIdx.x >= R.ctas) return;
  if (warp == 9) {
    tc::tmem_alloc(tmem_at, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  constexpr uint32_t tmem = 0;               // all 512 columns are this block's, so they begin at 0
  // columns: S (and in its place P) of half h, tile b at 128 h + 64 b, O at 256 and 384
  auto s_at = [&](int h, int b) { return tmem + 128u * h + 64u * b; };
  auto o_at = [&](int h) { return tmem + 256u + 128u * h; };

  // counts of tiles and phases are 32-bit (a range has fewer), whose division by the ring's length is cheap
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    if (!tc::mbar_wait(bar, phase & 1, gave_up) && !*gave_up) {
      *gave_up = 1;
      atomicOr(P.err, 1);
    }
  };

  auto landed = [&](uint32_t n) { wait(&full[n % L::kRing], n / L::kRing); };
  auto release = [&](uint32_t n) {
    if (lane == 0) tc::mbar_arrive(&empty[n % L::kRing]);
  };
  // the end of a product-issuing warp: its products are done
  auto drain = [&] {
    if (elect()) tc::mma_commit(drained);
    __syncwarp();
    if (!tc::mbar_wait_sleep(drained, 0)) atomicOr(P.err, 1);
  };

  Walk<kChunkRows, kChunkKeys> w;
  w.first(P, R, group);
  // 512 threads x 128 registers at launch = 256 x 176 + 256 x 80

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 8) {
      // ------------------------------------------------ key and value tiles
      const int none = P.num_pages > 0 ? (int)P.num_pages : 1;        // a page past the end reads as zeros
      const int parts = kChunkKeys / F.box;                            // of one tile
      uint32_t n = 0;                                                  // tiles issued
      bool stop = false;                                               // a wait of the block gave up: nothing more is
      do {
        const int64_t key0 = (w.lo / kChunkKeys) * kChunkKeys;
        const int32_t* table = P.page_table + (int64_t)w.req * P.max_pages;
        // lane i has part i's page (parts <= 4), read one unit ahead
        auto page_of = [&](int u, int& page) {                       // false: no row needs it
          const int64_t p = (key0 + (int64_t)u * kChunkKeys + (int64_t)lane * F.box) >> F.page_shift;
          const int64_t from = p << F.page_shift;
          const bool need = u < w.u1 && lane < parts && from < w.hi && from + P.page_size > w.lo;
          page = need ? table[p] : none;
          return need;
        };
        int next;
        bool needed = page_of(w.u0, next);
        for (int u = w.u0; u < w.u1 && !stop; ++u) {
          const int64_t key = key0 + (int64_t)u * kChunkKeys;
          int page = next;
          const bool bad = needed && (page < 0 || page >= P.num_pages);
          needed = page_of(u + 1, next);
          if (bad) {
            atomicOr(P.err, kErrIndex);
            page = none;
          }
          const int cell = (int)((key + (int64_t)lane * F.box) & (P.page_size - 1));
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const uint32_t slot = n % L::kRing, use = n / L::kRing;
            if (use > 0) wait(&empty[slot], use - 1);
            if ((stop = given_up(gave_up))) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(&full[slot], L::kTile);
            __syncwarp();
            if (lane < parts)
              load_cells(ring + slot * L::kTile + lane * F.box * D * 2, kv ? &vmap : &kmap, cell >> 3, page, P.kv_heads,
                         w.head, &full[slot]);
          }
        }
      } while (!stop && w.next(P, R, group));
      // copies end before the block does, whoever gives up and when: the last ones to each place of the ring
      if (lane == 0) {
        for (uint32_t j = n < L::kRing ? 0 : n - L::kRing; j < n; ++j)
          if (!tc::mbar_wait_sleep(&full[j % L::kRing], (j / L::kRing) & 1)) break;
      }
    } else if (warp == 9 || warp == 10) {
      // ----------------------------------------------------------- S = Q K^T
      // of a unit when its S tile is free: the P V of two units before is done (which also frees that unit's values).
      // Each half goes at its own pace; a ring tile is free when both have let it go.
      constexpr uint32_t kQK = tc::idesc_f16(128, kChunkKeys, BF16);
      const int h = warp - 9;
      const uint32_t q_at = (q_smem + h * L::kQTile) >> 4;
      uint32_t n0 = 0, item = 0;            // ring tiles before this item: K of unit u is n0 + 2 u, V the next
      uint32_t uses0 = 0, uses1 = 0;        // of this half's S tiles, before this item
      do {
        const int units = w.u1 - w.u0;
        if (h * 128 >= w.s.n * group - w.tile * kChunkRows) {      // no rows: only let the values go
          for (int u = 0; u < units; ++u) {
            landed(n0 + 2 * u + 1);
            release(n0 + 2 * u + 1);
          }
          n0 += 2 * units;
          continue;
        }
        wait(&q_full[h], item++);
        tc::fence_after_sync();
        for (int u = 0; u < units + 2 && !given_up(gave_up); ++u) {
          const int b = u & 1;
          if (u >= 2) {
            wait(&pv_done[2 * h + b], (b ? uses1 : uses0) + (u >> 1) - 1);
            tc::fence_after_sync();
            release(n0 + 2 * (u - 2) + 1);
          }
          if (u < units) {
            const uint32_t n = n0 + 2 * u, k_at = (ring + n % L::kRing * L::kTile) >> 4;
            landed(n);
            if (elect()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                tc::mma_f16_ss(s_at(h, b), desc(q_at + (((k >> 2) * L::kQHalf + (k & 3) * 32) >> 4), 16, 1024),
                               desc(k_at + (((k >> 2) * C::kNext + (k & 3) * 32) >> 4), 16, C::kGroup), kQK, k > 0);
              tc::mma_commit(&s_full[2 * h + b]);
            }
            __syncwarp();
          }
        }
        n0 += 2 * units;
        uses0 += (units + 1) >> 1;
        uses1 += units >> 1;
        if (given_up(gave_up)) break;
      } while (w.next(P, R, group));
      drain();
    } else if (warp == 12 || warp == 13) {
      // ------------------------------------------------------------ O += P V
      // of a unit when its P is there (so its S is done, and its keys may go)
      constexpr uint32_t kPV = tc::idesc_f16(128, D, BF16) | (1u << 16);        // B: K is its slow dimension
      const int h = warp - 12;
      uint32_t n0 = 0, uses0 = 0, uses1 = 0;
      do {
        const int units = w.u1 - w.u0;
        if (h * 128 >= w.s.n * group - w.tile * kChunkRows) {      // no rows: only let the keys go
          for (int u = 0; u < units; ++u) {
            landed(n0 + 2 * u);
            release(n0 + 2 * u);
          }
          n0 += 2 * units;
          continue;
        }
        const int64_t key0 = (w.lo / kChunkKeys) * kChunkKeys;
        for (int u = 0; u < units && !given_up(gave_up); ++u) {
          const int b = u & 1;
          const uint32_t n = n0 + 2 * u;
          landed(n + 1);
          const int64_t key = key0 + (int64_t)(w.u0 + u) * kChunkKeys;
          if (key < w.lo || key + kChunkKeys > w.hi) {
            // values that no row of the tile sees may be anything: they become zeros (both halves write them)
            const int first = w.lo > key ? (int)min(w.lo - key, (int64_t)kChunkKeys) : 0;
            const int end = w.hi > key ? (int)min(w.hi - key, (int64_t)kChunkKeys) : 0;
            uint8_t* v = smem + L::kQ + (n + 1) % L::kRing * L::kTile;
            for (int i = lane; i < kChunkKeys * (D / 8); i += 32) {
              const int r = i / (D / 8), c = i % (D / 8);
              if (r < first || r >= end)
                *reinterpret_cast<uint4*>(v + C::at(r, c >> 3, c & 7)) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
          }
          wait(&p_full[2 * h + b], (b ? uses1 : uses0) + (u >> 1));
          tc::fence_after_sync();
          const uint32_t v_at = (ring + (n + 1) % L::kRing * L::kTile) >> 4;
          if (elect()) {
            mma_f16_ts(o_at(h), s_at(h, b), desc(v_at, C::kNext, C::kGroup), kPV, u % kChunkFold != 0);
#pragma unroll
            for (int k = 1; k < kChunkKeys / 16; ++k)
              mma_f16_ts(o_at(h), s_at(h, b) + 8 * k, desc(v_at + (k * 2 * C::kGroup >> 4), C::kNext, C::kGroup), kPV, 1);
            tc::mma_commit(&pv_done[2 * h + b]);
          }
          __syncwarp();
          release(n);
        }
        n0 += 2 * units;
        uses0 += (units + 1) >> 1;
        uses1 += units >> 1;
        if (given_up(gave_up)) break;
      } while (w.next(P, R, group));
      drain();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // ------------------------------------------------------------- softmax
    const int h = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float c = fmaxf(fabsf(P.scale) * 1.4426950408889634f, 1e-30f);   // a scale of 0 must not meet -inf
    const uint32_t flip = P.scale < 0.f ? 0x80008000u : 0u;
    float* pieces = reinterpret_cast<float*>(static_cast<uint8_t*>(P.workspace) + kPieceBytes);
    uint32_t uses0 = 0, uses1 = 0;              // of this half's S tiles, before this item
    // This thread's row of the item's Q, negated where the scale is, so that the largest score has the largest weight
    auto load_q = [&](const Walk<kChunkRows, kChunkKeys>& x) {
      const int r = h * 128 + row, rows = min(kChunkRows, x.s.n * group - x.tile * kChunkRows);
      if (h * 128 >= rows) return;
      uint8_t* dst = smem + h * L::kQTile;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.q)) +
                         (r < rows ? out_row(P, x.s, x.head, group, x.tile * kChunkRows + r) * (D / 8) : 0);
      uint4 v[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) v[i] = r < rows ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        v[i].x ^= flip, v[i].y ^= flip, v[i].z ^= flip, v[i].w ^= flip;
        *reinterpret_cast<uint4*>(dst + (i >> 3) * L::kQHalf + tc::sw128_offset(row, i & 7)) = v[i];
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&q_full[h]);
    };
    load_q(w);
    bool more;
    do {
      const int row0 = w.tile * kChunkRows, rows = min(kChunkRows, w.s.n * group - row0);
      const int halves = rows > 128 ? 2 : 1, r = h * 128 + row, units = w.u1 - w.u0;
      const bool mine = r < rows;
      float m = -INFINITY, l = 0.f;
      // where the item's piece goes; until then, and for a whole item too, what O held before it started again
      auto piece = [&] { return pieces + ((size_t)blockIdx.x * 2 + (w.u0 == 0 ? 1 : 0)) * piece_floats<kChunkRows, D>(); };
      float held = -INFINITY;                  // the maximum that those sums are relative to
      const int64_t out_at = mine ? out_row(P, w.s, w.head, group, row0 + r) * D : 0;
      if (h < halves) {
        // the keys this row sees, as positions within the item
        const int64_t key0 = (w.lo / kChunkKeys) * kChunkKeys;
        const int64_t pos = w.s.kv - w.s.n + (row0 + r) / group, from = P.window ? pos - P.window + 1 : 0;
        const int hi = mine && pos + 1 > key0 ? (int)(pos + 1 - key0) : 0, lo = from > key0 ? (int)(from - key0) : 0;
        for (int begin = 0; begin < units;) {
          const int end = min(begin + kChunkFold, units);
          for (int i = begin; i < end; ++i) {
            const int b = i & 1;
            const uint32_t use = (b ? uses1 : uses0) + (i >> 1);
            wait(&s_full[2 * h + b], use);
            tc::fence_after_sync();
            uint32_t s[kChunkKeys];
#pragma unroll
            for (int k = 0; k < kChunkKeys / 32; ++k)
              tc::tmem_ld32(s_at(h, b) + lanes + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * k));
            tc::tmem_wait_ld();
            const int at = (w.u0 + i) * kChunkKeys;
            if (lo > at || hi - at < kChunkKeys) {
              const int x = lo - at, y = hi - at;
#pragma unroll
              for (int k = 0; k < kChunkKeys; ++k) s[k] = k >= x && k < y ? s[k] : 0xff800000u;      // -infinity
            }
            float t[4] = {max3(s[0], s[1], s[2]), max3(s[3], s[4], s[5]), max3(s[6], s[7], s[8]), max3(s[9], s[10], s[11])};
#pragma unroll
            for (int k = 12; k + 1 < kChunkKeys; k += 2) t[(k >> 1) & 3] = max3(__float_as_uint(t[(k >> 1) & 3]), s[k], s[k + 1]);
            const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * c;     // c >= 0
            float f = 1.f;
            bool grow = false;
            if (m == -INFINITY) {
              m = top;                       // nothing seen so far: O and l are zero
            } else if (top > m + kChunkGrow) {
              f = ex2(m - top);
              m = top;
              grow = true;
            }
            l *= f;
            if (__any_sync(0xffffffffu, grow) && i > begin) {
              // O holds every unit before this one: wait for the last of their products
              wait(&pv_done[2 * h + 1 - b], (b ? uses0 : uses1) + ((i - 1) >> 1));
              tc::fence_after_sync();
#pragma unroll 1
              for (int k = 0; k < D / 16; ++k) {
                uint32_t o[16];
                tc::tmem_ld16(o_at(h) + lanes + 16 * k, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tc::tmem_st16(o_at(h) + lanes + 16 * k, o);
              }
            }
            const float sub = m == -INFINITY ? 0.f : m - kChunkLift;
            const uint64_t c2 = pair(c, c), sub2 = pair(-sub, -sub);
            uint64_t add[2] = {0, 0};
            uint32_t p[kChunkKeys / 2];
#pragma unroll
            for (int e = 0; e < kChunkKeys / 2; ++e) {
              const float2 z = unpair(fma2(pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, sub2));
              const float x = ex2(z.x), y = ex2(z.y);
              add[e & 1] = add2(add[e & 1], pair(x, y));
              p[e] = pack2<BF16>(x, y);
            }
            tc::tmem_st32(s_at(h, b) + lanes, p);
            const float2 sum = unpair(add2(add[0], add[1]));
            l += sum.x + sum.y;
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_full[2 * h + b]);
          }
          begin = end;
          if (end == units) break;
          // O up to here, to the sums held
          wait(&pv_done[2 * h + ((end - 1) & 1)], ((end - 1) & 1 ? uses1 : uses0) + ((end - 1) >> 1));
          tc::fence_after_sync();
          const float g = held == -INFINITY ? 0.f : ex2(held - m);
          held = m;
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint32_t o[16];
            tc::tmem_ld16(o_at(h) + lanes + 16 * k, o);
            tc::tmem_wait_ld();
            if (mine) {
#pragma unroll
              for (int e = 0; e < 4; ++e) add_held(piece() + ((4 * k + e) * kChunkRows + r) * 4, o + 4 * e, g, true);
            }
          }
        }
      }
      // every score of this item is there, so Q's place is free: the next item's first scores are made while this
      // item's results are written
      auto x = w;
      more = x.next(P, R, group);
      if (more) load_q(x);
      if (h < halves) {
        // the item's last product (the ones before it are done when it is)
        wait(&pv_done[2 * h + ((units - 1) & 1)], ((units - 1) & 1 ? uses1 : uses0) + ((units - 1) >> 1));
        tc::fence_after_sync();
        uses0 += (units + 1) >> 1;
        uses1 += units >> 1;
      }
      const bool whole = w.u0 == 0 && w.u1 == w.units;
      const float g = held == -INFINITY ? 0.f : ex2(held - m);
      if (whole) {
        if (h < halves) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          uint16_t* out = static_cast<uint16_t*>(P.out) + out_at;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tc::tmem_ld32(o_at(h) + lanes + 32 * i, o);
            tc::tmem_wait_ld();
            if (mine) {
              if (g != 0.f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) add_held(piece() + ((8 * i + e) * kChunkRows + r) * 4, o + 4 * e, g, false);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  v[k] = pack2<BF16>(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                *reinterpret_cast<uint4*>(out + 32 * i + 8 * e) = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          }
          tc::fence_before_sync();
        }
      } else {
        if (tid == 0 && w.u0 == 0) {
          split->q0 = w.s.q0, split->head = w.head, split->row0 = row0, split->rows = rows;
          split->last_cta = owner(w.at + w.units - 1, R);
        }
        if (h < halves) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tc::tmem_ld32(o_at(h) + lanes + 32 * i, o);
            tc::tmem_wait_ld();
            if (mine) {
#pragma unroll
              for (int e = 0; e < 8; ++e) add_held(piece() + ((8 * i + e) * kChunkRows + r) * 4, o + 4 * e, g, true);
            }
          }
          tc::fence_before_sync();
          if (mine) {
            __stcg(piece() + kChunkRows * D + r, m);
            __stcg(piece() + kChunkRows * D + kChunkRows + r, l);
          }
        }
      }
      w = x;
    } while (more);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Puts the items together that several CTAs have pieces of: blocks (c, i) the
// one that begins in CTA c's range and goes on past it, rows 32 i .., a lane
// per row, D / 8 values a warp.  All SMs share this; the last CTA of an item
// doing it alone, as the few-row kernel's does, took 10 us of a 55 us call.
// Its pieces are laid out [D/4][rows][4], so that a warp reads whole lines.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) paged_attn_join_kernel(const AttnParams P) {
  // every block waits for the kernel before, so that this one does not end before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int group = P.heads / P.kv_heads, c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4* at_split = reinterpret_cast<const int4*>(static_cast<const uint8_t*>(P.workspace) + kTicketBytes) + 2 * c0;
  const int4 first = __ldcg(at_split);
  const int c1 = first.x, row0 = first.w, r = blockIdx.y * 32 + lane, rows = __ldcg(at_split + 1).x;
  if (c1 < 0 || r >= rows) return;
  const Shape s{first.y, 0, 0};
  const float* pieces = reinterpret_cast<const float*>(static_cast<const uint8_t*>(P.workspace) + kPieceBytes);
  auto piece = [&](int c) { return pieces + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * piece_floats<kChunkRows, D>(); };
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) m = fmaxf(m, __ldcg(piece(c) + kChunkRows * D + r));
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float mc = __ldcg(piece(c) + kChunkRows * D + r), lc = __ldcg(piece(c) + kChunkRows * D + kChunkRows + r);
    l += mc == -INFINITY ? 0.f : ex2(mc - m) * lc;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  constexpr int N = D / 32;                                   // float4 of a lane
  float4 a[N];
#pragma unroll
  for (int q = 0; q < N; ++q) a[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float mc = __ldcg(piece(c) + kChunkRows * D + r), f = mc == -INFINITY ? 0.f : ex2(mc - m) * inv;
    const float* from = piece(c) + ((size_t)(warp * N) * kChunkRows + r) * 4;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(from + q * kChunkRows * 4));
      a[q].x = fmaf(f, v.x, a[q].x), a[q].y = fmaf(f, v.y, a[q].y);
      a[q].z = fmaf(f, v.z, a[q].z), a[q].w = fmaf(f, v.w, a[q].w);
    }
  }
  const int64_t at = out_row(P, s, first.z, group, row0 + r) * D + warp * N * 4;
#pragma unroll
  for (int q = 0; q < N; ++q) store4<BF16>(P.out, false, at + 4 * q, a[q]);
}

template <int D, bool BF16>
cudaError_t launch_chunk(const CUtensorMap& kmap, const CUtensorMap& vmap, const ChunkParams& f, int ctas,
                         cudaStream_t s);

template <int D, bool BF16>
cudaError_t launch_chunk_kernel(const CUtensorMap& kmap, const CUtensorMap& vmap, const ChunkParams& f, int ctas,
                                cudaStream_t s) {
  auto kernel = paged_attn_chunk_kernel<D, BF16>;
  constexpr int smem = ChunkLayout<D>::kSmem;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kChunkThreads, smem, s>>>(kmap, vmap, f);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, kChunkRows / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<D, BF16>, f.a);
}

}  // namespace attn
}  // namespace q4k
