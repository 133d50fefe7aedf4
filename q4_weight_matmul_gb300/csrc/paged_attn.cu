// q4k_paged_attn: causal attention of new tokens over the paged cache (host
// side: the kernel, its workspace and its tensor maps).
#include "paged_attn_chunk.cuh"
#include "paged_attn_few.cuh"
#include "tmap.h"

#include <algorithm>

namespace q4k {
namespace {

using namespace attn;

// The few-row kernel's kind (see FewConfig) and the rows of its tiles.
int few_kind(const AttnParams& p, int* rows) {
  const int64_t n = p.max_q * (p.heads / p.kv_heads);
  const int kind = n <= 4 ? 0 : n <= 8 ? 1 : n <= 16 ? 16 : n <= 32 ? 32 : 64;
  *rows = kind == 0 ? 4 : kind == 1 ? 8 : kind;
  return kind;
}

// The many-row kernel keeps its weights at 16 bits, so it gives 16-bit
// results.  It pays 128 rows per half whatever their number, the few-row
// kernel one pass over the keys' operands per 16 rows.  Few | many rows, us,
// 8 key heads of 128, pages of 16:
//   rows per key head       12            16            32            36            128
//   1 request,    512 keys  11.3 | 12.1   11.7 | 12.2   13.9 | 13.0   15.3 | 12.9   18.6 | 14.1
//   1 request,  32768 keys  47.6 | 56.6   48.5 | 51.7   58.3 | 49.5   82.4 | 56.2   140  | 52.5
//   8 requests,  4096 keys  45.5 | 41.6   46.3 | 41.2   52.8 | 40.7   74.4 | 41.9   135  | 43.3
//   8 requests, 32768 keys  245  | 196    246  | 196    272  | 180    455  | 185    898  | 180
// (16 rows and fewer keep the weights' bits, whatever the number of requests.)
bool many_rows(const AttnParams& p) { return !p.out_f32 && p.max_q * (p.heads / p.kv_heads) > 16; }

int cta_count() {
  int dev = 0;
  cudaGetDevice(&dev);
  return std::min(device_info(dev).sm_count, kMaxCtas);
}

// A cache array as (64 values, 8 cells, 64s of values, groups of 8 cells,
// pages and heads), copied `box` cells of a page at a time (see Cells).
bool cache_map(CUtensorMap* map, const AttnParams& p, const void* base, int box) {
  const uint64_t cell = (uint64_t)p.dim * 2, halves = p.dim / 64;
  const uint64_t dims[5] = {64, 8, halves, (uint64_t)p.page_size / 8,
                            (uint64_t)std::max<int64_t>(p.num_pages, 1) * p.kv_heads};
  const uint64_t strides[4] = {cell, 128, 8 * cell, cell * p.page_size};
  const uint32_t boxes[5] = {64, 8, (uint32_t)halves, (uint32_t)box / 8, 1};
  return encode_tmap(map, p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, base, dims,
                     strides, boxes, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

size_t paged_attn_workspace(const AttnParams& p) {
  int rows;
  few_kind(p, &rows);
  if (many_rows(p)) rows = kChunkRows;
  return kPieceBytes + (size_t)cta_count() * 2 * rows * (p.dim + 2) * sizeof(float);
}

cudaError_t launch_paged_attn(const AttnParams& p, cudaStream_t s) {
  const bool many = many_rows(p);
  const int box = std::min(p.page_size, many ? kChunkKeys : kUnit), ctas = cta_count();
  int shift = 4;
  while ((1 << shift) < p.page_size) ++shift;
  CUtensorMap kmap, vmap;
  if (!cache_map(&kmap, p, p.k_cache, box) || !cache_map(&vmap, p, p.v_cache, box)) return cudaErrorInvalidValue;
  if (many) {
    const ChunkParams f{p, shift, box, 2};
    if (p.dim == 128)
      return p.bf16 ? launch_chunk<128, true>(kmap, vmap, f, ctas, s) : launch_chunk<128, false>(kmap, vmap, f, ctas, s);
    return p.bf16 ? launch_chunk<64, true>(kmap, vmap, f, ctas, s) : launch_chunk<64, false>(kmap, vmap, f, ctas, s);
  }
  int rows;
  const int kind = few_kind(p, &rows);
  const FewParams f{p, shift, box, 2};
  if (p.dim == 128)
    return p.bf16 ? launch_few<128, true>(kmap, vmap, f, kind, ctas, s)
                  : launch_few<128, false>(kmap, vmap, f, kind, ctas, s);
  return p.bf16 ? launch_few<64, true>(kmap, vmap, f, kind, ctas, s)
                : launch_few<64, false>(kmap, vmap, f, kind, ctas, s);
}

}  // namespace q4k
