// The many-row attention kernel, bf16.
#include "paged_attn_chunk.cuh"

namespace q4k {
namespace attn {
template <>
cudaError_t launch_chunk<64, true>(const CUtensorMap& kmap, const CUtensorMap& vmap, const ChunkParams& f, int ctas,
                                  cudaStream_t s) {
  return launch_chunk_kernel<64, true>(kmap, vmap, f, ctas, s);
}
template <>
cudaError_t launch_chunk<128, true>(const CUtensorMap& kmap, const CUtensorMap& vmap, const ChunkParams& f, int ctas,
                                   cudaStream_t s) {
  return launch_chunk_kernel<128, true>(kmap, vmap, f, ctas, s);
}
}  // namespace attn
}  // namespace q4k
