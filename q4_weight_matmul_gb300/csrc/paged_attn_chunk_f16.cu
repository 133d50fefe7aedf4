// The many-row attention kernel, f16.
#include "paged_attn_chunk.cuh"

namespace q4k {
namespace attn {
template <>
cudaError_t launch_chunk<64, false>(const CUtensorMap& kmap, const CUtensorMap& vmap, const ChunkParams& f, int ctas,
                                  cudaStream_t s) {
  return launch_chunk_kernel<64, false>(kmap, vmap, f, ctas, s);
}
template <>
cudaError_t launch_chunk<128, false>(const CUtensorMap& kmap, const CUtensorMap& vmap, const ChunkParams& f, int ctas,
                                   cudaStream_t s) {
  return launch_chunk_kernel<128, false>(kmap, vmap, f, ctas, s);
}
}  // namespace attn
}  // namespace q4k
