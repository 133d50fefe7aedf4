// The few-row attention kernel for head size 64, bf16.
#include "paged_attn_few.cuh"

namespace q4k {
namespace attn {
template <>
cudaError_t launch_few<64, true>(const CUtensorMap& kmap, const CUtensorMap& vmap, const FewParams& f, int variant,
                                int ctas, cudaStream_t s) {
  switch (variant) {
    case 0: return launch_few_variant<64, true, 1, true>(kmap, vmap, f, ctas, s);
    case 1: return launch_few_variant<64, true, 1, false>(kmap, vmap, f, ctas, s);
    case 2: return launch_few_variant<64, true, 2, false>(kmap, vmap, f, ctas, s);
    default: return launch_few_variant<64, true, 4, false>(kmap, vmap, f, ctas, s);
  }
}
}  // namespace attn
}  // namespace q4k
