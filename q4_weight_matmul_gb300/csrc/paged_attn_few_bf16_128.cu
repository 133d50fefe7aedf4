// The few-row attention kernel for head size 128, bf16.
#include "paged_attn_few.cuh"

namespace q4k {
namespace attn {
template <>
cudaError_t launch_few<128, true>(const CUtensorMap& kmap, const CUtensorMap& vmap, const FewParams& f, int kind,
                                int ctas, cudaStream_t s) {
  switch (kind) {
    case 0: return launch_few_variant<128, true, 0>(kmap, vmap, f, ctas, s);
    case 1: return launch_few_variant<128, true, 1>(kmap, vmap, f, ctas, s);
    case 16: return launch_few_variant<128, true, 16>(kmap, vmap, f, ctas, s);
    case 32: return launch_few_variant<128, true, 32>(kmap, vmap, f, ctas, s);
    default: return launch_few_variant<128, true, 64>(kmap, vmap, f, ctas, s);
  }
}
}  // namespace attn
}  // namespace q4k
