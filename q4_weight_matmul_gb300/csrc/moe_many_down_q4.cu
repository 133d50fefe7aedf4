// The products of many rows an expert: an instantiation of its own, so that they compile in parallel.
#include "moe_many.cuh"

namespace q4k {

cudaError_t launch_moe_many_down_q4(const MoeProduct& p, void* work, float* out, cudaStream_t s) {
  return p.plan.tokens * p.plan.top_k <= kMoeSmallTiles * p.plan.experts ? many::launch<many::kDownQ4, 32>(p, work, out, s)
                                                                       : many::launch<many::kDownQ4, 112>(p, work, out, s);
}

}  // namespace q4k
