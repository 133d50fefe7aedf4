// The products of many rows an expert: an instantiation of its own, so that they compile in parallel.
#include "moe_many.cuh"

namespace q4k {

cudaError_t launch_moe_many_gate_up(const MoeProduct& p, void* work, float* out, cudaStream_t s) {
  return p.plan.tokens * p.plan.top_k <= kMoeSmallTiles * p.plan.experts ? many::launch<many::kGateUp, 32>(p, work, out, s)
                                                                       : many::launch<many::kGateUp, 112>(p, work, out, s);
}

size_t moe_many_workspace(int64_t pairs, int experts, int64_t cols) {
  const int64_t small = kMoeSmallTiles * experts;
  const size_t need = many::places(std::min(pairs, small), experts, cols, 32).end;
  return pairs <= small ? need : std::max(need, many::places(pairs, experts, cols, 112).end);
}

}  // namespace q4k
