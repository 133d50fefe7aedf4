// The products of many rows an expert: an instantiation of its own, so that they compile in parallel.
#include "moe_many.cuh"

namespace q4k {

cudaError_t launch_moe_many_gate_up(const MoeProduct& p, void* work, float* out, cudaStream_t s) {
  return many::launch<many::kGateUp>(p, work, out, s);
}

size_t moe_many_workspace(int64_t pairs, int experts, int64_t cols) { return many::places(pairs, experts, cols).end; }

}  // namespace q4k
