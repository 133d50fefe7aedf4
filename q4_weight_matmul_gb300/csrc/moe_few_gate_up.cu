// The products of few rows an expert: an instantiation of its own, so that they compile in parallel.
#include "moe_few.cuh"

namespace q4k {

cudaError_t launch_moe_few_gate_up(const MoeProduct& p, void* work, float* out, cudaStream_t s) {
  return few::launch_mode<few::kGateUp>(p, work, out, s);
}

}  // namespace q4k
