// q4k_moe_gate_up and q4k_moe_down: products of the experts' quantised
// matrices with the rows of the pairs that chose them.
//
#include "moe.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 256;

// y = residual + the weighted rows of z.
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(const MoeProduct P, const float* z) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MoePlan& L = P.plan;
  const int64_t t = blockIdx.x, pairs = L.tokens * L.top_k;
  const int32_t* place = L.place + t * L.top_k;
  if (place[0] == -2) return;
  for (int64_t r = threadIdx.x; r < P.rows; r += kThreads) {
    float y = P.residual ? P.residual[t * P.rows + r] : 0.0f;
    for (int j = 0; j < L.top_k; ++j) {
      const int at = place[j];
      if (at >= 0 && at < pairs) y = fmaf(L.weight[t * L.top_k + j], z[at * P.rows + r], y);
      else if ((at >= pairs || at < -1) && threadIdx.x == 0) atomicOr(P.err, kErrIndex);
    }
    P.out[t * P.rows + r] = y;
  }
}

}  // namespace

size_t moe_gate_up_workspace(int64_t, int, int, int64_t, int64_t) { return 0; }
size_t moe_down_workspace(int64_t tokens, int top_k, int, int64_t rows, int64_t) {
  return sizeof(float) * (size_t)(tokens * top_k) * (size_t)rows;
}

cudaError_t launch_moe_gate_up(const MoeProduct& p, cudaStream_t s) { return launch_moe_few_gate_up(p, p.out, s); }

cudaError_t launch_moe_down(const MoeProduct& p, cudaStream_t s) {
  float* z = static_cast<float*>(p.workspace);
  cudaError_t e = p.q6k ? launch_moe_few_down_q6(p, z, s) : launch_moe_few_down_q4(p, z, s);
  if (e != cudaSuccess) return e;
  return launch_after(moe_combine_kernel, dim3((unsigned)p.plan.tokens), kThreads, 0, s, p, (const float*)z);
}

}  // namespace q4k
