// q4k_moe_gate_up and q4k_moe_down: products of the experts' quantised
// matrices with the rows of the pairs that chose them.
//
#include "moe.cuh"

#include <algorithm>
#include <type_traits>

namespace q4k {
namespace {

constexpr int kThreads = 256;

// y = residual + the weighted rows of z: a thread adds up V neighbouring
// outputs of one token, its loads of up to kBatch rows in flight at once.
constexpr int kBatch = 8;

template <int V>
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(const MoeProduct P, const float* z) {
  using F = std::conditional_t<V == 4, float4, float>;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MoePlan& L = P.plan;
  const int64_t per = P.rows / V, at = (int64_t)blockIdx.x * kThreads + threadIdx.x, t = at / per;
  if (t >= L.tokens) return;
  const int64_t r = (at - t * per) * V;
  const int32_t* place = L.place + t * L.top_k;
  const float* weight = L.weight + t * L.top_k;
  const int64_t made = L.offsets[0], pairs = min((int64_t)L.offsets[L.experts], L.tokens * L.top_k);   // rows of z from made to pairs - 1
  if (place[0] == -2) return;
  alignas(16) float y[V] = {};
  if (P.residual) *reinterpret_cast<F*>(y) = *reinterpret_cast<const F*>(P.residual + t * P.rows + r);
  for (int j0 = 0; j0 < L.top_k; j0 += kBatch) {
    alignas(16) float v[kBatch][V];
    float w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int p = j0 + j < L.top_k ? place[j0 + j] : -1;
      const bool have = p >= 0 && p >= made && p < pairs;
      if (!have && p != -1 && r == 0) atomicOr(P.err, kErrIndex);
      w[j] = have ? weight[j0 + j] : 0.0f;
      if (have) {
        *reinterpret_cast<F*>(v[j]) = *reinterpret_cast<const F*>(z + p * P.rows + r);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = fmaf(w[j], v[j][i], y[i]);
  }
  *reinterpret_cast<F*>(P.out + t * P.rows + r) = *reinterpret_cast<const F*>(y);
}

cudaError_t combine(const MoeProduct& p, const float* z, cudaStream_t s) {
  const int64_t n = p.plan.tokens * p.rows;
  if (p.rows % 4 == 0)
    return launch_after(moe_combine_kernel<4>, dim3((unsigned)((n / 4 + kThreads - 1) / kThreads)), kThreads, 0, s, p, z);
  return launch_after(moe_combine_kernel<1>, dim3((unsigned)((n + kThreads - 1) / kThreads)), kThreads, 0, s, p, z);
}

}  // namespace

// Many pairs an expert go to the tensor cores' tiles of up to 112 pairs, few
// to the kernel that streams the weights once per 16 pairs: its time grows with
// the pairs, that of a tile hardly does until it is full.  One rule for the
// three products; down Q6_K alone would take the other side from some 6 pairs
// on (up to 11 %).  Measured (us; gate and up, down Q4_K, down Q6_K), few | many:
//   pairs an expert   128 experts, 2048 x 768              32 experts, 2560 x 1536
//         6           82 / 55 / 82   | 86 / 55 / 74        50 / 35 / 52 | 67 / 39 / 51
//        10          104 / 69 / 98   | 96 / 58 / 78        66 / 44 / 63 | 68 / 49 / 59
//        16          141 / 91 / 124  | 101 / 65 / 85       92 / 55 / 77 | 69 / 50 / 59
constexpr int64_t kMany = 10;
static bool many(int64_t tokens, int top_k, int experts) { return tokens * top_k >= kMany * experts; }

// Operands for any number of pairs up to this one.
static size_t operands(int64_t tokens, int top_k, int experts, int64_t cols) {
  const int64_t pairs = tokens * top_k;
  const size_t few = moe_few_workspace(std::min(pairs, kMany * experts), experts, cols);
  return many(tokens, top_k, experts) ? std::max(few, moe_many_workspace(pairs, experts, cols)) : few;
}
// The down products' rows, before they are put together, lie behind them.
static size_t rows_at(size_t operands) { return (operands + 255) / 256 * 256; }

size_t moe_gate_up_workspace(int64_t tokens, int top_k, int experts, int64_t, int64_t cols) {
  return operands(tokens, top_k, experts, cols);
}
size_t moe_down_workspace(int64_t tokens, int top_k, int experts, int64_t rows, int64_t cols) {
  return rows_at(operands(tokens, top_k, experts, cols)) + sizeof(float) * (size_t)(tokens * top_k) * (size_t)rows;
}

cudaError_t launch_moe_gate_up(const MoeProduct& p, cudaStream_t s) {
  if (many(p.plan.tokens, p.plan.top_k, p.plan.experts)) return launch_moe_many_gate_up(p, p.workspace, p.out, s);
  return launch_moe_few_gate_up(p, p.workspace, p.out, s);
}

cudaError_t launch_moe_down(const MoeProduct& p, cudaStream_t s) {
  float* z = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) +
                                      rows_at(operands(p.plan.tokens, p.plan.top_k, p.plan.experts, p.cols)));
  const bool m = many(p.plan.tokens, p.plan.top_k, p.plan.experts);
  cudaError_t e = p.q6k ? (m ? launch_moe_many_down_q6 : launch_moe_few_down_q6)(p, p.workspace, z, s)
                        : (m ? launch_moe_many_down_q4 : launch_moe_few_down_q4)(p, p.workspace, z, s);
  if (e != cudaSuccess) return e;
  return combine(p, z, s);
}

}  // namespace q4k
