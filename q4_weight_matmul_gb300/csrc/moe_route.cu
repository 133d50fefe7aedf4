// q4k_moe_route: each token's best experts and their weights from the router's
// logits, and the (token, expert) pairs grouped by expert.
//
//   chosen(t) = the top_k experts with the largest logits l[t][e] > -inf, the
//   best first, the lower index first where logits are equal;
//   w[t][j] = scale * exp(l_j - max) / (sum over chosen(t), or over all e).
//   Pair p = t * top_k + j; the pairs of expert e stand at order[offsets[e]] ..
//   order[offsets[e+1] - 1] in ascending p, and place[p] is p's position.
//
// One warp per token: lane i holds the logits of experts i, i + 32, ..; each of
// the top_k rounds is two warp reductions (the largest key, the lowest index
// that has it), and lane j keeps what round j found.  Keys are the logits' bits
// in an order that unsigned comparison keeps, so the choice is exact.
//
// The grouping counts, so that it needs no atomics and always gives the same
// order: a warp ranks its own tokens' pairs within each expert as it goes, a
// CTA of 32 warps turns the warps' counts into starts.  Up to kOneCta tokens
// one CTA does it all in one launch.  More tokens are shared out over about an
// SM each in chunks of whole warps; the first launch leaves every chunk's
// counts, and in the second each CTA adds up those of the chunks before its own
// and of all (E x chunks integers from L2) and writes the pairs' final places.
//
// Measured: 1 token, 8 of 128 experts 3.4 us; 208 tokens, 4 of 60 experts 6.1;
// 8192 tokens, 8 of 128 experts 12.0 (5.2 MB: 0.8 us at the copy rate).  Bound:
// latency, of the launches, the loads that wait for one another (15.4 us before
// the next token's logits and a chunk's pairs were asked for ahead), and top_k
// rounds of two warp reductions a token.
#include "moe.cuh"

namespace q4k {
namespace {

constexpr int kWarps = 32;
constexpr int kThreads = 32 * kWarps;
constexpr int64_t kOneCta = 128;      // tokens
constexpr int64_t kMaxChunks = 152;

struct RouteParams {
  MoePlan plan;
  const float* logits;
  const int32_t* n_tokens;
  int* err;
  int32_t* counts;                    // [chunks][experts]
  int per_warp;                       // tokens of a warp; a chunk has 32 times as many
  bool renormalize;
  float scale;
};

// Larger logits have larger keys; 0 where the expert is not to be had (-inf, NaN).
__device__ __forceinline__ uint32_t key_of(float v) {
  if (!(v > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(v + 0.0f);            // -0 as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}
// exp(l - top) where l may be +inf as top is, or -inf
__device__ __forceinline__ float share(float l, float top) { return l == top ? 1.0f : expf(l - top); }

__device__ __forceinline__ int64_t valid_tokens(const RouteParams& P) {
  if (!P.n_tokens) return P.plan.tokens;
  const int64_t n = *P.n_tokens;
  if ((n < 0 || n > P.plan.tokens) && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.err, kErrIndex);
  return n < 0 ? 0 : n > P.plan.tokens ? P.plan.tokens : n;
}

// The exclusive sum of total[0 .. n-1] in off[0 .. n]; one warp.
__device__ void scan_experts(const int* total, int* off, int n) {
  const int lane = threadIdx.x & 31;
  int run = 0;
  for (int e0 = 0; e0 < n; e0 += 32) {
    const int e = e0 + lane, v = e < n ? total[e] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += u;
    }
    if (e < n) off[e] = run + s - v;
    run += __shfl_sync(~0u, s, 31);
  }
  if (lane == 0) off[n] = run;
}

// NV logits a lane: up to 32 NV experts.
template <int NV, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) route_choose_kernel(const RouteParams P) {
  __shared__ uint16_t counts[kWarps][32 * NV];             // a warp's pairs of each expert; then where they start
  __shared__ int total[32 * NV], off[32 * NV + 1];
  if constexpr (!ONE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const MoePlan& L = P.plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = L.experts, k = L.top_k;
  for (int e = lane; e < 32 * NV; e += 32) counts[warp][e] = 0;
  __syncwarp();
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * P.per_warp, last = min(first + P.per_warp, L.tokens);
  // the next token's logits are on their way while one's experts are chosen (more than 256 experts: registers for it lack)
  float next[NV];
  const auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) next[i] = 32 * i + lane < E && t < last ? P.logits[t * E + 32 * i + lane] : 0.0f;
  };
  load(first);
  const int64_t live = valid_tokens(P);
  int kept[2] = {-1, -1}, ranks[2] = {-1, -1};             // of the first two tokens
  for (int64_t t = first; t < last; ++t) {
    int expert = -1, rank = -1;
    float weight = 0.0f;
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = 32 * i + lane < E ? key_of(next[i]) : 0;
    if constexpr (NV <= 8) load(t + 1);
    if (t < live) {
      uint32_t mine = 0;                                   // what round `lane` found
      float top = 0.0f, all = 0.0f;
      uint32_t left[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) left[i] = key[i];
      for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (left[i] > best) best = left[i], at = 32 * i + lane;
        const uint32_t most = __reduce_max_sync(~0u, best);
        if (most == 0) break;
        const int e = (int)__reduce_min_sync(~0u, best == most ? (unsigned)at : ~0u);
        if (j == 0) top = logit_of(most);
        if (lane == j) mine = most, expert = e;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (32 * i + lane == e) left[i] = 0;
      }
      if (expert >= 0) weight = share(logit_of(mine), top);
      if (P.renormalize) {
        all = weight;
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (key[i]) all += share(logit_of(key[i]), top);
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) all += __shfl_xor_sync(~0u, all, o);
      if (expert >= 0) {
        weight = weight / all * P.scale;
        rank = counts[warp][expert];                       // the token's experts differ
        counts[warp][expert] = (uint16_t)(rank + 1);
      }
      __syncwarp();
    }
    if (lane < k) {
      const int64_t p = t * k + lane;
      L.expert[p] = expert;
      L.weight[p] = weight;
      L.place[p] = t < live ? rank : -2;
    }
    if constexpr (NV > 8) load(t + 1);
    if (t == first) kept[0] = expert, ranks[0] = rank;
    if (t == first + 1) kept[1] = expert, ranks[1] = rank;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int run = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int c = counts[w][e];
      counts[w][e] = (uint16_t)run;
      run += c;
    }
    if constexpr (ONE) total[e] = run;
    else P.counts[(int64_t)blockIdx.x * E + e] = run;
  }
  __syncthreads();
  if constexpr (ONE) {
    if (warp == 0) scan_experts(total, off, E);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kThreads) L.offsets[e] = off[e];
    for (int64_t p = off[E] + threadIdx.x; p < L.tokens * k; p += kThreads) L.order[p] = -1;
  }
  // the lanes that wrote a pair finish it
  for (int64_t t = first; t < last; ++t) {
    if (lane >= k) break;
    const int64_t p = t * k + lane;
    const int e = t == first ? kept[0] : t == first + 1 ? kept[1] : L.expert[p];
    if (e < 0) continue;
    int at = (t == first ? ranks[0] : t == first + 1 ? ranks[1] : L.place[p]) + counts[warp][e];
    if constexpr (ONE) {
      at += off[e];
      L.order[at] = (int32_t)p;
    }
    L.place[p] = at;
  }
}

__global__ void __launch_bounds__(kThreads, 1) route_place_kernel(const RouteParams P, int chunks) {
  __shared__ int part[2][kThreads];
  __shared__ int total[kMoeMaxExperts], off[kMoeMaxExperts + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MoePlan& L = P.plan;
  const int E = L.experts, width = (E + 31) / 32 * 32, groups = kThreads / width;
  const int g = threadIdx.x / width, e = threadIdx.x - g * width, c = blockIdx.x;
  const int64_t first = (int64_t)c * kWarps * P.per_warp * L.top_k,
                last = min(first + (int64_t)kWarps * P.per_warp * L.top_k, L.tokens * L.top_k), p0 = first + threadIdx.x;
  const int expert0 = p0 < last ? L.expert[p0] : -1, rank0 = p0 < last ? L.place[p0] : 0;
  int before = 0, all = 0;
  if (g < groups && e < E) {
#pragma unroll 16
    for (int i = g; i < chunks; i += groups) {
      const int v = P.counts[(int64_t)i * E + e];
      all += v;
      before += i < c ? v : 0;
    }
  }
  part[0][threadIdx.x] = before;
  part[1][threadIdx.x] = all;
  __syncthreads();
  if (threadIdx.x < width && e < E) {
    for (int i = 1; i < groups; ++i) before += part[0][i * width + e], all += part[1][i * width + e];
    total[e] = all;
  }
  __syncthreads();
  if (threadIdx.x < 32) scan_experts(total, off, E);
  __syncthreads();
  if (c == 0)
    for (int i = threadIdx.x; i <= E; i += kThreads) L.offsets[i] = off[i];
  const int pairs = off[E];
  if (threadIdx.x < width && e < E) total[e] = off[e] + before;
  __syncthreads();
  for (int64_t p = p0; p < last; p += kThreads) {
    const int x = p == p0 ? expert0 : L.expert[p];
    if (x >= 0) {
      const int at = (p == p0 ? rank0 : L.place[p]) + total[x];
      L.place[p] = at;
      L.order[at] = (int32_t)p;
    }
    if (p >= pairs) L.order[p] = -1;
  }
}

int per_warp(int64_t tokens, int64_t ctas) { return (int)((tokens + ctas * kWarps - 1) / (ctas * kWarps)); }

template <int NV>
cudaError_t launch(RouteParams& P, cudaStream_t s) {
  const int64_t tokens = P.plan.tokens;
  if (tokens <= kOneCta) {
    P.per_warp = per_warp(tokens, 1);
    route_choose_kernel<NV, true><<<1, kThreads, 0, s>>>(P);
    return cudaGetLastError();
  }
  P.per_warp = per_warp(tokens, kMaxChunks);
  const int chunks = (int)((tokens + kWarps * P.per_warp - 1) / (kWarps * P.per_warp));
  route_choose_kernel<NV, false><<<chunks, kThreads, 0, s>>>(P);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(route_place_kernel, dim3(chunks), kThreads, 0, s, P, chunks);
}

}  // namespace

size_t moe_route_workspace(int64_t tokens, int experts) {
  return tokens <= kOneCta ? 0 : sizeof(int32_t) * (size_t)experts * kMaxChunks;
}

cudaError_t launch_moe_route(const MoePlan& plan, const float* logits, const int32_t* n_tokens, bool renormalize,
                             float scale, void* workspace, int* err, cudaStream_t s) {
  RouteParams P{plan, logits, n_tokens, err, static_cast<int32_t*>(workspace), 0, renormalize, scale};
  if (plan.experts <= 32) return launch<1>(P, s);
  if (plan.experts <= 64) return launch<2>(P, s);
  if (plan.experts <= 128) return launch<4>(P, s);
  if (plan.experts <= 256) return launch<8>(P, s);
  return launch<16>(P, s);
}

}  // namespace q4k
