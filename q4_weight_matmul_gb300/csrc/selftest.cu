// Self-tests of the bounded-wait error path: a kernel waits on an mbarrier
// that nothing ever arrives at.  The wait gives up after the library's limit
// (tc::kTimeoutCycles; the warps' waits after a short one), the kernel records
// the timeout in the device error word and returns normally, so the context
// stays usable.
#include "moe_few.cuh"

namespace q4k {
namespace {

__global__ void wait_timeout_selftest_kernel(int* err) {
  __shared__ uint64_t bar;
  if (threadIdx.x != 0) return;
  tc::mbar_init(&bar, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (!tc::mbar_wait_sleep(&bar, 0)) atomicOr(err, 4);
}

// The waits of the routed experts' kernels, one warp, one after the other.
constexpr long long kShort = 1 << 26;        // cycles: some 32 ms

__global__ void warp_waits_selftest_kernel(int32_t* out, int* err) {
  __shared__ uint64_t never, done;
  __shared__ uint32_t issued;
  __shared__ int flag, word;
  const int lane = threadIdx.x;
  volatile int* gave_up = &flag;
  if (lane == 0) {
    tc::mbar_init(&never, 1);
    tc::mbar_init(&done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tc::mbar_arrive(&done);
    issued = 1;                               // stage 0
  }
  __syncwarp();
  for (int i = 0; i < 7; ++i) {
    if (lane == 0) *gave_up = i == 1, word = 0;
    __syncwarp();
    const long long t0 = clock64();
    bool ok = false;
    if (i <= 1) ok = warp_wait<kShort>(&never, 0, gave_up, &word);
    if (i == 2) ok = warp_wait<kShort>(&done, 0, &never, 0, gave_up, &word);
    if (i == 3) ok = warp_wait<kShort>(&done, 0, &done, 0, gave_up, &word);
    if (i == 4) ok = few::warp_wait_issued<kShort>(&issued, 1, gave_up, &word);
    if (i == 5) ok = few::warp_wait_issued<kShort>(&issued, 0, gave_up, &word);
    if (i == 6) ok = agreed(lane != 7, gave_up, &word);
    const int took = (int)((clock64() - t0) >> 16);
    out[32 * i + lane] = ok;
    __syncwarp();
    if (lane == 0) {
      out[32 * 7 + i] = word | *gave_up << 8;
      out[32 * 7 + 8 + i] = took;
      if (i == 0) atomicOr(err, word);
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_warp_waits_selftest(int32_t* out, int* err, cudaStream_t s) {
  warp_waits_selftest_kernel<<<1, 32, 0, s>>>(out, err);
  return cudaGetLastError();
}

cudaError_t launch_wait_timeout_selftest(int* err, cudaStream_t s) {
  wait_timeout_selftest_kernel<<<1, 32, 0, s>>>(err);
  return cudaGetLastError();
}

}  // namespace q4k
