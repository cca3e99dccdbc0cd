// Self-test of the bounded-wait path every pipeline kernel relies on: a wait
// on an mbarrier that nothing arrives on runs out after the given number of
// clocks, sets the abort flag and reports DSA_STATUS_TIMEOUT in the status
// word, and the kernel returns normally (no trap, the context stays usable).
// A second wait of the whole warp is met in half of its lanes and runs out in
// the others: every lane has to learn that it did, or DSA_STATUS_INTERNAL is
// reported as well.
#include "common.cuh"

namespace dsa {

namespace {
__global__ void wait_timeout_kernel(long long limit_clocks, int32_t* dev_status) {
  __shared__ __align__(8) uint64_t bar, met;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    mbar_init(&met, 1);
    abort_flag = 0;
    fence_mbar_init();
    mbar_arrive(&met);
    if (!mbar_wait_limit(&bar, 0, &abort_flag, limit_clocks)) set_status(dev_status, DSA_STATUS_TIMEOUT);
    abort_flag = 0;
  }
  __syncwarp();
  if (mbar_wait_warp_limit(threadIdx.x < 16 ? &met : &bar, 0, &abort_flag, limit_clocks))
    set_status(dev_status, DSA_STATUS_INTERNAL);
}
}  // namespace

int run_wait_timeout_selftest(cudaStream_t stream, long long limit_clocks, int32_t* dev_status) {
  wait_timeout_kernel<<<1, 32, 0, stream>>>(limit_clocks, dev_status);
  DSA_CHECK_LAUNCH();
  return DSA_OK;
}

}  // namespace dsa
