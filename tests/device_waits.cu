// device_waits.cu -- the bounded waits of aqfq_sm100_pair.cuh on their own: a warp whose lanes
// reach their limits at different times.  Nothing here faults or waits without a limit.
#include "aqfq_sm100_pair.cuh"

using namespace aqfq::sm100;

// One warp waits, lane i at most (i + 1) `unit` cycles; another thread completes the phase
// after half of the longest limit.  own[i]: lane i's answer alone, on a second barrier that is
// completed at the same time; all[i]: the warp's.
__global__ void uneven_limits(long long unit, int* own, int* all) {
  __shared__ uint64_t bar[2];
  if (threadIdx.x == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_barrier_init();
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 64) {
    const int w = threadIdx.x >> 5;
    const long long limit = (lane + 1) * unit;
    if (w == 0) own[lane] = mbar_wait_long(&bar[0], 0, limit);
    else all[lane] = mbar_wait_warp(&bar[1], 0, limit);
  } else if (threadIdx.x == 64) {
    const long long t0 = clock64();
    while (clock64() - t0 < 16 * unit) {}
    mbar_arrive(&bar[0]);
    mbar_arrive(&bar[1]);
  }
}

extern "C" int run_uneven_limits(long long unit, int* own, int* all) {
  uneven_limits<<<1, 96>>>(unit, own, all);
  return int(cudaDeviceSynchronize());
}
