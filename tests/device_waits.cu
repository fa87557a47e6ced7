// device_waits.cu -- the bounded waits of aqfq_sm100_pair.cuh on their own: a warp whose lanes
// reach their limits at different times, and the drain of loads after a wait that gave up.
// Nothing here faults or waits without a limit.
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

// One warp issues 5 loads of 1 KiB on 3 stages (reusing a stage only after its load landed),
// optionally announces a sixth whose bytes never come, drains, and copies the stages out.
__global__ void drain(const uint8_t* src, int missing, long long limit, uint8_t* out, int* done) {
  constexpr int N = 1024, STAGES = 3, LOADS = 5;
  __shared__ __align__(128) uint8_t stage[STAGES][N];
  __shared__ uint64_t full[STAGES];
  const int lane = threadIdx.x;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  bool ok = true;
  for (int i = 0; i < LOADS && ok; ++i) {
    const int s = i % STAGES;
    if (i >= STAGES) ok = mbar_wait_warp(&full[s], (i / STAGES - 1) & 1);
    if (ok && lane == 0) {
      mbar_arrive_expect_tx(&full[s], N);
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              smem_u32(stage[s])),
          "l"(src + i * N), "r"(N), "r"(smem_u32(&full[s]))
          : "memory");
    }
    __syncwarp();
  }
  int issued = LOADS;
  if (missing && ok) {
    const int s = issued % STAGES;
    ok = mbar_wait_warp(&full[s], (issued / STAGES - 1) & 1);
    if (ok && lane == 0) mbar_arrive_expect_tx(&full[s], N);
    ++issued;
  }
  drain_loads(full, STAGES, issued, limit);
  for (int i = lane; i < STAGES * N; i += 32) out[i] = (&stage[0][0])[i];
  if (lane == 0) *done = ok ? 1 : 2;
}

extern "C" int run_drain(const uint8_t* src, int missing, long long limit, uint8_t* out, int* done) {
  drain<<<1, 32>>>(src, missing, limit, out, done);
  return int(cudaDeviceSynchronize());
}

// One thread runs a ring of 3 stages over `turns` loads of 1 KiB, refilling a stage after its
// turn; the loads from turn `lost` on are announced but never issued.  At the wait that gives up
// it drains what is on its way and stops; *done: the turn, out: the stages.
__global__ void ring(const uint8_t* src, int turns, int lost, long long limit, uint8_t* out, int* done) {
  constexpr int N = 1024, STAGES = 3;
  __shared__ __align__(128) uint8_t stage[STAGES][N];
  __shared__ uint64_t full[STAGES];
  for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1);
  fence_barrier_init();
  auto fetch = [&](int i) {
    if (i >= turns) return;
    const int s = i % STAGES;
    mbar_arrive_expect_tx(&full[s], N);
    if (i < lost)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              smem_u32(stage[s])),
          "l"(src + i * N), "r"(N), "r"(smem_u32(&full[s]))
          : "memory");
  };
  for (int i = 0; i < STAGES; ++i) fetch(i);
  int st = 0, i = 0;
  uint32_t phase = 0;
  for (; i < turns; ++i) {
    if (!mbar_wait_long(&full[st], phase, limit)) {
      const int left = turns - i, most = i == 0 ? STAGES : STAGES - 1;
      drain_ring(full, STAGES, st, phase, left < most ? left : most, limit);
      break;
    }
    if (i > 0) fetch(i + STAGES - 1);
    if (++st == STAGES) st = 0, phase ^= 1;
  }
  for (int k = 0; k < STAGES * N; ++k) out[k] = (&stage[0][0])[k];
  *done = i;
}

extern "C" int run_ring(const uint8_t* src, int turns, int lost, long long limit, uint8_t* out, int* done) {
  ring<<<1, 1>>>(src, turns, lost, limit, out, done);
  return int(cudaDeviceSynchronize());
}
