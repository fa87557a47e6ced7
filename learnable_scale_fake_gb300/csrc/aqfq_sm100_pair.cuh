// aqfq_sm100_pair.cuh -- building blocks for a pair of CTAs (a cluster of two)
// that share one tcgen05 tile: addresses in the peer's shared memory, cluster
// barriers, TMA loads that signal the leader's mbarrier, and the cta_group::2
// forms of the tensor-memory and MMA instructions.  Inline PTX from the PTX
// ISA; the single-CTA forms are in aqfq_sm100.cuh.
#pragma once

#include "aqfq_sm100.cuh"

namespace aqfq {
namespace sm100 {

// true in one lane of a converged warp.  The tcgen05 and TMA instructions take
// uniform registers: issued under this predicate in a warp-uniform loop they need
// no per-lane serialisation.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{ .reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p; }"
      : "=r"(p));
  return p != 0;
}

// Waits for a phase: one try first, for a phase that is complete already or soon;
// then tries that may suspend the warp for long (hint in ns), which leaves the issue
// slots to the others.  Gives up after `limit` cycles (2^31: ~1 s) and returns false.
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity, uint32_t hint) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint)
      : "memory");
  return ok != 0;
}
constexpr long long kWaitCycles = 1ll << 31;
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity,
                                               long long limit = kWaitCycles) {
  if (mbar_try(bar, parity, 1000000u)) return true;
  const long long t0 = clock64();
  while (clock64() - t0 <= limit)
    if (mbar_try(bar, parity, 1000000u)) return true;
  return false;
}
// The same for a converged warp, with one answer for all of it: every lane has its own
// clock, and at the limit some could give up while others go on to a warp-wide instruction.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity,
                                               long long limit = kWaitCycles) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_long(bar, parity, limit));
}

// After a wait that gave up: waits, bounded, for the loads still on their way, at most one
// per stage.  issued: loads so far, number i on the barrier of stage i % stages.  A warp
// calls it before its block ends, so that no copy lands in the next block's memory.
__device__ __forceinline__ void drain_loads(uint64_t* full, int stages, int issued,
                                            long long limit = kWaitCycles) {
  for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
    mbar_wait_warp(&full[i % stages], (i / stages) & 1, limit);
}

// The same for one thread that refills a ring itself: `left` loads are on their way, the
// oldest on the barrier of stage st with this phase.
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, int st, uint32_t phase, int64_t left,
                                           long long limit = kWaitCycles) {
  for (int64_t i = 0; i < left; ++i) {
    mbar_wait_long(&full[st], phase, limit);
    if (++st == stages) st = 0, phase ^= 1;
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// address of the same variable in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
// one arrival on an mbarrier given by its cluster address.  Relaxed: it hands over
// tensor memory whose loads are complete, no data in memory, and a release would
// first wait for the thread's outstanding global stores.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// 2D tile into this CTA's shared memory, its bytes counted on the mbarrier at
// cluster address `bar` (in either CTA of the pair)
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, uint32_t bar,
                                                 int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// one warp of each CTA of the pair
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(slot)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// one thread of the pair's leader: both CTAs' operand halves, both accumulators
__device__ __forceinline__ void tc_mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// when the prior MMAs are complete: one arrival on the mbarrier at this offset in
// the CTAs of `mask` (cluster ranks)
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar, uint32_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(uint16_t(mask))
      : "memory");
}

// Shared-memory matrix descriptor of an operand whose row axis (M or N) is
// contiguous, 128-byte swizzle: atoms of 64 row elements (128 bytes) x 8 of k
// (1024 bytes).  Along k the atoms follow each other (stride byte offset 1024);
// the next 64 row elements start `block` bytes further (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= uint64_t((saddr & 0x3FFFFu) >> 4);
  d |= uint64_t(block >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}
// instruction descriptor bits of a row-contiguous A / B operand
constexpr uint32_t kIdescTransA = 1u << 15, kIdescTransB = 1u << 16;

}  // namespace sm100
}  // namespace aqfq
