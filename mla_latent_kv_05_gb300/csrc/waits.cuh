// Small pieces that warp-specialised tcgen05 kernels share: bounded mbarrier
// waits with little code (the roles share the instruction caches, and an
// unrolled wait in every place costs the other roles their lines) and the
// election of an issuing lane.
#pragma once
#include "common.cuh"

namespace mla {

// TMA boxes from a tensor map that spans less than 128 KiB load about three
// times slower (a 100-row expansion took 30 us, a 128-row one 13 us, and the
// 100 rows with a wider stride 13 us).  Maps over tensors that may be that
// small get one more dimension of two entries this many bytes apart; only its
// entry 0 is ever addressed.
constexpr uint64_t kTmaFar = uint64_t{1} << 24;

// As wait_bounded<false> (common.cuh): false, with MLA_STATUS_TIMEOUT recorded
// and the abort flag raised, when the phase did not complete in time; false
// too once another thread of the grid gave up.  kCluster: acquire at cluster
// scope, for phases that another CTA's arrivals complete.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity, PlanHeader* hdr) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1; !(kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)); ++n) {
    if ((n & 1023u) != 0) continue;
    const uint64_t now = ptx::globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 > MLA_WAIT_TIMEOUT_NS) {
      set_status(&hdr->status, MLA_STATUS_TIMEOUT);
      atomicExch(&hdr->abort_flag, 1);
      return false;
    }
    if (read_status(&hdr->abort_flag) != 0) return false;
  }
  return true;
}

// The same for a converged warp, which leaves together.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_short_warp(uint32_t bar, uint32_t parity, PlanHeader* hdr) {
  return __all_sync(0xffffffffu, wait_short<kCluster>(bar, parity, hdr));
}

// One lane of a converged warp.  The compiler knows that a branch on it is
// taken by a single thread and keeps what it issues in uniform registers: a
// commit costs about 2 cycles to issue in such a branch, 46 under lane == 0 and
// 60 as a predicated instruction, and an MMA's descriptors no moves.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

}  // namespace mla
