// Bounded mbarrier waits with little code: kernels whose warps play different
// roles share the instruction caches, and an unrolled wait in every place
// costs the other roles their lines.
#pragma once
#include "common.cuh"

namespace mla {

// As wait_bounded<false> (common.cuh): false, with MLA_STATUS_TIMEOUT recorded
// and the abort flag raised, when the phase did not complete in time; false
// too once another thread of the grid gave up.
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity, PlanHeader* hdr) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1; !ptx::mbar_try_wait(bar, parity); ++n) {
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
__device__ __forceinline__ bool wait_short_warp(uint32_t bar, uint32_t parity, PlanHeader* hdr) {
  return __all_sync(0xffffffffu, wait_short(bar, parity, hdr));
}

}  // namespace mla
