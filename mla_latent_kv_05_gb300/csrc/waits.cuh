// Small pieces that warp-specialised tcgen05 kernels share: bounded mbarrier
// waits with little code (the roles share the instruction caches, and an
// unrolled wait in every place costs the other roles their lines) and the
// election of an issuing lane.
#pragma once
#include "common.cuh"

namespace mla {

namespace ptx {

// tcgen05 over a pair of CTAs (cta_group::2)
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A B^T over the pair: A and D rows 128 of each CTA, B rows half from each
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// arrive on the barrier at this offset in both CTAs once this thread's MMAs are done
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
// Tell the pair's leader, in the other CTA or in this one.  What the arrival
// hands over lies in this CTA's own shared memory (written, and made visible to
// the MMAs by fence.proxy.async, before it) or tensor memory (read or written,
// tcgen05.fence).  So the release at cluster scope, which the waiter's acquire
// needs to see this CTA's writes, is restricted to shared memory; an unrestricted
// one also waits for the CTA's writes to global memory, 1000 cycles a tile.
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
               "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
// tiled loads whose bytes are counted on a barrier of either CTA of the pair (a cluster address)
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z,
                                             uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
               " [%0], [%1, {%3, %4, %5}], [%2], %6;"
               :: "r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy) : "memory");
}
}  // namespace ptx

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
