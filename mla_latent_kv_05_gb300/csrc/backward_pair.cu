// The query pass of the backward pass (backward.cu) on CTA pairs: dq, where dS is not stored.
//
// A pair holds 256 queries, 128 in each CTA, and streams tiles of 128 keys past them
// with cta_group::2 MMAs, each of which reads its second operand half from either
// CTA.  Where one CTA alone reads 8 KiB of shared memory for a 64-cycle MMA of S or
// dP (all that shared memory gives in that time, and the copies come on top: an S
// took 1200 cycles instead of 768), each CTA of a pair reads 6, and 3 instead of 6
// for dq; and the streamed tiles' shares are small enough to be held twice.
// Measured, with nothing stored: 2,580 cycles a step against 3,450 (of 2,048 of MMAs),
// 4096 causal tokens 1,605 us a call against 1,695; 3 x 777 full 597 and 615, 2 x 512 queries over 7,500
// keys more 1,686 and 1,808.  Not for short sequences (backward_rows): a pair's tiles
// of 256 rows are half empty in them (8 x up to 1024 tokens 648 us instead of 611).
// Nor for the key pass, whose S and dP share one place in tensor memory: every
// hand-over between the MMAs and the warps is in its chain, and those between two
// CTAs are longer (1,664 us instead of 1,605).
//
// The products split the streamed tile differently: S and dP along its rows (each CTA
// 64 of the 128), dq along its values (each CTA half of the 128 and half of the 64
// RoPE values).  So each CTA loads both forms of K, together about as much as one
// whole tile, and each is freed by its own products.
//   shared memory: Q 48 KiB, dO 32, K in the first form 2 x 24 and in the second
//       2 x 32 (of the RoPE chunk's 64 columns 32 are used), V 2 x 16;
//   tensor memory: dq 192 | dP 128 | S 128 | dS 64; dq lies as the MMAs produce it:
//       values 0..63, RoPE 0..31, values 64..127, RoPE 32..63;
//   warp 0: work items and the queries; warps 3, 4 and 5 load K in either form and V,
//   warp 1 issues S and dP, warp 2 dq (rank 0's, for both), warps 8..23 compute dS and
//   write the results (thread = a quarter row).
// Rank 0 claims the items and issues all MMAs; both ranks load their shares and
// compute dS of their rows, whose arrivals go to rank 0's barriers.
#include "backward_tile.cuh"

namespace mla {

namespace {

using namespace bwd;

constexpr int kHelpers = 8;                            // warps that load and issue
constexpr int kThreads = 32 * (kHelpers + kWarps);
constexpr uint32_t kHalf = 64u * 128u;                 // 8 KiB: 64 rows x 64 values
constexpr uint32_t kOffR1 = 0, kOffR2 = 3 * kChunk, kOffC1S = 5 * kChunk, kOffC1D = kOffC1S + 6 * kHalf,
                   kOffC2 = kOffC1D + 4 * kChunk;
constexpr uint32_t kOffBar = kOffC2 + 4 * kHalf;
constexpr int kItemSlots = 2;
enum Bar {
  // rank 0's, which count both ranks' copies (S: K in the first form, D: in the second) ...
  R1FULL, R2FULL, C1SFULL, C2FULL = C1SFULL + 2, C1DFULL = C2FULL + 2,
  // ... or arrivals of both ranks' warps
  SREAD = C1DFULL + 2, DPREAD, DSREADY, ACCFREE,
  // each rank's own copies that have to be cleared before they are used
  TAIL,
  // commits, in both ranks
  R1EMPTY, R2EMPTY, C1SEMPTY, C2EMPTY = C1SEMPTY + 2, C1DEMPTY = C2EMPTY + 2, SFULL = C1DEMPTY + 2, DPFULL, DSDONE, DRAIN,
  // items: to rank 1 and its answer, and to each rank's roles
  ITEM, ITEMACK = ITEM + kItemSlots, IFULL = ITEMACK + kItemSlots, IEMPTY = IFULL + kItemSlots,
  NBAR = IEMPTY + kItemSlots
};
constexpr uint32_t kOffTmem = kOffBar + 8 * NBAR;
constexpr uint32_t kOffNext = kOffTmem + 4;                      // item numbers for rank 1
constexpr uint32_t kOffItems = (kOffNext + 4 * kItemSlots + 15) & ~15u;
constexpr uint32_t kSmem = kOffItems + kItemBytes * kItemSlots;
static_assert(kSmem <= 232448, "shared memory budget");

constexpr uint32_t kIdescS = ptx::idesc_bf16(256, 128, 0, 0);    // both K-major
constexpr uint32_t kIdesc192 = ptx::idesc_bf16(256, 192, 0, 1);

// As pair_mma_ss with A in tensor memory (each CTA's own rows).
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// A tiled load whose bytes are counted on a barrier of either CTA (a cluster address).
__device__ __forceinline__ void pair_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int x, int row, int chunk, int head) {
  asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%3, %4, %5, %6}], [%2];"
               :: "r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(row), "r"(chunk), "r"(head) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
backward_pair_kernel(const __grid_constant__ PassMaps maps, const __grid_constant__ BackwardParams p, const BackwardWs L) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t rank = ptx::cluster_ctarank();
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  BackwardPlan* plan = reinterpret_cast<BackwardPlan*>(p.ws + L.plan);
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  auto LEAD = [&](int i) { return ptx::mapa(BAR(i), 0); };   // rank 0's barrier, from either rank
  constexpr uint32_t kDp = kAcc2;              // dP is in the place of the key pass's second accumulator
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i) {
      int n = 1;                                       // copies, MMA commits
      if (i >= SREAD && i <= ACCFREE) n = 2 * kWarps;  // one arrival a warp of both ranks
      if (i == C1DFULL || i == C1DFULL + 1) n = 2;     // one arrival a rank
      if (i == DRAIN) n = 2;                           // both issuing warps
      // (roles that walk the items: R and the C copies, on rank 0 the two that issue)
      if (i >= IEMPTY && i < IEMPTY + kItemSlots) n = kWarps + 3 + (rank == 0 ? 2 : 0);
      ptx::mbar_init(BAR(i), n);
    }
    ptx::fence_barrier_init();
  }
  if (warp == 2) {
    ptx::pair_tmem_alloc(sbase + kOffTmem, 512);
    ptx::pair_tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::cluster_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem), 0);
  begin_pass<false>(p);
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  const int causal = p.causal;

  struct Walk { int slot = 0; uint32_t phase = 0; };
  // The next item of this role's walk: its tile and first head, false when there is none.
  auto next_warp = [&](Walk& w, Tile& t, int& head) {
    if (!wait_short_warp(BAR(IFULL + w.slot), w.phase, hdr)) return false;
    read_item(smem + kOffItems + kItemBytes * w.slot, t, head);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(IEMPTY + w.slot));
    if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
    return head >= 0;
  };

  // A role's walk over the steps of all items: f(tile, head, step of the item, number
  // of the step so far) is false when a wait gave up.  Returns the number of steps.
  auto walk_steps = [&](bool& ok, auto f) {
    Walk w;
    Tile t;
    int head;
    uint32_t n = 0;
    while (ok && next_warp(w, t, head))
      for (int i = 0; i < t.steps && ok; ++i) {
        ok = f(t, head, i, n);
        if (ok) ++n;
      }
    return n;
  };
  // Waits at the end of a role that loads: no copy may land after the CTA has left, nor
  // any arrival; rank 0's commits arrive in both ranks, and that it has seen its own
  // says nothing about the other's.  (After a wait that gave up the pause at the end
  // covers what is not waited for here.)
  auto settle = [&](bool ok, uint32_t n, int full, int empty) {
    if (!ok) return;
#pragma unroll 1
    for (uint32_t s = 0; s < 2 && s < n; ++s) {
      const uint32_t ph = ((n + 1 - s) / 2 - 1) & 1u;
      if (rank == 0) wait_drain(BAR(full + static_cast<int>(s)), ph, hdr);
      wait_short<true>(BAR(empty + static_cast<int>(s)), ph, hdr);
    }
  };
  auto col_of = [&](const Tile& t, int i) { return t.c0 + (t.first + i) * kTile; };
  if (smem_ok && warp == 0) {
    // ------------------------------------------------------------ items, and the loads of R1 and R2
    regs_issue();
    if (elect_one()) {
      const Tile* tiles = reinterpret_cast<const Tile*>(p.ws + L.tiles[1]);
      const Schedule sched(plan, 1, kHeads, stored(plan));
      Walk w;
      uint32_t loads = 0;
      bool ok = true;
      int item = static_cast<int>(ptx::cluster_id_x());
      while (ok) {
        // rank 1 hears of the item from rank 0
        if (rank == 0) {
          ok = wait_short<true>(BAR(ITEMACK + w.slot), w.phase ^ 1u, hdr);
          if (!ok) break;
          ptx::st_async_b32(ptx::mapa(sbase + kOffNext + 4u * w.slot, 1), static_cast<uint32_t>(item),
                            ptx::mapa(BAR(ITEM + w.slot), 1));
        } else {
          ptx::mbar_arrive_expect_tx(BAR(ITEM + w.slot), 4);
          ok = wait_short<true>(BAR(ITEM + w.slot), w.phase, hdr);
          if (!ok) break;
          item = *reinterpret_cast<volatile int*>(smem + kOffNext + 4 * w.slot);
          ptx::mbar_arrive_remote(LEAD(ITEMACK + w.slot));
        }
        Tile t = {};
        int tile, head = -1;
        if (sched.find(item, tile, head)) t = read_tile(tiles + tile);
        ok = wait_short(BAR(IEMPTY + w.slot), w.phase ^ 1u, hdr);
        if (!ok) break;
        write_item(smem + kOffItems + kItemBytes * w.slot, t, head);
        ptx::mbar_arrive(BAR(IFULL + w.slot));
        if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
        if (head < 0) break;
        const int row = t.r0 + kTile * static_cast<int>(rank);
        if (t.steps > 0) {
          ok = wait_short<true>(BAR(R1EMPTY), (loads & 1u) ^ 1u, hdr);
          if (!ok) break;
          if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(R1FULL), 6 * kChunk);
          pair_load_4d(sbase + kOffR1, &maps.r1n, LEAD(R1FULL), 0, row, 0, head);
          pair_load_4d(sbase + kOffR1 + 2 * kChunk, &maps.r1r, LEAD(R1FULL), 0, row, 0, head);
          ok = wait_short<true>(BAR(R2EMPTY), (loads & 1u) ^ 1u, hdr);
          if (!ok) break;
          if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(R2FULL), 4 * kChunk);
          pair_load_4d(sbase + kOffR2, &maps.r2, LEAD(R2FULL), 0, row, 0, head);
          ++loads;
        }
        // claimed when the item's rows are on their way: its steps are still to come
        if (rank == 0) item = atomicAdd(&plan->next[1], 1);
      }
      if (ok && loads > 0) {
        if (rank == 0) {
          wait_drain(BAR(R1FULL), (loads - 1) & 1u, hdr);
          wait_drain(BAR(R2FULL), (loads - 1) & 1u, hdr);
        }
        wait_short<true>(BAR(R1EMPTY), (loads - 1) & 1u, hdr);
        wait_short<true>(BAR(R2EMPTY), (loads - 1) & 1u, hdr);
        if (rank == 1) wait_short<true>(BAR(DRAIN), 0u, hdr);   // the last commits
      }
    }
    __syncwarp();
  } else if (smem_ok && warp == 3) {
    // ------------------------------------------------------------ loads of K, first form
    // (Each form has a warp of its own: a copy costs its thread 160 cycles to issue, and
    // one thread that waited for four forms' buffers in turn held up the others.)
    regs_issue();
    bool ok = true;
    const uint32_t n = walk_steps(ok, [&](const Tile& t, int head, int i, uint32_t n) {
      const uint32_t buf = n & 1u;
      if (!wait_short_warp<true>(BAR(C1SEMPTY + buf), ((n >> 1) & 1u) ^ 1u, hdr)) return false;
      if (elect_one()) {
        const int col = col_of(t, i) + 64 * static_cast<int>(rank);
        if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(C1SFULL + buf), 6 * kHalf);
        pair_load_4d(sbase + kOffC1S + buf * 3 * kHalf, &maps.c1n, LEAD(C1SFULL + buf), 0, col, 0, head);
        pair_load_4d(sbase + kOffC1S + (buf * 3 + 2) * kHalf, &maps.c1r, LEAD(C1SFULL + buf), 0, col, 0, 0);
      }
      __syncwarp();
      return true;
    });
    settle(ok, n, C1SFULL, C1SEMPTY);
  } else if (smem_ok && warp == 4) {
    // ------------------------------------------------------------ loads of K, second form
    // Counted on rank 0's barrier, or where keys past the sequence's end have to be
    // cleared first (they may be another sequence's, and hold NaN; dS = 0 there), on this
    // rank's, and then told to rank 0.
    regs_issue();
    bool ok = true;
    uint32_t tails = 0;
    const uint32_t n = walk_steps(ok, [&](const Tile& t, int head, int i, uint32_t n) {
      const uint32_t buf = n & 1u, at = kOffC1D + buf * 2 * kChunk;
      const int valid = t.nc - (t.first + i) * kTile, full = C1DFULL + static_cast<int>(buf);
      if (!wait_short_warp<true>(BAR(C1DEMPTY + buf), ((n >> 1) & 1u) ^ 1u, hdr)) return false;
      if (elect_one()) {
        const bool tail = valid < kTile;
        const uint32_t bar = tail ? ptx::mapa(BAR(TAIL), rank) : LEAD(full);
        ptx::mbar_arrive_expect_tx_remote(bar, 2 * kChunk);
        pair_load_4d(sbase + at, &maps.c1n_d, bar, 0, col_of(t, i), static_cast<int>(rank), head);
        // RoPE columns 32 rank and up: the first half of the chunk is used
        pair_load_4d(sbase + at + kChunk, &maps.c1r_d, bar, 32 * static_cast<int>(rank), col_of(t, i), 0, 0);
      }
      __syncwarp();
      if (valid >= kTile) return true;
      if (!wait_short_warp<true>(BAR(TAIL), tails & 1u, hdr)) return false;
      ++tails;
#pragma unroll 1
      for (uint32_t c = 0; c < 2; ++c) {
        uint4* dst = reinterpret_cast<uint4*>(smem + at + c * kChunk);
        for (int e = valid * 8 + lane; e < kTile * 8; e += 32) dst[e] = make_uint4(0, 0, 0, 0);
      }
      ptx::fence_proxy_async_cta();
      __syncwarp();
      if (elect_one()) ptx::arrive_leader(LEAD(full));
      return true;
    });
    settle(ok, n, C1DFULL, C1DEMPTY);
  } else if (smem_ok && warp == 5) {
    // ------------------------------------------------------------ loads of V
    regs_issue();
    bool ok = true;
    const uint32_t n = walk_steps(ok, [&](const Tile& t, int head, int i, uint32_t n) {
      const uint32_t buf = n & 1u;
      if (!wait_short_warp<true>(BAR(C2EMPTY + buf), ((n >> 1) & 1u) ^ 1u, hdr)) return false;
      if (elect_one()) {
        if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(C2FULL + buf), 4 * kHalf);
        pair_load_4d(sbase + kOffC2 + buf * 2 * kHalf, &maps.c2, LEAD(C2FULL + buf), 0,
                     col_of(t, i) + 64 * static_cast<int>(rank), 0, head);
      }
      __syncwarp();
      return true;
    });
    settle(ok, n, C2FULL, C2EMPTY);
  } else if (smem_ok && warp == 1 && rank == 0) {
    regs_issue();
    // ------------------------------------------------------------ S = R1 C1^T, dP = R2 C2^T
    Walk w;
    Tile t;
    int head;
    const uint64_t r1 = ptx::sdesc_sw128(sbase + kOffR1, 16, 1024), r2 = ptx::sdesc_sw128(sbase + kOffR2, 16, 1024);
    const uint64_t c1 = ptx::sdesc_sw128(sbase + kOffC1S, 16, 1024), c2 = ptx::sdesc_sw128(sbase + kOffC2, 16, 1024);
    constexpr uint64_t kChunkD = kChunk >> 4, kHalfD = kHalf >> 4;
    uint32_t n = 0, loads = 0;
    bool ok = true;
#ifdef MLA_TEST_STALL_WAIT
    // Test builds only: a wait on a barrier that nothing arrives on before the end
    // of the kernel, so that its limit runs out and every role leaves.
    ok = wait_short_warp<true>(BAR(DRAIN), 0u, hdr);
#endif
    while (ok && next_warp(w, t, head)) {
      const int steps = __shfl_sync(0xffffffffu, t.steps, 0);
      for (int i = 0; i < steps && ok; ++i, ++n) {
        const uint32_t buf = n & 1u;
        if (i == 0) ok = wait_short_warp<true>(BAR(R1FULL), loads & 1u, hdr);
        if (ok) ok = wait_short_warp<true>(BAR(C1SFULL + buf), (n >> 1) & 1u, hdr);
        // S's place: the last one has been read
        if (ok && n > 0) ok = wait_short_warp<true>(BAR(SREAD), (n - 1) & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::pair_mma_ss(tmem + kX, r1 + c * kChunkD + 2u * k, c1 + (3u * buf + c) * kHalfD + 2u * k, kIdescS,
                               (c > 0 || k > 0) ? 1u : 0u);
          ptx::pair_commit(BAR(SFULL));
          ptx::pair_commit(BAR(C1SEMPTY + buf));
          if (i == steps - 1) ptx::pair_commit(BAR(R1EMPTY));
        }
        __syncwarp();
        if (i == 0) ok = wait_short_warp<true>(BAR(R2FULL), loads & 1u, hdr);
        if (ok) ok = wait_short_warp<true>(BAR(C2FULL + buf), (n >> 1) & 1u, hdr);
        if (ok && n > 0) ok = wait_short_warp<true>(BAR(DPREAD), (n - 1) & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::pair_mma_ss(tmem + kDp, r2 + c * kChunkD + 2u * k, c2 + (2u * buf + c) * kHalfD + 2u * k, kIdescS,
                               (c > 0 || k > 0) ? 1u : 0u);
          ptx::pair_commit(BAR(DPFULL));
          ptx::pair_commit(BAR(C2EMPTY + buf));
          if (i == steps - 1) ptx::pair_commit(BAR(R2EMPTY));
        }
        __syncwarp();
      }
      if (steps > 0) ++loads;
    }
    // every MMA completes before the pair may leave (the commits to rank 1 are
    // waited for there, by its loader)
    if (n > 0 && elect_one()) {   // the lane that issued them
      ptx::pair_commit(BAR(DRAIN));
      if (ok) wait_drain(BAR(DRAIN), 0u, hdr);
    }
    __syncwarp();
  } else if (smem_ok && warp == 2 && rank == 0) {
    regs_issue();
    // ------------------------------------------------------------ dq += dS K
    Walk w;
    Tile t;
    int head;
    // along the other axis: 64-value chunks kChunk apart, 8-row groups 1 KiB
    const uint64_t c1 = ptx::sdesc_sw128(sbase + kOffC1D, kChunk, 1024);
    uint32_t n = 0, heads = 0;               // steps, and heads with steps, so far
    bool ok = true;
    while (ok && next_warp(w, t, head)) {
      const int steps = __shfl_sync(0xffffffffu, t.steps, 0);
      for (int i = 0; i < steps && ok; ++i, ++n) {
        const uint32_t buf = n & 1u;
        // the accumulator has been read
        if (i == 0) ok = wait_short_warp<true>(BAR(ACCFREE), (heads & 1u) ^ 1u, hdr);
        if (ok) ok = wait_short_warp<true>(BAR(C1DFULL + buf), (n >> 1) & 1u, hdr);
        if (ok) ok = wait_short_warp<true>(BAR(DSREADY), n & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        if (elect_one()) {
          const uint64_t b = c1 + buf * (2 * kChunk >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            pair_mma_ts(tmem + kAcc1, tmem + kY + 8u * k, b + 128u * k, kIdesc192, (i > 0 || k > 0) ? 1u : 0u);
          ptx::pair_commit(BAR(DSDONE));
          ptx::pair_commit(BAR(C1DEMPTY + buf));
        }
        __syncwarp();
      }
      if (steps > 0) ++heads;
    }
    if (n > 0 && elect_one()) {
      ptx::pair_commit(BAR(DRAIN));
      if (ok) wait_drain(BAR(DRAIN), 0u, hdr);
    }
    __syncwarp();
  } else if (smem_ok && warp < kHelpers) {
    regs_issue();   // (idle: a register split is the whole warpgroup's)
  } else if (smem_ok) {
    // ------------------------------------------------------------ dS (thread = a quarter row), results
    regs_compute();
    const int quarter = (warp - kHelpers) >> 2, rl = (warp & 3) * 32 + lane, r = kTile * static_cast<int>(rank) + rl;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t x_addr = tmem + lane_base + kX + 32u * quarter, dp_addr = tmem + lane_base + kDp + 32u * quarter;
    const uint32_t y_addr = tmem + lane_base + kY + 16u * quarter, acc1 = tmem + lane_base + kAcc1 + 96u * (quarter >> 1) + 32u * (quarter & 1),
                   acc1r = tmem + lane_base + kAcc1 + 96u * (quarter >> 1) + 64u + 16u * (quarter & 1);
    const float c = p.scale * kLog2e;
    Walk w;
    Tile t;
    int head;
    uint32_t n = 0;
    bool ok = true;
    auto arrive = [&](int bar) {
      ptx::tc_fence_before();
      __syncwarp();
      if (elect_one()) ptx::arrive_leader(LEAD(bar));
    };
    while (ok && next_warp(w, t, head)) {
      const size_t row = static_cast<size_t>(t.r0) + r;
      const bool mine = r < t.rows;
      float row_lse = 0.f, row_delta = 0.f;
      if (mine) {
        const float* st = reinterpret_cast<const float*>(p.ws + L.stats) +
                          (static_cast<size_t>(t.stat + static_cast<int>(rank)) * kHeads + head) * 2 * kTile;
        row_lse = __ldcg(st + rl);
        row_delta = __ldcg(st + kTile + rl);
      }
      for (int i = 0; i < t.steps; ++i, ++n) {
        // columns below hi of this thread's 32 are seen
        const int at = (t.first + i) * kTile + kCols * quarter;
        const int hi = causal ? min(t.nc - at, t.lim + r - at) : t.nc - at;
        const bool all = __all_sync(0xffffffffu, hi >= kCols);
        ok = wait_short_warp(BAR(SFULL), n & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[kCols], d[kCols], pk[kCols / 2];
        ptx::tmem_ld32(x_addr, s);
        ptx::tmem_wait_ld();
        arrive(SREAD);
        probabilities<false>(s, nullptr, row_lse, c, all, 0, hi);
        ok = wait_short_warp(BAR(DPFULL), n & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        ptx::tmem_ld32(dp_addr, d);
        ptx::tmem_wait_ld();
        arrive(DPREAD);
        gradients<false>(s, d, nullptr, row_delta, all, 0, hi, pk);
        // the last step's dS has been read
        if (n > 0) ok = wait_short_warp(BAR(DSDONE), (n - 1) & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        tmem_st16(y_addr, pk);
        ptx::tmem_wait_st();
        arrive(DSREADY);
      }
      if (!ok) break;
      uint32_t nope[16], rope[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) nope[e] = rope[e] = 0;
      if (t.steps > 0) {
        ok = wait_short_warp(BAR(DSDONE), (n - 1) & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t a[32];
        ptx::tmem_ld32(acc1, a);
        ptx::tmem_ld16(acc1r, rope);
        ptx::tmem_wait_ld();
        to_bf16<16>(a, p.scale, nope);
        to_bf16<8>(rope, p.scale, rope);
        arrive(ACCFREE);
      }
      if (mine) store_results<false>(p, L, row, head, 0, quarter, true, nope, nullptr, rope);
    }
  }
  // ------------------------------------------------------------ teardown
  // after a wait gave up, loads may be in flight uncounted: give them time to land
  if (read_status(&hdr->abort_flag) != 0) spin_ns(20000);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::pair_tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_backward_pairs(const PassMaps& maps, const BackwardParams& p, const BackwardWs& L, int pairs,
                                  cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = allow_smem(backward_pair_kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(backward_pair_kernel, dim3(2 * pairs), dim3(kThreads), kSmem, stream, maps, p, L);
}

}  // namespace mla
