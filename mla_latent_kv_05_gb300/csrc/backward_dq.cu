// dq of the backward pass (backward.cu) from the dS tiles that the key pass has stored:
// dq = scale sum_j dS_j K_j, one product over 192 values instead of three.
//
// An item is a query tile of 128 rows and a head; dq stays in tensor memory (two of
// them, so that the next item's products run while one is stored).  The tiles of 128
// keys come in halves of 64: of dS 16 KiB, laid out by the key pass as the MMAs read them
// (A, MN-major: the rows of a tile are keys), in one bulk copy, and K 16 + 8 KiB; five
// halves are held.  Warp 0: items and dS; warp 1 issues the MMAs; warp 2 loads K; warps
// 4..19 write the results (thread = a quarter row).
//
// Bound: reading dS, 32 KiB for 768 cycles of MMAs: 152 SMs would take 12 TB/s.  4096
// causal tokens, 2.2 GB: 393 us, 5.6 TB/s (325 at the copy's rate).
#include "backward_tile.cuh"

namespace mla {

namespace {

using namespace bwd;

constexpr int kHelpers = 4;
constexpr int kThreads = 32 * (kHelpers + kWarps);
constexpr int kHalfRows = 64;                               // keys of a stage
constexpr uint32_t kPart = kHalfRows * 128u;                // 8 KiB: 64 rows x 64 values
constexpr uint32_t kStage = 5 * kPart;                      // dS 2, K 3
constexpr int kStages = 5, kItemSlots = 2;
constexpr uint32_t kOffBar = kStages * kStage;
enum Bar {
  FULL, EMPTY = FULL + kStages, ACCFULL = EMPTY + kStages, ACCFREE = ACCFULL + 2, IFULL = ACCFREE + 2, IEMPTY = IFULL + kItemSlots,
  DRAIN = IEMPTY + kItemSlots, NBAR
};
constexpr uint32_t kOffTmem = kOffBar + 8 * NBAR;
constexpr uint32_t kOffQuit = kOffTmem + 4;
constexpr uint32_t kOffItems = (kOffQuit + 4 + 15) & ~15u;
constexpr uint32_t kSmem = kOffItems + kItemBytes * kItemSlots;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr uint32_t kAccCols = 256;                          // from one accumulator to the other
constexpr uint32_t kIdesc = ptx::idesc_bf16(128, 192, 1, 1);   // both MN-major

// As sdesc_sw128 without swizzle.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  return ptx::sdesc_sw128(saddr, lbo_bytes, sbo_bytes) & ~(7ull << 61);
}

__global__ void __launch_bounds__(kThreads, 1)
backward_dq_kernel(const __grid_constant__ PassMaps maps, const __grid_constant__ BackwardParams p, const BackwardWs L) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  BackwardPlan* plan = reinterpret_cast<BackwardPlan*>(p.ws + L.plan);
  volatile uint32_t* const quit = reinterpret_cast<volatile uint32_t*>(smem + kOffQuit);
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  if (threadIdx.x == 0) {
    *quit = 0;
    for (int i = 0; i < NBAR; ++i) {
      int n = 1;                                           // MMA commits, items
      if (i >= FULL && i < FULL + kStages) n = 2;          // dS and K
      if (i == ACCFREE || i == ACCFREE + 1) n = kWarps;    // one arrival a warp
      if (i >= IEMPTY && i < IEMPTY + kItemSlots) n = kWarps + 2;
      ptx::mbar_init(BAR(i), n);
    }
    ptx::fence_barrier_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc(sbase + kOffTmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem), 0);
  ptx::grid_dep_wait();   // the dS tiles
  ptx::grid_dep_launch();
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);

  struct Walk { int slot = 0; uint32_t phase = 0; };
  // The next item of a warp's walk: its tile and head, false when there is none.
  auto next_warp = [&](Walk& w, Tile& t, int& head) {
    if (!wait_cta_warp(BAR(IFULL + w.slot), w.phase, quit)) return false;
    read_item(smem + kOffItems + kItemBytes * w.slot, t, head);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(IEMPTY + w.slot));
    if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
    return head >= 0;
  };
  // keys of the sequence that the tile's last row sees
  auto keys_of = [&](const Tile& t) { return t.steps == 0 ? 0 : p.causal ? max(0, min(t.nc, t.lim + t.rows - 1)) : t.nc; };
  struct Ring { int at = 0; uint32_t phase = 0; __device__ void next() { if (++at == kStages) { at = 0; phase ^= 1u; } } };

  if (smem_ok && warp == 0) {
    // ------------------------------------------------------------ items, and the loads of dS
    if (elect_one()) {
      const Tile* tiles = reinterpret_cast<const Tile*>(p.ws + L.tiles[1]);
      const int* slots = reinterpret_cast<const int*>(p.ws + L.slots);
      const Schedule sched(plan, 1, kHeads, !stored(plan));
      const uint64_t once = ptx::policy_evict_first();
      Walk w;
      Ring ring;
      bool ok = true;
      int item = static_cast<int>(blockIdx.x);
      while (ok) {
        Tile t = {};
        int tile, head = -1;
        if (sched.find(item, tile, head)) {
          t = read_tile(tiles + tile);
          head = kHeads - 1 - head;                        // the heads stored last are still in L2
        }
        ok = wait_cta(BAR(IEMPTY + w.slot), w.phase ^ 1u, quit);
        if (!ok) break;
        write_item(smem + kOffItems + kItemBytes * w.slot, t, head);
        ptx::mbar_arrive(BAR(IFULL + w.slot));
        if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
        if (head < 0) break;
        const int keys = keys_of(t);
        int next = keys > 0 ? __ldcg(slots + t.slot) : 0;
        for (int k = 0; k < keys && ok; k += kTile) {
          const uint8_t* src = p.ws + L.ds + (static_cast<size_t>(next + t.tile) * kHeads + head) * kDsTile;
          if (k + kTile < keys) next = __ldcg(slots + t.slot + k / kTile + 1);
          for (int h = 0; h < 2 && k + kHalfRows * h < keys; ++h) {
            ok = wait_cta(BAR(EMPTY + ring.at), ring.phase ^ 1u, quit);
            if (!ok) break;
            ptx::mbar_arrive_expect_tx(BAR(FULL + ring.at), 2 * kPart);
            ptx::bulk_load(sbase + ring.at * kStage, src + h * 2 * kPart, 2 * kPart, BAR(FULL + ring.at), once);
            ring.next();
          }
        }
        // claimed when the item's last copies are on their way: its products are still to come
        item = atomicAdd(&plan->next[1], 1);
      }
    }
    __syncwarp();
  } else if (smem_ok && warp == 2) {
    // ------------------------------------------------------------ loads of K
    Walk w;
    Tile t;
    int head;
    Ring ring;
    bool ok = true;
    while (ok && next_warp(w, t, head)) {
      const int keys = __shfl_sync(0xffffffffu, keys_of(t), 0);
      for (int k = 0; k < keys && ok; k += kHalfRows) {
        ok = wait_cta_warp(BAR(EMPTY + ring.at), ring.phase ^ 1u, quit);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t at = sbase + ring.at * kStage + 2 * kPart, bar = BAR(FULL + ring.at);
          ptx::mbar_arrive_expect_tx(bar, 3 * kPart);
          load_4d(at, &maps.c1n, bar, 0, t.c0 + k, 0, head);
          load_4d(at + 2 * kPart, &maps.c1r, bar, 0, t.c0 + k, 0, 0);
        }
        __syncwarp();
        ring.next();
      }
    }
  } else if (smem_ok && warp == 1) {
    // ------------------------------------------------------------ dq += dS K
    Walk w;
    Tile t;
    int head;
    Ring ring;
    // dS: 8 keys x 16 bytes in 128 bytes, 8 keys on 128 bytes on, 8 queries on 1 KiB on (no
    // swizzle); K: chunks of 64 values kPart apart, 8-row groups 1 KiB
    const uint64_t ds = sdesc_plain(sbase, 128, 1024), kk = ptx::sdesc_sw128(sbase + 2 * kPart, kPart, 1024);
    uint32_t heads = 0;                        // items with steps so far
    bool ok = true, issued = false;
#ifdef MLA_TEST_STALL_WAIT
    // Test builds only: a wait on a barrier that nothing arrives on before the end
    // of the kernel, so that its limit runs out and every role leaves.
    ok = wait_cta_warp(BAR(DRAIN), 0u, quit);
#endif
    while (ok && next_warp(w, t, head)) {
      const int keys = __shfl_sync(0xffffffffu, keys_of(t), 0), nc = __shfl_sync(0xffffffffu, t.nc, 0);
      if (keys == 0) continue;
      const uint32_t acc = heads & 1u;
      ok = wait_cta_warp(BAR(ACCFREE + acc), ((heads >> 1) & 1u) ^ 1u, quit);
      for (int k = 0; k < keys && ok; k += kHalfRows) {
        ok = wait_cta_warp(BAR(FULL + ring.at), ring.phase, quit);
        if (!ok) break;
        if (nc - k < kHalfRows) {
          // keys past the sequence's end have dS = 0; make their rows 0 too (they may be
          // another sequence's, and hold NaN)
#pragma unroll 1
          for (uint32_t c = 2; c < 5; ++c) {
            uint4* dst = reinterpret_cast<uint4*>(smem + ring.at * kStage + c * kPart);
            for (int i = (nc - k) * 8 + lane; i < kHalfRows * 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_cta();
          __syncwarp();
        }
        ptx::tc_fence_after();
        issued = true;
        if (elect_one()) {
          const uint64_t off = static_cast<uint64_t>(ring.at) * (kStage >> 4);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            ptx::mma_ss(tmem + acc * kAccCols, ds + off + 16u * e, kk + off + 128u * e, kIdesc, (k > 0 || e > 0) ? 1u : 0u);
          ptx::mma_commit(BAR(EMPTY + ring.at));
          if (k + kHalfRows >= keys) ptx::mma_commit(BAR(ACCFULL + acc));
        }
        __syncwarp();
        ring.next();
      }
      ++heads;
    }
    // every MMA completes before the CTA may leave
    if (issued && elect_one()) {               // the lane that issued them
      ptx::mma_commit(BAR(DRAIN));
      wait_issued(BAR(DRAIN), 0u, quit);
    }
    __syncwarp();
  } else if (smem_ok && warp >= kHelpers) {
    // ------------------------------------------------------------ results (thread = a quarter row)
    const int quarter = (warp - kHelpers) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Walk w;
    Tile t;
    int head;
    uint32_t heads = 0;
    while (next_warp(w, t, head)) {
      uint32_t nope[16], rope[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) nope[e] = rope[e] = 0;
      if (keys_of(t) > 0) {
        const uint32_t acc = heads & 1u;
        if (!wait_cta_warp(BAR(ACCFULL + acc), (heads >> 1) & 1u, quit)) break;
        ptx::tc_fence_after();
        uint32_t a[32];
        ptx::tmem_ld32(tmem + lane_base + acc * kAccCols + 32u * quarter, a);
        ptx::tmem_ld16(tmem + lane_base + acc * kAccCols + 128u + 16u * quarter, rope);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(BAR(ACCFREE + acc));
        to_bf16<16>(a, p.scale, nope);
        to_bf16<8>(rope, p.scale, rope);
        ++heads;
      }
      if (r < t.rows) store_results<false>(p, L, static_cast<size_t>(t.r0) + r, head, 0, quarter, true, nope, nullptr, rope);
    }
  }
  // ------------------------------------------------------------ teardown
  // after a wait gave up, copies may be in flight uncounted: give them time to land
  if (*quit != 0) spin_ns(20000);
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *quit != 0) set_status(&hdr->status, MLA_STATUS_TIMEOUT);
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_backward_dq(PFN_cuTensorMapEncodeTiled_v12000 encode, const BackwardParams& p, const BackwardWs& L, int ctas,
                               cudaStream_t stream) {
  PassMaps maps = {};
  if (!encode_chunks(encode, &maps.c1n, p.k_nope, 2, kHeads, p.nk, p.kn_t, p.kn_h, kHalfRows, 2) ||
      !encode_chunks(encode, &maps.c1r, p.k_rope, 1, 1, p.nk, p.kr_t, 64, kHalfRows, 1))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = allow_smem(backward_dq_kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(backward_dq_kernel, dim3(ctas), dim3(kThreads), kSmem, stream, maps, p, L);
}

}  // namespace mla
