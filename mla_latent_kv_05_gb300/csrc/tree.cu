// Tree decode over bf16 latent rows: every drafted node of a sequence attends
// to its context and its path, all nodes over the same cached rows.
//
// For a row (sequence b, node i), s = scale Q[128 x 576] . K^T over the tokens
// the node sees, P = softmax(s), O[128 x 512] = P . V with V the first 512
// columns of the same rows; out = O / l, lse = m + ln l.
//
// Bound: 2 * 128 * (576 + 512) operations per (node, token), with the rows of
// a sequence read from L2 once per node, so the tensor cores bound it.
//
// One row runs on a pair of CTAs with cta_group::2 MMAs of M = 128: each CTA
// holds 64 of the heads.  O of 64 heads takes 256 of an SM's 512 tensor memory
// columns, which leaves room for two S buffers, so scores, softmax and P.V of
// a head stay in one SM.  (The decode kernel gives one SM of a pair the scores
// and the other O of all 128 heads, and sends P between them: with the rows in
// L2 that transfer took half of its time, about 40 cycles a token for a row,
// where these MMAs need 17.)  An M = 128 pair MMA runs at the full rate of two
// SMs: 32 cycles for N = 128, 64 for N = 256, K = 16.
//
// Tiles of 128 tokens (two pages), 64 each for the pair's ranks:
//   S[128 heads x 128 tokens]: B is one page of K from each CTA, all 576
//       values of it (three groups of three 64-value chunks, 24 KiB each, so
//       that a group is reloaded as soon as its MMAs are done);
//   O += P V: two MMAs of N = 256 per 16 tokens; a CTA holds the half of the
//       latent columns [256 rank, +256) of all 128 tokens (32 KiB a page),
//       read as an MN-major operand, and a page's MMAs start on its own P and V.
// S and O land with a CTA's 64 heads on tensor memory lanes 0..63 for the first
// half of the columns and on lanes 64..127 for the second.  Four threads share
// a head: 32 tokens of S and 128 columns of O each.
// Shared memory: Q 72 KiB, K 72, V 64, P 16.  K and V are single-buffered by
// group and page: a group's next load has the rest of the tile's MMAs to arrive.
//
// Warp 0 of each rank loads Q and K, warp 3 V (V of a tile is free after K of
// the next but one: in one thread the later loads waited for it, 2300 cycles a
// tile), warp 1 of rank 0 issues the MMAs (S of tile j + 1 before P.V of tile j),
// warps 4..11 of each rank are softmax and output.  Rows split over several
// pairs leave fp32 partials for the merge: a row is cut into two parts or three
// here, so a bf16 rounding of each would be as large as the result's own.
// Every wait is bounded, as in the decode kernel.
//
// Rows are planned node by node, not sequence by sequence: pairs then work on
// different nodes of one sequence at a time and find its rows in L2 (64 x 4
// nodes over 4096 tokens: 247 us by sequence, 199 by node).
//
// Measured, whole call: 8 x 61 nodes over 4096 tokens 332 us (1690 TFLOP/s; the
// decode kernel's form of it 554), 16 x up to 16 over up to 8192 120 us (1180),
// 64 x 16 over 4096 720 us (1620), 8 nodes over 1000 18.7 us (four kernels of 2 to
// 9 us).  Scores that rise, so that every head's reference moves in every tile,
// cost a tenth: 8 x 61 369 us, 16 x 16 over 4096 193 and 207, 8 nodes 20.2.  A tile
// takes about 2300 cycles, 2184 of them MMAs; a segment's output another 4500,
// while the next segment's first scores wait.
#include <cuda.h>
#include <cuda_bf16.h>

#include "tree.cuh"
#include "waits.cuh"
#include "walk.cuh"

namespace mla {

namespace {

using dk::Segment;
using dk::SegWalker;
using dk::tree_bits;

constexpr int kThreads = 384;
constexpr uint32_t kChunk = 64u * 128u;                 // 8 KiB: 64 rows x 64 values
constexpr uint32_t kKGroupBytes = 3 * kChunk;           // 24 KiB
constexpr uint32_t kVPage = 4 * kChunk;                 // 32 KiB: 64 tokens x 256 values
constexpr uint32_t kOffK = 9 * kChunk;                  // after Q
constexpr uint32_t kOffV = kOffK + 9 * kChunk;
constexpr uint32_t kOffP = kOffV + 2 * kVPage;          // 64 heads x 128 tokens
constexpr uint32_t kOffX = kOffP + 2 * kChunk;          // fp32 exchange [4 quarters][64 heads]
constexpr uint32_t kOffBar = kOffX + 4 * 64 * 4;
enum Bar {
  QFULL = 0, QEMPTY, KFULL, KEMPTY = KFULL + 3, VFULL = KEMPTY + 3, VEMPTY = VFULL + 2, SFULL = VEMPTY + 2,
  SEMPTY = SFULL + 2, PREADY = SEMPTY + 2, PVDONE = PREADY + 2, OFREE, DRAIN, NBAR
};
constexpr uint32_t kOffTmem = kOffBar + 8 * NBAR;
constexpr uint32_t kSmem = kOffTmem + 16;
static_assert(kSmem <= 232448, "shared memory budget");

constexpr uint32_t kOCol = 0, kSCol = 256;              // O: two blocks of 128 columns; S: two buffers of 64
constexpr uint32_t kIdescS = ptx::idesc_bf16(128, 128, 0, 0);
constexpr uint32_t kIdescPV = ptx::idesc_bf16(128, 256, 0, 1);
constexpr float kLazy = 12.0f;                          // log2 units: P <= 2^12
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float max32(const uint32_t* s) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
  for (int e = 8; e < 32; e += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max3(m[i], __uint_as_float(s[e + 2 * i]), __uint_as_float(s[e + 2 * i + 1]));
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// Named barrier of the four warps that share heads, with an OR over their threads.
__device__ __forceinline__ bool any_of_group(int id, bool v) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\tbar.red.or.pred p, %1, 128, q;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(r) : "r"(id), "r"(static_cast<uint32_t>(v)) : "memory");
  return r != 0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
tree_kernel(const __grid_constant__ TreeMaps maps, const DecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t rank = ptx::cluster_ctarank();
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  auto LEAD = [&](int i) { return ptx::mapa(BAR(i), 0); };   // rank 0's barrier, from either rank
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i) {
      // softmax warps of both ranks arrive on rank 0's SEMPTY, PREADY and OFREE; the others take one arrival
      const bool all = i == SEMPTY || i == SEMPTY + 1 || i == OFREE, page = i == PREADY || i == PREADY + 1;
      ptx::mbar_init(BAR(i), all ? 16 : page ? 8 : 1);
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
  // everything above overlaps the planner, whose plan is read from here on
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();   // the merge may begin launching (it waits for this grid)
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  const int pl = static_cast<int>(ptx::cluster_id_x());
  const int* lens = reinterpret_cast<const int*>(p.ws + p.L.lens);
  const int* tile_start = reinterpret_cast<const int*>(p.ws + p.L.tile_start);
  const int* pair_lo = reinterpret_cast<const int*>(p.ws + p.L.pair_lo);
  const int lo = pair_lo[pl], hi = pair_lo[pl + 1];
  const int b0 = reinterpret_cast<const int*>(p.ws + p.L.pair_b0)[pl];

  // rows are planned node by node (see api.cu); queries and results lie by sequence
  auto out_row = [&](int row) { return row % p.tree_seqs * p.tree_nodes + row / p.tree_seqs; };
  // a tile's page (row of its first token): one past the segment, or a bad one, is
  // read outside the cache, which fills zeros
  auto page_row = [&](int b, int t, int t1) {
    const size_t at = static_cast<size_t>(b) * p.max_pages + t;
    const int page = t >= t1 ? -1 : p.block_table ? __ldg(p.block_table + at) : static_cast<int>(at);
    if (t < t1 && (page < 0 || page >= p.num_pages)) set_status(&hdr->status, MLA_STATUS_BAD_PAGE);
    return (page < 0 || page >= p.num_pages ? p.num_pages : page) * kPage;
  };
  if (smem_ok && warp == 0) {
    // ------------------------------------------------------------ loads of Q and K
    if (elect_one()) {
      const uint64_t pol = ptx::policy_evict_normal();
      SegWalker w; w.init(tile_start, p.batch, lo, hi, b0);
      Segment sg;
      uint32_t nq = 0, nt = 0;               // segments and tiles loaded so far
      bool ok = true;
      while (ok && w.next(sg)) {
        ok = wait_short<true>(BAR(QEMPTY), (nq & 1u) ^ 1u, hdr);
        if (!ok) break;
        if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(QFULL), 2 * 9 * kChunk);
        const int head = out_row(sg.b) * kHeads + static_cast<int>(rank) * 64;
        ptx::pair_load_3d(sbase, &maps.q, LEAD(QFULL), 0, head, 0, pol);
        ptx::pair_load_3d(sbase + 8 * kChunk, &maps.qr, LEAD(QFULL), 0, head, 0, pol);
        ++nq;
        const int seq = sg.b % p.tree_seqs;
        for (int t = sg.t0; t < sg.t1 && ok; t += 2) {
          const int row = page_row(seq, t + static_cast<int>(rank), sg.t1);
#pragma unroll 1
          for (int g = 0; g < 3 && ok; ++g) {
            ok = wait_short<true>(BAR(KEMPTY + g), (nt & 1u) ^ 1u, hdr);
            if (!ok) break;
            if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(KFULL + g), 2 * kKGroupBytes);
            ptx::pair_load_3d(sbase + kOffK + g * kKGroupBytes, &maps.k, LEAD(KFULL + g), 0, row, 3 * g, pol);
          }
          if (ok) ++nt;
        }
      }
      // no copy may land after the CTA has left (after a wait that gave up, the
      // pause at the end covers what is not waited for here)
      if (ok && rank == 0) {
        if (nq > 0) wait_drain(BAR(QFULL), (nq - 1) & 1u, hdr);
#pragma unroll 1
        for (int g = 0; g < 3; ++g)
          if (nt > 0) wait_drain(BAR(KFULL + g), (nt - 1) & 1u, hdr);
      }
      // nor any arrival: rank 0's commits arrive in both ranks, and that it has seen
      // its own says nothing about the other's
      if (ok && nt > 0) {
#pragma unroll 1
        for (int g = 0; g < 3; ++g) wait_short<true>(BAR(KEMPTY + g), (nt - 1) & 1u, hdr);
        wait_short<true>(BAR(QEMPTY), (nq - 1) & 1u, hdr);
      }
    }
  } else if (smem_ok && warp == 3) {
    // ------------------------------------------------------------ loads of V
    if (elect_one()) {
      const uint64_t pol = ptx::policy_evict_normal();
      SegWalker w; w.init(tile_start, p.batch, lo, hi, b0);
      Segment sg;
      uint32_t nt = 0;
      bool ok = true;
      while (ok && w.next(sg)) {
        const int seq = sg.b % p.tree_seqs;
        for (int t = sg.t0; t < sg.t1 && ok; t += 2) {
#pragma unroll 1
          for (int a = 0; a < 2 && ok; ++a) {
            const int row = page_row(seq, t + a, sg.t1);
            ok = wait_short<true>(BAR(VEMPTY + a), (nt & 1u) ^ 1u, hdr);
            if (!ok) break;
            ptx::mbar_arrive_expect_tx(BAR(VFULL + a), kVPage);
            ptx::tma_load_3d(sbase + kOffV + a * kVPage, &maps.v, BAR(VFULL + a), 0, row, 4 * static_cast<int>(rank), pol);
          }
          if (ok) ++nt;
        }
      }
      // no copy or arrival may land after the CTA has left (as for Q and K); the
      // commit to DRAIN is the last one
      if (ok && nt > 0) {
#pragma unroll 1
        for (int a = 0; a < 2; ++a) {
          wait_drain(BAR(VFULL + a), (nt - 1) & 1u, hdr);
          wait_short<true>(BAR(VEMPTY + a), (nt - 1) & 1u, hdr);
        }
        if (rank == 1) wait_short<true>(BAR(DRAIN), 0u, hdr);   // (here, not from the start: the limit is for a wait)
      }
    }
  } else if (smem_ok && warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint64_t desc_q = ptx::sdesc_sw128(sbase, 16, 1024), desc_k = ptx::sdesc_sw128(sbase + kOffK, 16, 1024);
    const uint64_t desc_p = ptx::sdesc_sw128(sbase + kOffP, 16, 1024);
    const uint64_t desc_v = ptx::sdesc_sw128(sbase + kOffV, kChunk, 1024);
    constexpr uint64_t kChunkD = kChunk >> 4;
    SegWalker w; w.init(tile_start, p.batch, lo, hi, b0);
    Segment sg;
    uint32_t n_s = 0, n_p = 0, n_seg = 0;    // S tiles, P.V tiles and segments begun so far
    bool ok = true;
#ifdef MLA_TEST_STALL_WAIT
    // Test builds only: a wait on a barrier that nothing arrives on before the end
    // of the kernel, so that its limit runs out and every role leaves through the
    // abort path.
    ok = wait_short_warp<true>(BAR(DRAIN), 0u, hdr);
#endif
    auto score = [&](bool last) {
      // S buffer n_s & 1 is free once its last scores were read
      ok = wait_short_warp<true>(BAR(SEMPTY + (n_s & 1u)), ((n_s >> 1) & 1u) ^ 1u, hdr);
#pragma unroll 1
      for (int g = 0; g < 3 && ok; ++g) {
        ok = wait_short_warp<true>(BAR(KFULL + g), n_s & 1u, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            // V4.1 rows: chunk 7 (latent dims 448..511) is left out, whatever the query holds there
            if (p.skip_chunk7 && g == 2 && c == 1) continue;
            const uint64_t o = static_cast<uint64_t>(3 * g + c) * kChunkD;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::pair_mma_ss(tmem + kSCol + 64u * (n_s & 1u), desc_q + o + 2u * k, desc_k + o + 2u * k, kIdescS,
                               (g > 0 || c > 0 || k > 0) ? 1u : 0u);
          }
          ptx::pair_commit(BAR(KEMPTY + g));
          if (g == 2) {
            ptx::pair_commit(BAR(SFULL + (n_s & 1u)));
            if (last) ptx::pair_commit(BAR(QEMPTY));
          }
        }
        __syncwarp();
      }
      ++n_s;
    };
    while (ok && w.next(sg)) {
      const int tiles = (sg.t1 - sg.t0 + 1) / 2;
      ok = wait_short_warp<true>(BAR(QFULL), n_seg & 1u, hdr);
      if (ok) score(tiles == 1);
      for (int j = 0; j < tiles && ok; ++j) {
        if (j + 1 < tiles) score(j + 2 == tiles);
        // the segment's first P.V overwrites O: the last segment's has been read
        if (ok && j == 0 && n_seg > 0) ok = wait_short_warp<true>(BAR(OFREE), (n_seg - 1) & 1u, hdr);
#pragma unroll 1
        for (int a = 0; a < 2 && ok; ++a) {
          // the page's P, and the V behind it, are in place in both ranks
          ok = wait_short_warp<true>(BAR(PREADY + a), n_p & 1u, hdr);
          if (!ok) break;
          ptx::tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int n = 0; n < 2; ++n)
                ptx::pair_mma_ss(tmem + kOCol + 128u * n, desc_p + a * kChunkD + 2u * k,
                                 desc_v + (4u * a + 2u * n) * kChunkD + 128u * k, kIdescPV, (j > 0 || a > 0 || k > 0) ? 1u : 0u);
            ptx::pair_commit(BAR(VEMPTY + a));
            if (a == 1) ptx::pair_commit(BAR(PVDONE));
          }
          __syncwarp();
        }
        ++n_p;
      }
      ++n_seg;
    }
    // every MMA completes before the pair may leave (the commits to rank 1 are
    // waited for there, by its loaders)
    if (n_s > 0 && elect_one()) {   // the lane that issued them
      ptx::pair_commit(BAR(DRAIN));
      wait_drain(BAR(DRAIN), 0u, hdr);
    }
    __syncwarp();
  } else if (smem_ok && warp >= 4) {
    // ------------------------------------------------------------ softmax and output
    // thread = (head, 32 tokens of the tile): lanes 0..63 hold its first page,
    // 64..127 the second, and a warp of each four takes half a page
    const int wq = warp & 3, hf = wq >> 1, cf = (warp >> 2) - 1;
    const int hl = (wq & 1) * 32 + lane, h = static_cast<int>(rank) * 64 + hl;
    const int group = 1 + (wq & 1);                        // named barrier of the four warps that share heads
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    uint8_t* p_row = smem + kOffP + hf * kChunk + hl * 128;
    const volatile float* shared = reinterpret_cast<const volatile float*>(smem + kOffX) + hl;
    volatile float* own = reinterpret_cast<volatile float*>(smem + kOffX) + hl + 64 * (2 * hf + cf);
    const int* slot_base = reinterpret_cast<const int*>(p.ws + p.L.slot_base);
    const int* n_parts = reinterpret_cast<const int*>(p.ws + p.L.n_parts);
    const int* first_pair = reinterpret_cast<const int*>(p.ws + p.L.first_pair);
    const int* pair_rank = reinterpret_cast<const int*>(p.ws + p.L.pair_rank);
    const uint64_t* tree_seen = reinterpret_cast<const uint64_t*>(p.ws + p.L.tree_seen);
    const float c = p.scale_log2;
    SegWalker w; w.init(tile_start, p.batch, lo, hi, b0);
    Segment sg;
    uint32_t n = 0;                          // tiles so far
    bool ok = true;
    // The warps of a group leave at the same place: what one of them knows alone
    // (a wait that gave up) takes effect only once the others have heard of it.
    while (w.next(sg)) {
      const int row = sg.b, len = lens[row];
      const int ctx = len - 1 - row / p.tree_seqs;         // tokens of the context
      const uint64_t seen = tree_seen[row];
      // where the result goes: read here, so that its latency passes beside the first tile's
      const int parts = n_parts[row];
      const int slot = parts > 1 ? slot_base[row] + pair_rank[pl] - pair_rank[first_pair[row]] : 0;
      float mc = 0.f, m_ref = -INFINITY, l = 0.f;
      bool quit = false;
      for (int t = sg.t0; t < sg.t1; t += 2) {
        if (!wait_short_warp(BAR(SFULL + (n & 1u)), (n >> 1) & 1u, hdr)) ok = false;
        ptx::tc_fence_after();
        uint32_t s[32];
        ptx::tmem_ld32(tmem + lane_base + kSCol + 64u * (n & 1u) + 32u * cf, s);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::arrive_leader(LEAD(SEMPTY + (n & 1u)));
        // this thread's tokens that the node sees (a page past the segment: none)
        const int tok = (t + hf) * kPage + 32 * cf;
        const uint32_t see = t + hf < sg.t1 ? static_cast<uint32_t>(tree_bits(seen, ctx - tok, len - tok)) : 0u;
        if (see != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((see >> e) & 1u)) s[e] = 0xFF800000u;    // -inf
        }
        float mx = max32(s);
        const bool up = !ok || t == sg.t0 || (m_ref == -INFINITY ? mx != -INFINITY : (mx - m_ref) * c > kLazy);
        float alpha = 1.f;
        const bool moving = any_of_group(group, up);
        if (moving) {
          // rare: agree on the heads' maxima and move the references that need it
          *own = mx;
          quit = any_of_group(group, !ok);
          mx = fmaxf(fmaxf(shared[0], shared[64]), fmaxf(shared[128], shared[192]));
          if (m_ref == -INFINITY ? mx != -INFINITY : (mx - m_ref) * c > kLazy) {
            const float nmc = mx * c;
            alpha = m_ref == -INFINITY ? 1.f : fast_exp2(mc - nmc);   // -inf: l = 0 and O = 0 so far
            m_ref = mx;
            mc = nmc;
            l *= alpha;
          }
        }
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                                      make_float2(c, c), make_float2(-mc, -mc));
          const float2 pv = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          if (e & 1) acc1 = __fadd2_rn(acc1, pv);
          else acc0 = __fadd2_rn(acc0, pv);
          const __nv_bfloat162 b = __floats2bfloat162_rn(pv.x, pv.y);
          pk[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        acc0 = __fadd2_rn(acc0, acc1);
        l += acc0.x + acc0.y;
        // the previous P.V has read P (and completed O)
        if (n > 0 && !wait_short_warp(BAR(PVDONE), (n - 1) & 1u, hdr)) ok = false;
        ptx::tc_fence_after();
        if (moving && t != sg.t0) {            // (a segment's first tile finds O empty)
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int q = 4 * cf; q < 4 * cf + 4; ++q) {
              uint32_t o[32];
              ptx::tmem_ld32(tmem + lane_base + kOCol + 32u * q, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              ptx::tmem_st32(tmem + lane_base + kOCol + 32u * q, o);
            }
            ptx::tmem_wait_st();
          }
          // A page's P.V adds to all columns of a head, lanes 0..63 and 64..127,
          // and starts on that page's P, which two of the four warps write (hf).
          // So each of them arrives only when all four have rescaled their lanes:
          // this barrier orders the other page's warps before the arrival below.
          ptx::tc_fence_before();
          any_of_group(group, false);
          ptx::tc_fence_after();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)          // 64 tokens = one 128-byte swizzled row
          *reinterpret_cast<uint4*>(p_row + (((4 * cf + q) ^ (hl & 7)) << 4)) =
              make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
        // V has landed; rows the node does not see get V = 0 (P = 0 alone would
        // turn an infinity or a NaN there into NaN)
        if (!wait_short_warp(BAR(VFULL + hf), n & 1u, hdr)) ok = false;
        if (see != 0xffffffffu) {              // the same for every thread of the warp
          // half of each row by either of the two warps that know of it, two rows at a time
          const int q = 16 * (wq & 1) + (lane & 15);
          uint8_t* dst = smem + kOffV + hf * kVPage + (q >> 3) * kChunk + (32 * cf + (lane >> 4)) * 128 + (q & 7) * 16;
#pragma unroll
          for (int r = 0; r < 32; r += 2)
            if (!((see >> (r + (lane >> 4))) & 1u)) *reinterpret_cast<uint4*>(dst + r * 128) = make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async_cta();
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::arrive_leader(LEAD(PREADY + hf));
        ++n;
        if (quit) break;
      }
      if (!quit && !wait_short_warp(BAR(PVDONE), (n - 1) & 1u, hdr)) ok = false;
      ptx::tc_fence_after();
      any_of_group(group, false);              // the partner has read what an exchange left here
      *own = l;
      if (any_of_group(group, !ok)) break;
      l = (shared[0] + shared[64]) + (shared[128] + shared[192]);
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // a NaN sum stays NaN
      if (hf == 0 && cf == 0) {
        const float lse = l == 0.f ? -INFINITY : (mc + log2f(l)) * kLn2;
        if (parts > 1) reinterpret_cast<float*>(p.ws + p.L.part_lse)[static_cast<size_t>(slot) * kHeads + h] = lse;
        else p.lse[static_cast<size_t>(out_row(row)) * kHeads + h] = lse;
      }
      // this thread's quarter of the latent columns: [256 hf + 128 cf, +128)
      float* part = reinterpret_cast<float*>(p.ws + p.L.part_out) + static_cast<size_t>(slot) * kHeads * kDc +
                    part_piece(2 * static_cast<int>(rank) + (wq & 1), 2 * hf + cf, 0) + 8 * lane;
      __nv_bfloat16* dst = p.out + (static_cast<size_t>(out_row(row)) * kHeads + h) * kDc + 256 * hf + 128 * cf;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        ptx::tmem_ld32(tmem + lane_base + kOCol + 128u * cf + 32u * q, o);
        ptx::tmem_wait_ld();
        if (q == 3) {
          // O is read: the next segment's first P.V may overwrite it
          ptx::tc_fence_before();
          __syncwarp();
          if (elect_one()) ptx::arrive_leader(LEAD(OFREE));
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
        if (parts > 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) ptx::st_global_v8(part + (4 * q + e) * 256, o + 8 * e);
        } else {
          uint32_t b16[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            b16[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          ptx::st_global_v8(dst + 32 * q, b16);
          ptx::st_global_v8(dst + 32 * q + 16, b16 + 8);
        }
      }
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

cudaError_t launch_tree(PFN_cuTensorMapEncodeTiled_v12000 encode, const DecodeParams& p, int n_pairs, bool pdl,
                        cudaStream_t stream) {
  TreeMaps maps;
  auto map = [&](CUtensorMap* m, const void* base, cuuint64_t rows, cuuint64_t chunks, cuuint64_t row_bytes,
                 cuuint32_t box_chunks) {
    const cuuint64_t dims[3] = {64, rows, chunks > 1 ? chunks : 2}, strides[2] = {row_bytes, chunks > 1 ? 128 : kTmaFar};
    const cuuint32_t box[3] = {64, 64, box_chunks}, es[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t heads = static_cast<cuuint64_t>(p.batch) * kHeads, tokens = static_cast<cuuint64_t>(p.num_pages) * kPage;
  if (!map(&maps.q, p.q_abs, heads, kDc / 64, kDc * 2, 8) || !map(&maps.qr, p.q_rope, heads, 1, kDr * 2, 1) ||
      !map(&maps.k, p.kv_bf16, tokens, kRow / 64, kRow * 2, 3) || !map(&maps.v, p.kv_bf16, tokens, kRow / 64, kRow * 2, 4))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = allow_smem(tree_kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * n_pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_kernel, maps, p);
}

}  // namespace mla
