// Gradients of the expanded-form MLA attention over ragged sequences (prefill.cu),
// with the probabilities recomputed from the forward's LSE.
//
// For query i, key j that it sees, and head h:
//     p  = exp(scale (q_i . k_j) - lse_i)         dv_j = sum_i p do_i
//     ds = p (do_i . v_j - delta_i) scale,        delta_i = do_i . out_i - dlse_i
//     dq_i = sum_j ds k_j,  dk_j = sum_i ds q_i,  the RoPE part of dk summed over the heads.
//
// Bound: five products over 192 or 128 values, 1664 operations per visible pair
// and head, so the tensor cores bound it.  dk and dv are sums over queries, dq
// over keys.  One pass would add dq tiles into global memory from every key tile,
// with an order that changes from run to run and 98 KiB of fp32 traffic a tile.
// Here the key pass holds 128 keys of a head and streams its queries (dk and dv stay in
// tensor memory), and stores each dS tile, 32 KiB of bf16; backward_dq.cu multiplies
// those with K.  Every sum has a fixed order, and nothing is added to global memory.  The
// rope part of dk stays in tensor memory over a group of heads; backward_last.cu adds
// the groups' sums.  The products are the least there are, 832 units of MMAs.
// Where the workspace has no room for all dS tiles (4 GiB, 1024 tiles of every head; the
// plan kernel counts them), the query pass computes dq instead: it holds 128 queries (or
// 256, backward_pair.cu) and streams the keys, for S and dO V^T once more, 512 units
// instead of 192.  Both sides measured: 4096 causal tokens (528 tiles) 1,493 us and
// 1,600, 3 x 777 full 542 and 595, 8 x up to 1024 557 and 617, 2 x 512 queries over 8,012
// keys 1,660 and 1,683, 5 x up to 33 64.7 and 66.7.
//
// One step is a 128 x 128 tile, rows = what is held, columns = what is streamed:
//     S = R1 C1^T, dP = R2 C2^T (R1, C1: 192 values, R2, C2: 128), then
//     keys:    ACC2 += P C2 (dv), ACC1 += dS C1 (dk);  queries: ACC1 += dS C1 (dq).
// P and dS are bf16 operands in tensor memory, a thread's row, so that no
// transposes are needed: the streamed operand of the second products is the same
// shared-memory tile, read along the other axis (MN-major).
//   tensor memory (512 columns): ACC1 192 | ACC2 128 | X 128 | Y 64.  Keys: X holds
//       S, then dP; Y holds P, then dS.  Queries: S is in X, dP in ACC2's place.
//   shared memory: R1 48 KiB, R2 32, two C1 tiles, one C2 tile, two query tiles' lse
//   and delta.
//   warp 0: work items, R1 and R2; warps 3 to 5 a chunk of C1 each and warp 6 C2 (a copy
//   costs its thread 160 cycles to issue), each chunk with its own barrier, warp 7 the
//   statistics; warp 1 issues S and dP, warp 2 the second products; warps 8..23 compute
//   P and dS (thread = a quarter row of 32 columns) and write the results.  S of the
//   next step runs while dS of this one is computed, and the second products of this
//   one while the next one's P is.
// Measured (4096 causal tokens, 1.79 TFLOP of the five products, 952 us at the peak):
// 1,481 us, 1,207 TFLOP/s; 3 x 777 full 542 (a floor of 205), 8 x up to 1024 550 (162),
// 2 x 512 queries over 8,012 keys 1,646 (900), 5 x up to 33 64.7.  With the query pass:
// 8192 causal tokens 5,950 (3,803), 32,768 90 ms (60.8), 1,024 queries over 30,000 keys
// 5,400 (3,422), 8 x 200 over 9,000 5,410 (1,614).  The key pass takes 995 of the first,
// of 754 that its MMAs need at the same peak: S, its reading, dP and its reading
// follow one another in one place of tensor memory, S's MMAs find shared memory busy with
// the copies (1,150 cycles of 768), and storing dS costs 125.  Tried for it and slower:
// two sets of eight warps on alternate steps (2,110 instead of 1,770 for the call),
// streamed tiles multicast to clusters of two (1,830 instead of 1,765), reading S and dP
// together (1,836 instead of 1,770), one warp that issues all products (1,672 instead of
// 1,605), one thread instead of a warp that waits and issues (1,645 instead of 1,609),
// chunks of R1 and R2 loaded one by one (1,705 instead of 1,600), four warps of their
// own that store dS (1,510 instead of 1,494).
//
// Every wait is bounded, as in prefill.cu.
#include <cmath>
#include <type_traits>

#include "backward_tile.cuh"

namespace mla {

namespace {

using namespace bwd;

constexpr int kHelpers = 8;                            // warps that load and issue
constexpr int kThreads = 32 * (kHelpers + kWarps);
constexpr uint32_t kOffR1 = 0, kOffR2 = 3 * kChunk, kOffC1 = 5 * kChunk, kOffC2 = 11 * kChunk, kOffStats = 13 * kChunk;
constexpr uint32_t kOffBar = kOffStats + 2 * kStatBytes;
constexpr int kItemSlots = 2;
enum Bar {
  R1FULL, R1EMPTY, R2FULL, R2EMPTY, C1FULL, C1EMPTY = C1FULL + 6, C2FULL = C1EMPTY + 2, C2EMPTY = C2FULL + 2, SFULL, SREAD, DPFULL,
  DPREAD, PREADY, PDONE, DSREADY, DSDONE, ACCFREE, STATFULL, IFULL = STATFULL + 2, IEMPTY = IFULL + kItemSlots, DRAIN = IEMPTY + kItemSlots,
  NBAR = DRAIN + 2
};
constexpr uint32_t kOffTmem = kOffBar + 8 * NBAR;
constexpr uint32_t kOffQuit = kOffTmem + 4;
constexpr uint32_t kOffItems = (kOffQuit + 4 + 15) & ~15u;
constexpr uint32_t kSmem = kOffItems + kItemBytes * kItemSlots;
static_assert(kSmem <= 232448, "shared memory budget");

constexpr uint32_t kIdescS = ptx::idesc_bf16(128, 128, 0, 0);    // both K-major
constexpr uint32_t kIdesc192 = ptx::idesc_bf16(128, 192, 0, 1), kIdesc128 = ptx::idesc_bf16(128, 128, 0, 1),
                   kIdesc64 = ptx::idesc_bf16(128, 64, 0, 1);    // A in tensor memory, B MN-major
// ---------------------------------------------------------------- plan
// One CTA: the sequences' first query tiles, and the lists of key tiles and of
// query tiles, those with most steps first (counting sort; every tile is computed
// on its own, so the order within a class does not matter).
constexpr int kClasses = 1024;
constexpr int kTailItems = 5;   // items per CTA of the heads that are taken together at the end

__global__ void __launch_bounds__(1024) backward_plan_kernel(const BackwardParams p, const BackwardWs L, int ctas_k, int ctas_q, int ctas_dq, int query_rows) {
  __shared__ int s_count[kClasses], s_warp[32], s_longest, s_shortest;
  __shared__ unsigned long long s_slots;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  BackwardPlan* plan = reinterpret_cast<BackwardPlan*>(p.ws + L.plan);
  int *base_k = reinterpret_cast<int*>(p.ws + L.base[0]), *base = reinterpret_cast<int*>(p.ws + L.base[1]);
  int* slots = reinterpret_cast<int*>(p.ws + L.slots);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ptx::grid_dep_launch();   // (what follows waits for this grid before it reads the plan)
  // inclusive sum over the CTA
  auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += s_warp[w];
    return v;
  };
  struct Seq { int q0, k0, nq, nk; bool ok; };
  auto sequence = [&](int b) {
    const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
    return Seq{q0, k0, q1 - q0, k1 - k0, q0 >= 0 && q1 >= q0 && q1 <= p.nq && k0 >= 0 && k1 >= k0 && k1 <= p.nk};
  };
  for (int side = 0; side < 2; ++side) {
    int before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 1024) {
      int tiles = 0;
      if (b0 + tid < p.batch) {
        const Seq s = sequence(b0 + tid);
        if (s.ok) tiles = ((side ? s.nq : s.nk) + kTile - 1) / kTile;
        else set_status(&hdr->status, MLA_STATUS_BAD_SEQ_LEN);
      }
      const int sum = scan(tiles);
      if (b0 + tid < p.batch) (side ? base : base_k)[b0 + tid] = before + sum - tiles;
      __syncthreads();
      if (tid == 1023) s_warp[0] = sum;
      __syncthreads();
      before += s_warp[0];
    }
  }
  bool from_ds = false;   // (known after the key tiles' first count)
  for (int side = 0; side < 2; ++side) {
    Tile* tiles = reinterpret_cast<Tile*>(p.ws + L.tiles[side]);
    __syncthreads();
    s_count[tid] = 0;
    if (tid == 0) {
      s_longest = 0;
      s_shortest = kClasses;
      s_slots = 0;
    }
    __syncthreads();
    for (int pass = 0; pass < 2; ++pass) {
      for (int b = warp; b < p.batch; b += 32) {
        const Seq s = sequence(b);
        if (!s.ok) continue;
        const int n = side ? s.nq : s.nk, rows = side && !from_ds ? query_rows : kTile, off = s.nk - s.nq;
        // (beyond the lists: overlapping sequences, cu decreased somewhere)
        const bool fits = base[b] + (s.nq + kTile - 1) / kTile <= L.max_tiles[1] && base_k[b] + (s.nk + kTile - 1) / kTile <= L.max_tiles[0];
        for (int i0 = 0; i0 * rows < n; i0 += 32) {
          Tile t;
          const int i = i0 + lane, at = i * rows;
          const bool tile = at < n;
          t.rows = min(rows, n - at);
          t.first = 0;
          if (side == 0) {
            t.r0 = s.k0 + at;
            t.c0 = s.q0;
            t.nc = s.nq;
            t.lim = at - off;
            if (p.causal) t.first = max(0, t.lim) / kTile;
            t.steps = max(0, (s.nq + kTile - 1) / kTile - t.first);
            t.stat = base[b];
            // places of dS tiles, for 32 key tiles at once
            const int mine = tile && fits ? t.steps : 0;
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int y = __shfl_up_sync(0xffffffffu, sum, o);
              if (lane >= o) sum += y;
            }
            unsigned long long from = 0;
            if (lane == 31) from = atomicAdd(&s_slots, static_cast<unsigned long long>(sum));
            t.slot = static_cast<int>(__shfl_sync(0xffffffffu, from, 31)) + sum - mine - t.first;
            if (pass == 1 && tile && fits) slots[base_k[b] + i] = t.slot;
          } else {
            t.r0 = s.q0 + at;
            t.c0 = s.k0;
            t.nc = s.nk;
            t.lim = at + off + 1;
            const int sees = p.causal ? max(0, min(s.nk, t.lim + t.rows - 1)) : s.nk;   // its last row
            t.steps = (sees + kTile - 1) / kTile;
            t.stat = base[b] + at / kTile;
            t.slot = base_k[b];
          }
          t.tile = i;
          if (!tile) continue;
          const int steps = min(kClasses - 1, t.steps), c = kClasses - 1 - steps;
          if (pass == 0) {
            atomicMax(&s_longest, steps);
            atomicMin(&s_shortest, steps);
          }
          const int pos = atomicAdd(&s_count[c], 1);
          if (pass == 1) {
            if (pos < L.max_tiles[side] && fits) tiles[pos] = t;
            else {
              if (pos < L.max_tiles[side]) {
                t.rows = t.steps = 0;
                tiles[pos] = t;
              }
              set_status(&hdr->status, MLA_STATUS_BAD_SEQ_LEN);
            }
          }
        }
      }
      __syncthreads();
      if (pass == 0) {
        if (side == 0) from_ds = ctas_k > 0 && s_slots <= static_cast<unsigned long long>(L.ds_tiles);
        // exclusive scan: s_count[c] becomes the first position of class c
        const int v = s_count[tid], x = scan(v);
        s_count[tid] = x - v;
        if (tid == 0) s_slots = 0;   // (all have read it: scan's barriers)
        if (tid == 1023) {
          const int n = min(x, L.max_tiles[side]), ctas = side ? (from_ds ? ctas_dq : ctas_q) : ctas_k, groups = side ? kHeads : kHeads / L.group;
          plan->tiles[side] = n;
          plan->next[side] = ctas;
          plan->odd[side] = 0;
          plan->stored = from_ds;
          plan->query_rows = from_ds ? kTile : query_rows;
          // (as in prefill: not where all tiles are about as long)
          const bool even = 2 * s_longest <= 3 * s_shortest;
          plan->tail[side] = even ? 1 : min(groups, (kTailItems * ctas + n - 1) / max(n, 1));
          hdr->abort_flag = 0;
        }
        __syncthreads();
      }
    }
  }
}

// ---------------------------------------------------------------- delta
// lse log2(e) and sum(d_out out) - d_lse per query tile and head: 32 rows and 8 heads a
// CTA, 16 threads a row and head, whose loads are all in flight together.
constexpr int kDeltaRows = 32;

__global__ void __launch_bounds__(256) backward_delta_kernel(const BackwardParams p, const BackwardWs L) {
  __shared__ float s_delta[8][kDeltaRows];
  BackwardPlan* plan = reinterpret_cast<BackwardPlan*>(p.ws + L.plan);
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int parts = *reinterpret_cast<const volatile int*>(&plan->query_rows) / kDeltaRows;
  const int i_tile = static_cast<int>(blockIdx.x) / parts, part = static_cast<int>(blockIdx.x) % parts;
  if (i_tile >= *reinterpret_cast<const volatile int*>(&plan->tiles[1])) return;
  const Tile t = reinterpret_cast<const Tile*>(p.ws + L.tiles[1])[i_tile];
  // (a stat tile is 128 rows: those past the sequence's end get zeros)
  const int r0 = part * kDeltaRows;
  if ((t.rows + kTile - 1) / kTile * kTile <= r0) return;
  const int h0 = 8 * blockIdx.y, lane16 = threadIdx.x & 15, first = threadIdx.x >> 4;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 a[8], b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = first + 16 * (8 * half + k), r = r0 + (i >> 3), h = h0 + (i & 7);
      a[k] = b[k] = make_uint4(0, 0, 0, 0);
      if (r < t.rows) {
        const size_t row = static_cast<size_t>(t.r0) + r;
        a[k] = __ldg(reinterpret_cast<const uint4*>(p.d_out + row * p.do_t + h * p.do_h) + lane16);
        b[k] = __ldg(reinterpret_cast<const uint4*>(p.out + (row * kHeads + h) * 128) + lane16);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t x[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, y[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum += __uint_as_float(x[e] << 16) * __uint_as_float(y[e] << 16);
        sum += __uint_as_float(x[e] & 0xFFFF0000u) * __uint_as_float(y[e] & 0xFFFF0000u);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int i = first + 16 * (8 * half + k);
      if (lane16 == 0) s_delta[i & 7][i >> 3] = sum;
    }
  }
  __syncthreads();
  const int h = threadIdx.x / kDeltaRows, r = threadIdx.x % kDeltaRows;
  float* stats = reinterpret_cast<float*>(p.ws + L.stats) +
                 (static_cast<size_t>(t.stat + r0 / kTile) * kHeads + h0 + h) * 2 * kTile + r0 % kTile + r;
  float l = 0.f, d = 0.f;
  if (r0 + r < t.rows) {
    const size_t at = (static_cast<size_t>(t.r0) + r0 + r) * kHeads + h0 + h;
    l = __ldg(p.lse + at) * kLog2e;
    d = s_delta[h][r] - (p.d_lse ? __ldg(p.d_lse + at) : 0.f);
    // a value of q, d_out or d_lse that is not finite is seen here, in the lse or in
    // delta; so are, for nothing, queries that see no key
    if (p.causal && !(isfinite(l) && isfinite(d))) plan->odd[0] = 1;
  }
  stats[0] = l;
  stats[kTile] = d;
}

// ---------------------------------------------------------------- the two passes
// kKeys: rows are keys (dk, dv), else queries (dq).
template <bool kKeys>
__global__ void __launch_bounds__(kThreads, 1)
backward_kernel(const __grid_constant__ PassMaps maps, const __grid_constant__ BackwardParams p, const BackwardWs L) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  BackwardPlan* plan = reinterpret_cast<BackwardPlan*>(p.ws + L.plan);
  volatile uint32_t* const quit = reinterpret_cast<volatile uint32_t*>(smem + kOffQuit);
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  constexpr int kSide = kKeys ? 0 : 1;
  constexpr uint32_t kDp = kKeys ? kX : kAcc2;
  const int group = kKeys ? L.group : 1, groups = kHeads / group;
  if (threadIdx.x == 0) {
    *quit = 0;
    for (int i = 0; i < NBAR; ++i) {
      int n = 1;                                   // copies, MMA commits
      if (i == SREAD || i == DPREAD || i == PREADY || i == DSREADY || i == ACCFREE) n = kWarps;   // one arrival a warp
      // (roles that walk the items: the C copies, the two that issue)
      if (i == C2EMPTY && kKeys) n = 2;            // dP and dv
      if (i >= IEMPTY && i < IEMPTY + kItemSlots) n = kWarps + (kKeys ? 7 : 6);
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
  begin_pass<kKeys>(p);
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  const int causal = p.causal;
  const bool keep = kKeys && stored(plan);   // dS, for dq

  struct Walk { int slot = 0; uint32_t phase = 0; };
  // The next item of this role's walk: its tile and first head, false when there is none.
  auto next_warp = [&](Walk& w, Tile& t, int& head) {
    if (!wait_cta_warp(BAR(IFULL + w.slot), w.phase, quit)) return false;
    read_item(smem + kOffItems + kItemBytes * w.slot, t, head);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(IEMPTY + w.slot));
    if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
    return head >= 0;
  };

  // A role's walk over the steps of all items: f(tile, head, step of the head, number
  // of the step so far) is false when a wait gave up.  Returns the number of steps.
  auto walk_steps = [&](auto f) {
    Walk w;
    Tile t;
    int head0;
    uint32_t n = 0;
    bool ok = true;
    while (ok && next_warp(w, t, head0)) {
      for (int g = 0; g < group && ok; ++g)
        for (int i = 0; i < t.steps && ok; ++i) {
          ok = f(t, head0 + g, i, n);
          if (ok) ++n;
        }
    }
    return n;
  };

  if (smem_ok && warp == 0) {
    // ------------------------------------------------------------ items, and the loads of R1 and R2
    regs_issue();
    if (elect_one()) {
      const Tile* tiles = reinterpret_cast<const Tile*>(p.ws + L.tiles[kSide]);
      const Schedule sched(plan, kSide, groups, !kKeys && stored(plan));
      Walk w;
      uint32_t loads = 0, loads2 = 0;
      bool ok = true;
      int item = static_cast<int>(blockIdx.x);
      while (ok) {
        Tile t = {};
        int tile, head0 = -1;
        if (sched.find(item, tile, head0)) {
          t = read_tile(tiles + tile);
          head0 *= group;
        }
        ok = wait_cta(BAR(IEMPTY + w.slot), w.phase ^ 1u, quit);
        if (!ok) break;
        write_item(smem + kOffItems + kItemBytes * w.slot, t, head0);
        ptx::mbar_arrive(BAR(IFULL + w.slot));
        if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
        if (head0 < 0) break;
        for (int g = 0; g < group && t.steps > 0 && ok; ++g) {
          const int head = head0 + g;
          ok = wait_cta(BAR(R1EMPTY), (loads & 1u) ^ 1u, quit);
          if (!ok) break;
          ++loads;
          ptx::mbar_arrive_expect_tx(BAR(R1FULL), 3 * kChunk);
          load_4d(sbase + kOffR1, &maps.r1n, BAR(R1FULL), 0, t.r0, 0, head);
          load_4d(sbase + kOffR1 + 2 * kChunk, &maps.r1r, BAR(R1FULL), 0, t.r0, 0, kKeys ? 0 : head);
          ok = wait_cta(BAR(R2EMPTY), (loads2 & 1u) ^ 1u, quit);
          if (!ok) break;
          ++loads2;
          ptx::mbar_arrive_expect_tx(BAR(R2FULL), 2 * kChunk);
          load_4d(sbase + kOffR2, &maps.r2, BAR(R2FULL), 0, t.r0, 0, head);
        }
        // Claimed when the item's last rows are on their way: its steps are still to come.
        item = atomicAdd(&plan->next[kSide], 1);
      }
      // no copy may land after the CTA has left
      if (loads > 0) wait_issued(BAR(R1FULL), (loads - 1) & 1u, quit);
      if (loads2 > 0) wait_issued(BAR(R2FULL), (loads2 - 1) & 1u, quit);
    }
    __syncwarp();
  } else if (smem_ok && warp >= 3 && warp < 6) {
    // ------------------------------------------------------------ loads of C1, a chunk of 64 values each
    // (A copy costs its thread 160 cycles to issue, and one thread that waited for all
    // buffers in turn held up one copy for another's sake.  The products of a chunk
    // begin when it has landed.)
    regs_issue();
    const int chunk = warp - 3;
    uint32_t queued = 0;
    walk_steps([&](const Tile& t, int head, int i, uint32_t n) {
      const uint32_t buf = n & 1u;
      const int bar = C1FULL + 3 * static_cast<int>(buf) + chunk;
      if (!wait_cta_warp(BAR(C1EMPTY + buf), ((n >> 1) & 1u) ^ 1u, quit)) return false;
      ++queued;
      if (elect_one()) {
        ptx::mbar_arrive_expect_tx(BAR(bar), kChunk);
        load_4d(sbase + kOffC1 + (buf * 3 + chunk) * kChunk, chunk < 2 ? &maps.c1n : &maps.c1r, BAR(bar), 0,
                t.c0 + (t.first + i) * kTile, chunk & 1, kKeys || chunk < 2 ? head : 0);
      }
      __syncwarp();
      return true;
    });
    for (uint32_t b = 0; b < 2 && b < queued; ++b)
      wait_issued(BAR(C1FULL + 3 * b + chunk), ((queued + 1 - b) / 2 - 1) & 1u, quit);
  } else if (smem_ok && warp == 6) {
    // ------------------------------------------------------------ loads of C2, a chunk each
    regs_issue();
    uint32_t queued = 0;
    walk_steps([&](const Tile& t, int head, int i, uint32_t n) {
      if (!wait_cta_warp(BAR(C2EMPTY), (n & 1u) ^ 1u, quit)) return false;
      ++queued;
      if (elect_one()) {
        for (int c = 0; c < 2; ++c) {
          ptx::mbar_arrive_expect_tx(BAR(C2FULL + c), kChunk);
          load_4d(sbase + kOffC2 + c * kChunk, &maps.c2, BAR(C2FULL + c), 0, t.c0 + (t.first + i) * kTile, c, head);
        }
      }
      __syncwarp();
      return true;
    });
    for (int c = 0; c < 2 && queued > 0; ++c) wait_issued(BAR(C2FULL + c), (queued - 1) & 1u, quit);
  } else if (kKeys && smem_ok && warp == 7) {
    // ------------------------------------------------------------ lse and delta of the streamed queries
    regs_issue();
    const float* stats = reinterpret_cast<const float*>(p.ws + L.stats);
    walk_steps([&](const Tile& t, int head, int i, uint32_t n) {
      // read while the step before the last, whose place they take, is still at work
      const uint32_t buf = n & 1u;
      const float4* src = reinterpret_cast<const float4*>(
          stats + (static_cast<size_t>(t.stat + t.first + i) * kHeads + head) * 2 * kTile) + lane;
      const float4 lse = __ldcg(src), delta = __ldcg(src + kTile / 4);
      // (its dS has been computed when the product with it is done)
      if (!wait_cta_warp(BAR(C1EMPTY + buf), ((n >> 1) & 1u) ^ 1u, quit)) return false;
      float4* dst = reinterpret_cast<float4*>(smem + kOffStats + buf * kStatBytes) + lane;
      dst[0] = lse;
      dst[kTile / 4] = delta;
      __syncwarp();
      if (elect_one()) ptx::mbar_arrive(BAR(STATFULL + static_cast<int>(buf)));
      return true;
    });
  } else if (smem_ok && warp == 1) {
    regs_issue();
    // ------------------------------------------------------------ S = R1 C1^T, dP = R2 C2^T
    Walk w;
    Tile t;
    int head;
    const uint64_t r1 = ptx::sdesc_sw128(sbase + kOffR1, 16, 1024), r2 = ptx::sdesc_sw128(sbase + kOffR2, 16, 1024);
    const uint64_t c1 = ptx::sdesc_sw128(sbase + kOffC1, 16, 1024), c2 = ptx::sdesc_sw128(sbase + kOffC2, 16, 1024);
    constexpr uint64_t kChunkD = kChunk >> 4;
    uint32_t n = 0, loads = 0;
    bool ok = true, issued = false;
#ifdef MLA_TEST_STALL_WAIT
    // Test builds only: a wait on a barrier that nothing arrives on before the end
    // of the kernel, so that its limit runs out and every role leaves.
    ok = wait_cta_warp(BAR(DRAIN), 0u, quit);
#endif
    while (ok && next_warp(w, t, head)) {
      const int steps = __shfl_sync(0xffffffffu, t.steps, 0);
      for (int g = 0; g < group && ok; ++g) {
        for (int i = 0; i < steps && ok; ++i, ++n) {
          const uint32_t buf = n & 1u;
          if (i == 0) ok = wait_cta_warp(BAR(R1FULL), loads & 1u, quit);
          // (who sees S finds the statistics)
          if (kKeys && ok) ok = wait_cta_warp(BAR(STATFULL + buf), (n >> 1) & 1u, quit);
          // S's place: the last dP has been read from it (keys), or the last S
          if (ok && n > 0) ok = wait_cta_warp(BAR(kKeys ? DPREAD : SREAD), (n - 1) & 1u, quit);
#pragma unroll 1
          for (int c = 0; c < 3 && ok; ++c) {
            ok = wait_cta_warp(BAR(C1FULL + 3 * static_cast<int>(buf) + c), (n >> 1) & 1u, quit);
            if (!ok) break;
            ptx::tc_fence_after();
            issued = true;
            if (elect_one()) {
              const uint64_t a = r1 + c * kChunkD, b = c1 + (3u * buf + c) * kChunkD;
#pragma unroll
              for (int k = 0; k < 4; ++k) ptx::mma_ss(tmem + kX, a + 2u * k, b + 2u * k, kIdescS, (c > 0 || k > 0) ? 1u : 0u);
              if (c == 2) {
                ptx::mma_commit(BAR(SFULL));
                if (i == steps - 1) ptx::mma_commit(BAR(R1EMPTY));
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (i == 0) ok = wait_cta_warp(BAR(R2FULL), loads & 1u, quit);
          if (ok && (kKeys || n > 0)) ok = wait_cta_warp(BAR(kKeys ? SREAD : DPREAD), (kKeys ? n : n - 1) & 1u, quit);
#pragma unroll 1
          for (int c = 0; c < 2 && ok; ++c) {
            ok = wait_cta_warp(BAR(C2FULL + c), n & 1u, quit);
            if (!ok) break;
            ptx::tc_fence_after();
            if (elect_one()) {
              const uint64_t a = r2 + c * kChunkD, b = c2 + c * kChunkD;
#pragma unroll
              for (int k = 0; k < 4; ++k) ptx::mma_ss(tmem + kDp, a + 2u * k, b + 2u * k, kIdescS, (c > 0 || k > 0) ? 1u : 0u);
              if (c == 1) {
                ptx::mma_commit(BAR(DPFULL));
                ptx::mma_commit(BAR(C2EMPTY));
                if (i == steps - 1) ptx::mma_commit(BAR(R2EMPTY));
              }
            }
            __syncwarp();
          }
        }
        if (steps > 0) ++loads;
      }
    }
    // every MMA this warp issued completes before the CTA may leave
    if (issued && elect_one()) {   // the lane that issued them
      ptx::mma_commit(BAR(DRAIN));
      wait_issued(BAR(DRAIN), 0u, quit);
    }
    __syncwarp();
  } else if (smem_ok && warp == 2) {
    regs_issue();
    // ------------------------------------------------------------ ACC2 += P C2 (keys), ACC1 += dS C1
    Walk w;
    Tile t;
    int head;
    // along the other axis: 64-value chunks kChunk apart, 8-row groups 1 KiB
    const uint64_t c1 = ptx::sdesc_sw128(sbase + kOffC1, kChunk, 1024), c2 = ptx::sdesc_sw128(sbase + kOffC2, kChunk, 1024);
    uint32_t n = 0, heads = 0;               // steps, and heads with steps, so far
    bool ok = true, issued = false;
    // columns past the sequence's end have P = dS = 0; make their rows 0 too (they
    // may be another sequence's, and hold NaN)
    auto clear = [&](uint32_t at, uint32_t chunks, int valid) {
#pragma unroll 1
      for (uint32_t c = 0; c < chunks; ++c) {
        uint4* dst = reinterpret_cast<uint4*>(smem + at + c * kChunk);
        for (int i = valid * 8 + lane; i < kTile * 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
      }
      ptx::fence_proxy_async_cta();
      __syncwarp();
    };
    // In a tile with hidden pairs, whose P and dS are 0, values that are not finite count
    // as 0 too; where the call may have any (backward_last.cu adds what was left out).
    auto finite_alone = [&](uint32_t at, uint32_t chunks) {
      uint4* x = reinterpret_cast<uint4*>(smem + at);
#pragma unroll 1
      for (uint32_t i = lane; i < chunks * (kChunk / 16); i += 32) {
        uint4 v = x[i];
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u;
          if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu;
        }
        x[i] = v;
      }
      ptx::fence_proxy_async_cta();
      __syncwarp();
    };
    // (two bodies: with the test in one, 4096 causal tokens took 1,524 us instead of 1,498)
    auto walk = [&](auto form) {
      constexpr bool careful = decltype(form)::value;
      while (ok && next_warp(w, t, head)) {
        const int steps = __shfl_sync(0xffffffffu, t.steps, 0);
        for (int g = 0; g < group && ok; ++g) {
          for (int i = 0; i < steps && ok; ++i, ++n) {
            const uint32_t buf = n & 1u;
            const bool edge = careful && (t.first + i) * kTile < mask_end(t);
            const int valid = __shfl_sync(0xffffffffu, t.nc - (t.first + i) * kTile, 0);
            // a head's first products overwrite the accumulators: they must have been read
            if (i == 0) ok = wait_cta_warp(BAR(ACCFREE), (heads & 1u) ^ 1u, quit);
            if constexpr (kKeys) {
              for (int c = 0; c < 2 && ok; ++c) ok = wait_cta_warp(BAR(C2FULL + c), n & 1u, quit);
              if (ok) ok = wait_cta_warp(BAR(PREADY), n & 1u, quit);
              if (ok && edge) ok = wait_cta_warp(BAR(DPFULL), n & 1u, quit);   // dP has been formed of what is there
              if (!ok) break;
              if (valid < kTile) clear(kOffC2, 2, valid);
              if (edge) finite_alone(kOffC2, 2);
              ptx::tc_fence_after();
              issued = true;
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  ptx::mma_ts(tmem + kAcc2, tmem + kY + 8u * k, c2 + 128u * k, kIdesc128, (i > 0 || k > 0) ? 1u : 0u);
                ptx::mma_commit(BAR(PDONE));
                ptx::mma_commit(BAR(C2EMPTY));
              }
              __syncwarp();
            }
            for (int c = 0; c < 3 && ok; ++c) ok = wait_cta_warp(BAR(C1FULL + 3 * static_cast<int>(buf) + c), (n >> 1) & 1u, quit);
            if (ok) ok = wait_cta_warp(BAR(DSREADY), n & 1u, quit);
            if (!ok) break;
            if (valid < kTile) clear(kOffC1 + buf * 3 * kChunk, 3, valid);
            if (edge) finite_alone(kOffC1 + buf * 3 * kChunk, 3);
            ptx::tc_fence_after();
            issued = true;
            if (elect_one()) {
              const uint64_t b = c1 + buf * (3 * kChunk >> 4);
              if (i == 0) {
                // the RoPE columns go on from the group's last head
                ptx::mma_ts(tmem + kAcc1, tmem + kY, b, kIdesc128, 0u);
                ptx::mma_ts(tmem + kAcc1 + 128, tmem + kY, b + 2 * (kChunk >> 4), kIdesc64, g > 0 ? 1u : 0u);
              } else {
                ptx::mma_ts(tmem + kAcc1, tmem + kY, b, kIdesc192, 1u);
              }
#pragma unroll
              for (int k = 1; k < 8; ++k) ptx::mma_ts(tmem + kAcc1, tmem + kY + 8u * k, b + 128u * k, kIdesc192, 1u);
              ptx::mma_commit(BAR(DSDONE));
              ptx::mma_commit(BAR(C1EMPTY + buf));
            }
            __syncwarp();
          }
          if (steps > 0) ++heads;
        }
      }
    };
    if (kKeys && causal && *reinterpret_cast<const volatile int*>(&plan->odd[0]) != 0) walk(std::bool_constant<kKeys>());
    else walk(std::false_type());
    if (issued && elect_one()) {
      ptx::mma_commit(BAR(DRAIN + 1));
      wait_issued(BAR(DRAIN + 1), 0u, quit);
    }
    __syncwarp();
  } else if (smem_ok && warp < kHelpers) {
    regs_issue();   // (idle: a register split is the whole warpgroup's)
  } else if (smem_ok) {
    // ------------------------------------------------------------ P and dS (thread = a quarter row), results
    regs_compute();
    const int quarter = (warp - kHelpers) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t x_addr = tmem + lane_base + kX + 32u * quarter, dp_addr = tmem + lane_base + kDp + 32u * quarter;
    const uint32_t y_addr = tmem + lane_base + kY + 16u * quarter;
    const float c = p.scale * kLog2e;
    Walk w;
    Tile t;
    int head0;
    uint32_t n = 0;
    bool ok = true;
    auto arrive = [&](int bar) {
      ptx::tc_fence_before();
      __syncwarp();
      if (elect_one()) ptx::mbar_arrive(BAR(bar));
    };
    while (ok && next_warp(w, t, head0)) {
      const size_t row = static_cast<size_t>(t.r0) + r;
      const bool mine = r < t.rows;
      for (int g = 0; g < group && ok; ++g) {
        const int head = head0 + g;
        float row_lse = 0.f, row_delta = 0.f;
        if constexpr (!kKeys) {
          const float* st = reinterpret_cast<const float*>(p.ws + L.stats) + (static_cast<size_t>(t.stat) * kHeads + head) * 2 * kTile;
          row_lse = __ldcg(st + r);
          row_delta = __ldcg(st + kTile + r);
        }
        for (int i = 0; i < t.steps; ++i, ++n) {
          const uint32_t buf = n & 1u;
          // columns [lo, hi) of this thread's 32 are seen
          const int at = (t.first + i) * kTile + kCols * quarter;
          int lo = 0, hi = t.nc - at;
          if (causal) {
            if constexpr (kKeys) lo = t.lim + r - at;
            else hi = min(hi, t.lim + r - at);
          }
          const bool all = __all_sync(0xffffffffu, lo <= 0 && hi >= kCols);
          ok = wait_cta_warp(BAR(SFULL), n & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t s[kCols], pk[kCols / 2];
          ptx::tmem_ld32(x_addr, s);
          ptx::tmem_wait_ld();
          arrive(SREAD);
          const float4* lse4 = reinterpret_cast<const float4*>(smem + kOffStats + buf * kStatBytes) + kCols / 4 * quarter;
          probabilities<kKeys>(s, lse4, row_lse, c, all, lo, hi);
          if constexpr (kKeys) {
            pack(s, pk);
            // the last step's dS has been read
            if (n > 0) ok = wait_cta_warp(BAR(DSDONE), (n - 1) & 1u, quit);
            if (!ok) break;
            ptx::tc_fence_after();
            tmem_st16(y_addr, pk);
            ptx::tmem_wait_st();
            arrive(PREADY);
          }
          ok = wait_cta_warp(BAR(DPFULL), n & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t d[kCols];
          ptx::tmem_ld32(dp_addr, d);
          ptx::tmem_wait_ld();
          arrive(DPREAD);
          gradients<kKeys>(s, d, lse4 + kTile / 4, row_delta, all, lo, hi, pk);
          // P (keys), or the last step's dS, has been read
          if (kKeys) ok = wait_cta_warp(BAR(PDONE), n & 1u, quit);
          else if (n > 0) ok = wait_cta_warp(BAR(DSDONE), (n - 1) & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          tmem_st16(y_addr, pk);
          ptx::tmem_wait_st();
          arrive(DSREADY);
          if (kKeys && keep) {
            if (!mine) {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0;
            }
            store_ds(p.ws + L.ds + (static_cast<size_t>(t.slot + t.first + i) * kHeads + head) * kDsTile, r, quarter, pk);
          }
        }
        if (!ok) break;
        // results of the head
        const bool last = g == group - 1;
        uint32_t nope[16], second[16], rope[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) nope[e] = second[e] = rope[e] = 0;
        if (t.steps > 0) {
          ok = wait_cta_warp(BAR(DSDONE), (n - 1) & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t a[32], b[32];
          ptx::tmem_ld32(tmem + lane_base + kAcc1 + 32u * quarter, a);
          if constexpr (kKeys) ptx::tmem_ld32(tmem + lane_base + kAcc2 + 32u * quarter, b);
          if (!kKeys || last) ptx::tmem_ld16(tmem + lane_base + kAcc1 + 128u + 16u * quarter, rope);
          ptx::tmem_wait_ld();
          to_bf16<16>(a, p.scale, nope);
          if constexpr (kKeys) to_bf16<16>(b, 1.f, second);
          else to_bf16<8>(rope, p.scale, rope);
          arrive(ACCFREE);
        }
        if (mine) store_results<kKeys>(p, L, row, head, head0 / group, quarter, last, nope, second, rope);
      }
    }
  }
  // ------------------------------------------------------------ teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *quit != 0) set_status(&hdr->status, MLA_STATUS_TIMEOUT);
  if constexpr (kKeys) ptx::grid_dep_wait();   // (see begin_pass)
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Rows of a query tile in the query pass: 256, on CTA pairs (backward_pair.cu), unless
// too many of their rows and columns are masked.  Of an average sequence, a pair's tiles
// of 256 instead of 128 rows are 64 rows more at its end and, where causal, 64 columns
// more a row at the diagonal; a pair's query pass is about a sixth faster on full tiles.
// Shares, and us a call that stores nothing with tiles of 128 and of 256: 2 x 512 over
// 8,012 keys 0.13, 1,808 and 1,686; 2 x 800 over 1,200 0.16, 497 and 497; 4 x 1024 causal
// 0.19, 716 and 702; 4 x 300 over 4,300 0.23, 1,782 and 1,808; 4 x 300 full 0.21, 235 and
// 243; 8 x up to 1024 0.37, 611 and 648.
int backward_rows(const BackwardParams& p) {
  const double n_q = static_cast<double>(p.nq) / p.batch, n_k = static_cast<double>(p.nk) / p.batch;
  const double seen = p.causal ? std::fmax(n_k - n_q / 2, 1.0) : std::fmax(n_k, 1.0);
  return 64.0 / n_q + (p.causal ? 64.0 / seen : 0.0) <= 0.2 ? 2 * kTile : kTile;
}

}  // namespace

cudaError_t launch_backward(PFN_cuTensorMapEncodeTiled_v12000 encode, BackwardParams p, int sms, cudaStream_t stream) {
  const BackwardWs L = backward_ws(p.batch, p.nq, p.nk);
  const int query_rows = backward_rows(p);
  auto ctas = [&](int side, int most) {
    const long long items = static_cast<long long>(L.max_tiles[side]) * (side ? kHeads : kHeads / L.group);
    return static_cast<int>(items < most ? items : most);
  };
  const int keys = ctas(0, sms), queries = ctas(1, sms * kTile / query_rows), dq = ctas(1, sms);
  // the query pass is needed where not all dS tiles may find room, or there is no key pass
  const bool query_pass = queries > 0 && (!L.ds_always || keys == 0);
  p.key_waits = !query_pass;
  cudaError_t e = launch_kernel(backward_plan_kernel, dim3(1), dim3(1024), 0, stream, p, L, keys, queries, dq, query_rows);
  PassMaps maps;
  static std::atomic<uint64_t> configured_q{0}, configured_k{0};
  if (e == cudaSuccess && queries)
    e = launch_dependent(backward_delta_kernel, dim3(L.max_tiles[1] * (query_rows / kDeltaRows), kHeads / 8), dim3(256), 0, stream,
                         p, L);
  if (e == cudaSuccess && query_pass) {
    if (!pass_maps(encode, p, false, query_rows == kTile ? kTile : kTile / 2, &maps)) e = cudaErrorInvalidValue;
    if (e == cudaSuccess && query_rows > kTile) {
      e = launch_backward_pairs(maps, p, L, queries, stream);
    } else if (e == cudaSuccess) {
      e = allow_smem(backward_kernel<false>, kSmem, configured_q);
      if (e == cudaSuccess)
        e = launch_dependent(backward_kernel<false>, dim3(queries), dim3(kThreads), kSmem, stream, maps, p, L);
    }
  }
  if (e == cudaSuccess && keys) {
    if (!pass_maps(encode, p, true, kTile, &maps)) e = cudaErrorInvalidValue;
    if (e == cudaSuccess) e = allow_smem(backward_kernel<true>, kSmem, configured_k);
    if (e == cudaSuccess) e = launch_dependent(backward_kernel<true>, dim3(keys), dim3(kThreads), kSmem, stream, maps, p, L);
    if (e == cudaSuccess && queries) e = launch_backward_dq(encode, p, L, dq, stream);
    if (e == cudaSuccess) e = launch_backward_last(p, L, stream);
  }
  return e;
}

}  // namespace mla
