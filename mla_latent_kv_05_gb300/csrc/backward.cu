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
// Here two passes of one kernel compute S and dO V^T each: one holds 128 keys of
// a head and streams its queries (dk and dv stay in tensor memory), the other
// holds 128 queries and streams the keys (dq stays).  That is 640 + 512 units of
// MMAs where 832 would be the least, every sum has a fixed order, and nothing is
// added to global memory.  In the first the rope part of dk stays in tensor memory
// over a group of heads; the groups' sums are added by a last small kernel.
//
// One step is a 128 x 128 tile, rows = what is held, columns = what is streamed:
//     S = R1 C1^T, dP = R2 C2^T (R1, C1: 192 values, R2, C2: 128), then
//     keys:    ACC2 += P C2 (dv), ACC1 += dS C1 (dk);  queries: ACC1 += dS C1 (dq).
// P and dS are bf16 operands in tensor memory, a thread's row, so that no
// transposes are needed: the streamed operand of the second products is the same
// shared-memory tile, read along the other axis (MN-major).
//   tensor memory (512 columns): ACC1 192 | ACC2 128 | X 128 | Y 64.  Keys: X holds
//       S, then dP; Y holds P, then dS.  Queries: S is in X, dP in ACC2's place.
//   shared memory: R1 48 KiB, R2 32, two C1 tiles, one C2 tile.
//   warp 0: work items and TMA loads; warp 1 issues S and dP, warp 2 the second
//   products; warps 4..11 compute P and dS (thread = half a row) and write the
//   results.  S of the next step runs while dS of this one is computed, and the
//   second products of this one while the next one's P is.
//
// Every wait is bounded, as in prefill.cu.
#include <climits>

#include "backward.cuh"

namespace mla {

namespace {

constexpr int kTile = kBackwardTile;
constexpr int kThreads = 384;
constexpr uint32_t kChunk = kTile * 128u;          // 16 KiB: 128 rows x 64 values
constexpr uint32_t kOffR1 = 0, kOffR2 = 3 * kChunk, kOffC1 = 5 * kChunk, kOffC2 = 11 * kChunk, kOffStats = 13 * kChunk;
constexpr uint32_t kStatBytes = 2 * kTile * 4;     // lse and delta of a query tile
constexpr uint32_t kOffBar = kOffStats + 2 * kStatBytes;
constexpr int kItemSlots = 2;
enum Bar {
  R1FULL, R1EMPTY, R2FULL, R2EMPTY, C1FULL, C1EMPTY = C1FULL + 2, C2FULL = C1EMPTY + 2, C2EMPTY, SFULL, SREAD, DPFULL,
  DPREAD, PREADY, PDONE, DSREADY, DSDONE, ACCFREE, IFULL, IEMPTY = IFULL + kItemSlots, DRAIN = IEMPTY + kItemSlots,
  NBAR = DRAIN + 2
};
constexpr uint32_t kOffTmem = kOffBar + 8 * NBAR;
constexpr uint32_t kOffQuit = kOffTmem + 4;
constexpr uint32_t kOffItems = (kOffQuit + 4 + 15) & ~15u;
constexpr uint32_t kSmem = kOffItems + 48 * kItemSlots;
static_assert(kSmem <= 232448, "shared memory budget");

constexpr uint32_t kAcc1 = 0, kAcc2 = 192, kX = 320, kY = 448;   // tensor memory columns
constexpr uint32_t kIdescS = ptx::idesc_bf16(128, 128, 0, 0);    // both K-major
constexpr uint32_t kIdesc192 = ptx::idesc_bf16(128, 192, 0, 1), kIdesc128 = ptx::idesc_bf16(128, 128, 0, 1),
                   kIdesc64 = ptx::idesc_bf16(128, 64, 0, 1);    // A in tensor memory, B MN-major
constexpr float kLog2e = 1.4426950408889634f;

// A tile of rows: keys (key pass) or queries (query pass).
struct Tile {
  int r0, rows;   // first packed row, rows (1..128)
  int c0, nc;     // first packed column of the sequence, its columns
  int lim;        // row r sees the columns from lim + r (keys), or those below lim + r (queries), where causal
  int first;      // first column tile
  int steps;      // column tiles
  int stat;       // query tile number of column tile 0 (keys), or of the tile itself (queries)
};
static_assert(sizeof(Tile) == 32, "tile record");

// ---------------------------------------------------------------- plan
// One CTA: the sequences' first query tiles, and the lists of key tiles and of
// query tiles, those with most steps first (counting sort; every tile is computed
// on its own, so the order within a class does not matter).
constexpr int kClasses = 1024;
constexpr int kTailItems = 5;   // items per CTA of the heads that are taken together at the end

__global__ void __launch_bounds__(1024) backward_plan_kernel(const BackwardParams p, const BackwardWs L, int ctas_k, int ctas_q) {
  __shared__ int s_count[kClasses], s_warp[32], s_longest, s_shortest;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  BackwardPlan* plan = reinterpret_cast<BackwardPlan*>(p.ws + L.plan);
  int* base = reinterpret_cast<int*>(p.ws + L.base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  int before = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 1024) {
    int tiles = 0;
    if (b0 + tid < p.batch) {
      const Seq s = sequence(b0 + tid);
      if (s.ok) tiles = (s.nq + kTile - 1) / kTile;
      else set_status(&hdr->status, MLA_STATUS_BAD_SEQ_LEN);
    }
    const int sum = scan(tiles);
    if (b0 + tid < p.batch) base[b0 + tid] = before + sum - tiles;
    __syncthreads();
    if (tid == 1023) s_warp[0] = sum;
    __syncthreads();
    before += s_warp[0];
  }
  for (int side = 0; side < 2; ++side) {
    Tile* tiles = reinterpret_cast<Tile*>(p.ws + L.tiles[side]);
    __syncthreads();
    s_count[tid] = 0;
    if (tid == 0) {
      s_longest = 0;
      s_shortest = kClasses;
    }
    __syncthreads();
    for (int pass = 0; pass < 2; ++pass) {
      for (int b = warp; b < p.batch; b += 32) {
        const Seq s = sequence(b);
        if (!s.ok) continue;
        const int n = side ? s.nq : s.nk, off = s.nk - s.nq;
        for (int i = lane; i * kTile < n; i += 32) {
          Tile t;
          const int at = i * kTile;
          t.rows = min(kTile, n - at);
          t.first = 0;
          if (side == 0) {
            t.r0 = s.k0 + at;
            t.c0 = s.q0;
            t.nc = s.nq;
            t.lim = at - off;
            if (p.causal) t.first = max(0, t.lim) / kTile;
            t.steps = max(0, (s.nq + kTile - 1) / kTile - t.first);
            t.stat = base[b];
          } else {
            t.r0 = s.q0 + at;
            t.c0 = s.k0;
            t.nc = s.nk;
            t.lim = at + off + 1;
            const int sees = p.causal ? max(0, min(s.nk, t.lim + t.rows - 1)) : s.nk;   // its last row
            t.steps = (sees + kTile - 1) / kTile;
            t.stat = base[b] + i;
          }
          const int steps = min(kClasses - 1, t.steps), c = kClasses - 1 - steps;
          if (pass == 0) {
            atomicMax(&s_longest, steps);
            atomicMin(&s_shortest, steps);
          }
          const int pos = atomicAdd(&s_count[c], 1);
          if (pass == 1) {
            // (beyond the list: overlapping sequences, cu decreased somewhere)
            if (pos < L.max_tiles[side] && base[b] + (s.nq + kTile - 1) / kTile <= L.max_tiles[1]) tiles[pos] = t;
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
        // exclusive scan: s_count[c] becomes the first position of class c
        const int v = s_count[tid], x = scan(v);
        s_count[tid] = x - v;
        if (tid == 1023) {
          const int n = min(x, L.max_tiles[side]), ctas = side ? ctas_q : ctas_k, groups = side ? kHeads : kHeads / L.group;
          plan->tiles[side] = n;
          plan->next[side] = ctas;
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
// lse log2(e) and sum(d_out out) - d_lse per query tile and head, 8 heads a CTA.
__global__ void __launch_bounds__(256) backward_delta_kernel(const BackwardParams p, const BackwardWs L) {
  __shared__ float s_delta[8][kTile];
  const BackwardPlan* plan = reinterpret_cast<const BackwardPlan*>(p.ws + L.plan);
  if (static_cast<int>(blockIdx.x) >= plan->tiles[1]) return;
  const Tile t = reinterpret_cast<const Tile*>(p.ws + L.tiles[1])[blockIdx.x];
  const int h0 = 8 * blockIdx.y, lane16 = threadIdx.x & 15;
#pragma unroll 4
  for (int i = threadIdx.x >> 4; i < 8 * kTile; i += 16) {
    const int r = i >> 3, h = i & 7;
    float sum = 0.f;
    if (r < t.rows) {
      const size_t row = static_cast<size_t>(t.r0) + r;
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p.d_out + row * p.do_t + (h0 + h) * p.do_h) + lane16);
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(p.out + (row * kHeads + h0 + h) * 128) + lane16);
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum += __uint_as_float(x[e] << 16) * __uint_as_float(y[e] << 16);
        sum += __uint_as_float(x[e] & 0xFFFF0000u) * __uint_as_float(y[e] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane16 == 0) s_delta[h][r] = sum;
  }
  __syncthreads();
  float* stats = reinterpret_cast<float*>(p.ws + L.stats) + (static_cast<size_t>(t.stat) * kHeads + h0) * 2 * kTile;
  for (int i = threadIdx.x; i < 8 * kTile; i += 256) {
    const int h = i / kTile, r = i % kTile;
    float l = 0.f, d = 0.f;
    if (r < t.rows) {
      const size_t at = (static_cast<size_t>(t.r0) + r) * kHeads + h0 + h;
      l = __ldg(p.lse + at) * kLog2e;
      d = s_delta[h][r] - (p.d_lse ? __ldg(p.d_lse + at) : 0.f);
    }
    stats[h * 2 * kTile + r] = l;
    stats[h * 2 * kTile + kTile + r] = d;
  }
}

// ---------------------------------------------------------------- the two passes
struct Maps {
  CUtensorMap qn, qr, kn, kr, v, d_out;
};

// kKeys: rows are keys (dk, dv), else queries (dq).
template <bool kKeys>
__global__ void __launch_bounds__(kThreads, 1)
backward_kernel(const __grid_constant__ Maps maps, const __grid_constant__ BackwardParams p, const BackwardWs L) {
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
      if (i == SREAD || i == DPREAD || i == PREADY || i == DSREADY || i == ACCFREE) n = 8;   // one arrival a warp
      if (i == C2EMPTY && kKeys) n = 2;            // dP and dv
      if (i >= IEMPTY && i < IEMPTY + kItemSlots) n = 10;
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
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  const int causal = p.causal;

  struct Walk { int slot = 0; uint32_t phase = 0; };
  // The next item of this role's walk: its tile and first head, false when there is none.
  auto next_warp = [&](Walk& w, Tile& t, int& head) {
    if (!wait_cta_warp(BAR(IFULL + w.slot), w.phase, quit)) return false;
    const volatile int* src = reinterpret_cast<const volatile int*>(smem + kOffItems + 48 * w.slot);
    t.r0 = src[0]; t.rows = src[1]; t.c0 = src[2]; t.nc = src[3]; t.lim = src[4]; t.first = src[5]; t.steps = src[6];
    t.stat = src[7];
    head = src[8];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(IEMPTY + w.slot));
    if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
    return head >= 0;
  };

  if (smem_ok && warp == 0) {
    // ------------------------------------------------------------ items and TMA loads
    if (lane == 0) {
      const uint64_t pol = ptx::policy_evict_normal();
      const Tile* tiles = reinterpret_cast<const Tile*>(p.ws + L.tiles[kSide]);
      const int n_tiles = *reinterpret_cast<const volatile int*>(&plan->tiles[kSide]);
      const int tail = *reinterpret_cast<const volatile int*>(&plan->tail[kSide]);
      const int items = n_tiles * groups, first_late = items - n_tiles * tail;
      const float* stats = reinterpret_cast<const float*>(p.ws + L.stats);
      Walk w;
      uint32_t n = 0, n2 = 0;                  // C1 and C2 tiles queued so far
      uint32_t loads = 0, loads2 = 0;          // R1 and R2 tiles
      bool ok = true;
      // 192 values of 128 rows: queries, or keys with the shared RoPE part
      auto load_qk = [&](uint32_t dst, int bar, bool keys, int head, int row) {
        const CUtensorMap* nope = keys ? &maps.kn : &maps.qn;
        ptx::tma_load_4d(dst, nope, BAR(bar), 0, head, row, 0, pol);
        ptx::tma_load_4d(dst + kChunk, nope, BAR(bar), 64, head, row, 0, pol);
        ptx::tma_load_4d(dst + 2 * kChunk, keys ? &maps.kr : &maps.qr, BAR(bar), 0, keys ? 0 : head, row, 0, pol);
      };
      auto load_vo = [&](uint32_t dst, int bar, bool keys, int head, int row) {
        const CUtensorMap* m = keys ? &maps.v : &maps.d_out;
        ptx::tma_load_4d(dst, m, BAR(bar), 0, head, row, 0, pol);
        ptx::tma_load_4d(dst + kChunk, m, BAR(bar), 64, head, row, 0, pol);
      };
      int item = static_cast<int>(blockIdx.x);
      while (ok) {
        // head by head, and the last heads tile by tile (as in prefill)
        Tile t = {0, 0, 0, 0, 0, 0, 0, 0};
        int head0 = -1;
        if (item < items) {
          const bool late = item >= first_late;
          const int left = late ? item - first_late : item, by = late ? tail : n_tiles;
          const int q = left / by, r = left - q * by;
          t = tiles[late ? q : r];
          head0 = (late ? groups - tail + r : q) * group;
        }
        ok = wait_cta(BAR(IEMPTY + w.slot), w.phase ^ 1u, quit);
        if (!ok) break;
        volatile int* dst = reinterpret_cast<volatile int*>(smem + kOffItems + 48 * w.slot);
        dst[0] = t.r0; dst[1] = t.rows; dst[2] = t.c0; dst[3] = t.nc; dst[4] = t.lim; dst[5] = t.first; dst[6] = t.steps;
        dst[7] = t.stat;
        dst[8] = head0;
        ptx::mbar_arrive(BAR(IFULL + w.slot));
        if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
        if (head0 < 0) break;
        const int total = group * t.steps;
        for (int g = 0; g < group && ok; ++g) {
          const int head = head0 + g;
          for (int i = 0; i < t.steps && ok; ++i) {
            if (g * t.steps + i == max(total - 2, 0)) item = atomicAdd(&plan->next[kSide], 1);
            if (i == 0) {
              ok = wait_cta(BAR(R1EMPTY), (loads & 1u) ^ 1u, quit);
              if (!ok) break;
              ++loads;
              ptx::mbar_arrive_expect_tx(BAR(R1FULL), 3 * kChunk);
              load_qk(sbase + kOffR1, R1FULL, kKeys, head, t.r0);
            }
            const int col = t.c0 + (t.first + i) * kTile;
            const uint32_t buf = n & 1u;
            ok = wait_cta(BAR(C1EMPTY + buf), ((n >> 1) & 1u) ^ 1u, quit);
            if (ok) {
              ptx::mbar_arrive_expect_tx(BAR(C1FULL + buf), 3 * kChunk + (kKeys ? kStatBytes : 0u));
              load_qk(sbase + kOffC1 + buf * 3 * kChunk, C1FULL + buf, !kKeys, head, col);
              if constexpr (kKeys)
                ptx::bulk_load(sbase + kOffStats + buf * kStatBytes,
                               stats + (static_cast<size_t>(t.stat + t.first + i) * kHeads + head) * 2 * kTile, kStatBytes,
                               BAR(C1FULL + buf), pol);
            }
            if (ok) ++n;
            if (i == 0 && ok) {
              ok = wait_cta(BAR(R2EMPTY), (loads2 & 1u) ^ 1u, quit);
              if (ok) {
                ++loads2;
                ptx::mbar_arrive_expect_tx(BAR(R2FULL), 2 * kChunk);
                load_vo(sbase + kOffR2, R2FULL, kKeys, head, t.r0);
              }
            }
            if (ok) ok = wait_cta(BAR(C2EMPTY), (n2 & 1u) ^ 1u, quit);
            if (ok) {
              ++n2;
              ptx::mbar_arrive_expect_tx(BAR(C2FULL), 2 * kChunk);
              load_vo(sbase + kOffC2, C2FULL, !kKeys, head, col);
            }
          }
        }
        if (t.steps == 0) item = atomicAdd(&plan->next[kSide], 1);
      }
      // no copy may land after the CTA has left: wait for the last phase armed on each barrier
#pragma unroll 1
      for (int b = 0; b < 5; ++b) {
        const uint32_t count = b == 0 ? loads : b == 1 ? loads2 : b == 2 ? n2 : (n + 4u - static_cast<uint32_t>(b)) / 2u;
        const int bar = b == 0 ? R1FULL : b == 1 ? R2FULL : b == 2 ? C2FULL : C1FULL + b - 3;
        if (count > 0) wait_issued(BAR(bar), (count - 1) & 1u, quit);
      }
    }
  } else if (smem_ok && warp == 1) {
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
          if (ok) ok = wait_cta_warp(BAR(C1FULL + buf), (n >> 1) & 1u, quit);
          // S's place: the last dP has been read from it (keys), or the last S
          if (ok && n > 0) ok = wait_cta_warp(BAR(kKeys ? DPREAD : SREAD), (n - 1) & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          issued = true;
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 3; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                ptx::mma_ss(tmem + kX, r1 + c * kChunkD + 2u * k, c1 + (3u * buf + c) * kChunkD + 2u * k, kIdescS,
                            (c > 0 || k > 0) ? 1u : 0u);
            ptx::mma_commit(BAR(SFULL));
            if (i == steps - 1) ptx::mma_commit(BAR(R1EMPTY));
          }
          __syncwarp();
          if (i == 0) ok = wait_cta_warp(BAR(R2FULL), loads & 1u, quit);
          if (ok) ok = wait_cta_warp(BAR(C2FULL), n & 1u, quit);
          if (ok && (kKeys || n > 0)) ok = wait_cta_warp(BAR(kKeys ? SREAD : DPREAD), (kKeys ? n : n - 1) & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                ptx::mma_ss(tmem + kDp, r2 + c * kChunkD + 2u * k, c2 + c * kChunkD + 2u * k, kIdescS,
                            (c > 0 || k > 0) ? 1u : 0u);
            ptx::mma_commit(BAR(DPFULL));
            ptx::mma_commit(BAR(C2EMPTY));
            if (i == steps - 1) ptx::mma_commit(BAR(R2EMPTY));
          }
          __syncwarp();
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
    while (ok && next_warp(w, t, head)) {
      const int steps = __shfl_sync(0xffffffffu, t.steps, 0);
      for (int g = 0; g < group && ok; ++g) {
        for (int i = 0; i < steps && ok; ++i, ++n) {
          const uint32_t buf = n & 1u;
          const int valid = __shfl_sync(0xffffffffu, t.nc - (t.first + i) * kTile, 0);
          // a head's first products overwrite the accumulators: they must have been read
          if (i == 0) ok = wait_cta_warp(BAR(ACCFREE), (heads & 1u) ^ 1u, quit);
          if constexpr (kKeys) {
            if (ok) ok = wait_cta_warp(BAR(C2FULL), n & 1u, quit);
            if (ok) ok = wait_cta_warp(BAR(PREADY), n & 1u, quit);
            if (!ok) break;
            if (valid < kTile) clear(kOffC2, 2, valid);
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
          if (ok) ok = wait_cta_warp(BAR(C1FULL + buf), (n >> 1) & 1u, quit);
          if (ok) ok = wait_cta_warp(BAR(DSREADY), n & 1u, quit);
          if (!ok) break;
          if (valid < kTile) clear(kOffC1 + buf * 3 * kChunk, 3, valid);
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
    if (issued && elect_one()) {
      ptx::mma_commit(BAR(DRAIN + 1));
      wait_issued(BAR(DRAIN + 1), 0u, quit);
    }
    __syncwarp();
  } else if (smem_ok && warp >= 4) {
    // ------------------------------------------------------------ P and dS (thread = half a row), results
    const int half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t x_addr = tmem + lane_base + kX + 64u * half, dp_addr = tmem + lane_base + kDp + 64u * half;
    const uint32_t y_addr = tmem + lane_base + kY + 32u * half;
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
    // 16 bf16 values to 32 bytes at dst (16-byte aligned)
    auto store16 = [&](__nv_bfloat16* dst, const uint32_t* v) {
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    };
    // 32 accumulator columns as bf16
    auto read32 = [&](uint32_t col, float mul, uint32_t* out16) {
      uint32_t a[32];
      ptx::tmem_ld32(tmem + lane_base + col, a);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(a[2 * e]) * mul, __uint_as_float(a[2 * e + 1]) * mul);
        out16[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
    };
    while (ok && next_warp(w, t, head0)) {
      const size_t row = static_cast<size_t>(t.r0) + r;
      const bool mine = r < t.rows;
      for (int g = 0; g < group && ok; ++g) {
        const int head = head0 + g;
        float row_lse = 0.f, row_delta = 0.f;
        if constexpr (!kKeys) {
          const float* st = reinterpret_cast<const float*>(p.ws + L.stats) + (static_cast<size_t>(t.stat) * kHeads + head) * 2 * kTile;
          row_lse = st[r];
          row_delta = st[kTile + r];
        }
        for (int i = 0; i < t.steps; ++i, ++n) {
          const uint32_t buf = n & 1u;
          // columns [lo, hi) of this thread's 64 are seen
          const int at = (t.first + i) * kTile + 64 * half;
          int lo = 0, hi = t.nc - at;
          if (causal) {
            if constexpr (kKeys) lo = t.lim + r - at;
            else hi = min(hi, t.lim + r - at);
          }
          const bool all = __all_sync(0xffffffffu, lo <= 0 && hi >= 64);
          ok = wait_cta_warp(BAR(SFULL), n & 1u, quit);
          if (ok && kKeys) ok = wait_cta_warp(BAR(C1FULL + buf), (n >> 1) & 1u, quit);   // the statistics
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t s[64], pk[32];
          ptx::tmem_ld32(x_addr, s);
          ptx::tmem_ld32(x_addr + 32u, s + 32);
          ptx::tmem_wait_ld();
          arrive(SREAD);
          const float4* lse4 = reinterpret_cast<const float4*>(smem + kOffStats + buf * kStatBytes) + 16 * half;
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            float4 l = make_float4(row_lse, row_lse, row_lse, row_lse);
            if constexpr (kKeys) l = lse4[e / 4];
            s[e] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(s[e]), c, -l.x)));
            s[e + 1] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(s[e + 1]), c, -l.y)));
            s[e + 2] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(s[e + 2]), c, -l.z)));
            s[e + 3] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(s[e + 3]), c, -l.w)));
          }
          if (!all) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (e < lo || e >= hi) s[e] = 0u;
          }
          if constexpr (kKeys) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
              pk[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            // the last step's dS has been read
            if (n > 0) ok = wait_cta_warp(BAR(DSDONE), (n - 1) & 1u, quit);
            if (!ok) break;
            ptx::tc_fence_after();
            ptx::tmem_st32(y_addr, pk);
            ptx::tmem_wait_st();
            arrive(PREADY);
          }
          ok = wait_cta_warp(BAR(DPFULL), n & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          const float4* delta4 = lse4 + kTile / 4;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t d[32];
            ptx::tmem_ld32(dp_addr + 32u * q, d);
            ptx::tmem_wait_ld();
            if (q == 1) arrive(DPREAD);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float4 m = make_float4(row_delta, row_delta, row_delta, row_delta);
              if constexpr (kKeys) m = delta4[8 * q + e / 4];
              const uint32_t* x = s + 32 * q + e;
              float y0 = __uint_as_float(x[0]) * (__uint_as_float(d[e]) - m.x), y1 = __uint_as_float(x[1]) * (__uint_as_float(d[e + 1]) - m.y);
              float y2 = __uint_as_float(x[2]) * (__uint_as_float(d[e + 2]) - m.z), y3 = __uint_as_float(x[3]) * (__uint_as_float(d[e + 3]) - m.w);
              if (!all) {                    // (0 times what is not finite)
                const int k = 32 * q + e;
                if (k < lo || k >= hi) y0 = 0.f;
                if (k + 1 < lo || k + 1 >= hi) y1 = 0.f;
                if (k + 2 < lo || k + 2 >= hi) y2 = 0.f;
                if (k + 3 < lo || k + 3 >= hi) y3 = 0.f;
              }
              const __nv_bfloat162 a = __floats2bfloat162_rn(y0, y1), b = __floats2bfloat162_rn(y2, y3);
              pk[16 * q + e / 2] = *reinterpret_cast<const uint32_t*>(&a);
              pk[16 * q + e / 2 + 1] = *reinterpret_cast<const uint32_t*>(&b);
            }
          }
          // P (keys), or the last step's dS, has been read
          if (kKeys) ok = wait_cta_warp(BAR(PDONE), n & 1u, quit);
          else if (n > 0) ok = wait_cta_warp(BAR(DSDONE), (n - 1) & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
          ptx::tmem_st32(y_addr, pk);
          ptx::tmem_wait_st();
          arrive(DSREADY);
        }
        if (!ok) break;
        // results of the head
        const bool last = g == group - 1;
        uint32_t nope[32], second[32], rope[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) nope[e] = second[e] = rope[e] = 0;
        if (t.steps > 0) {
          ok = wait_cta_warp(BAR(DSDONE), (n - 1) & 1u, quit);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            read32(kAcc1 + 64u * half + 32u * q, p.scale, nope + 16 * q);
            if constexpr (kKeys) read32(kAcc2 + 64u * half + 32u * q, 1.f, second + 16 * q);
          }
          if constexpr (kKeys) {
            if (last) {
              ptx::tmem_ld32(tmem + lane_base + kAcc1 + 128u + 32u * half, rope);
              ptx::tmem_wait_ld();
            }
          } else {
            read32(kAcc1 + 128u + 32u * half, p.scale, rope);
          }
          arrive(ACCFREE);
        }
        if (mine) {
          __nv_bfloat16* dst = kKeys ? p.dk_nope + row * p.dkn_t + head * p.dkn_h : p.dq_nope + row * p.dqn_t + head * p.dqn_h;
#pragma unroll
          for (int q = 0; q < 4; ++q) store16(dst + 64 * half + 16 * q, nope + 8 * q);
          if constexpr (kKeys) {
#pragma unroll
            for (int q = 0; q < 4; ++q) store16(p.dv + row * p.dv_t + head * p.dv_h + 64 * half + 16 * q, second + 8 * q);
            if (last) {
              float* part = reinterpret_cast<float*>(p.ws + L.rope) +
                            (static_cast<size_t>(head0 / group) * p.nk + row) * kDr + 32 * half;
#pragma unroll
              for (int q = 0; q < 4; ++q) ptx::st_global_v8(part + 8 * q, rope + 8 * q);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) store16(p.dq_rope + row * p.dqr_t + head * p.dqr_h + 32 * half + 16 * q, rope + 8 * q);
          }
        }
      }
    }
  }
  // ------------------------------------------------------------ teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *quit != 0) set_status(&hdr->status, MLA_STATUS_TIMEOUT);
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- RoPE part of dk
// The groups' sums of a key tile, in the groups' order; a thread has four values.
__global__ void __launch_bounds__(256) backward_rope_kernel(const BackwardParams p, const BackwardWs L) {
  const BackwardPlan* plan = reinterpret_cast<const BackwardPlan*>(p.ws + L.plan);
  if (static_cast<int>(blockIdx.x) >= plan->tiles[0]) return;
  const Tile t = reinterpret_cast<const Tile*>(p.ws + L.tiles[0])[blockIdx.x];
  const int r = blockIdx.y * 16 + (threadIdx.x >> 4), d = 4 * (threadIdx.x & 15);
  if (r >= t.rows) return;
  const size_t row = static_cast<size_t>(t.r0) + r;
  const float* part = reinterpret_cast<const float*>(p.ws + L.rope) + row * kDr + d;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int g = 0; g < kHeads / L.group; ++g) {
    const float4 x = *reinterpret_cast<const float4*>(part + static_cast<size_t>(g) * p.nk * kDr);
    sum.x += x.x;
    sum.y += x.y;
    sum.z += x.z;
    sum.w += x.w;
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(sum.x * p.scale, sum.y * p.scale);
  const __nv_bfloat162 b = __floats2bfloat162_rn(sum.z * p.scale, sum.w * p.scale);
  *reinterpret_cast<uint2*>(p.dk_rope + row * p.dkr_t + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

}  // namespace

cudaError_t launch_backward(PFN_cuTensorMapEncodeTiled_v12000 encode, const BackwardParams& p, int sms,
                            cudaStream_t stream) {
  const BackwardWs L = backward_ws(p.batch, p.nq, p.nk);
  Maps maps;
  // with no row at all nothing is loaded; the maps still need one
  const int nq = p.nq > 0 ? p.nq : 1, nk = p.nk > 0 ? p.nk : 1;
  if (!encode_map(encode, &maps.qn, p.q_nope, 128, kHeads, nq, p.qn_t, p.qn_h, kTile) ||
      !encode_map(encode, &maps.qr, p.q_rope, 64, kHeads, nq, p.qr_t, p.qr_h, kTile) ||
      !encode_map(encode, &maps.kn, p.k_nope, 128, kHeads, nk, p.kn_t, p.kn_h, kTile) ||
      !encode_map(encode, &maps.kr, p.k_rope, 64, 1, nk, p.kr_t, 64, kTile) ||
      !encode_map(encode, &maps.v, p.v, 128, kHeads, nk, p.v_t, p.v_h, kTile) ||
      !encode_map(encode, &maps.d_out, p.d_out, 128, kHeads, nq, p.do_t, p.do_h, kTile))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> configured_k{0}, configured_q{0};
  cudaError_t e = allow_smem(backward_kernel<true>, kSmem, configured_k);
  if (e == cudaSuccess) e = allow_smem(backward_kernel<false>, kSmem, configured_q);
  if (e != cudaSuccess) return e;
  const long long items_k = static_cast<long long>(L.max_tiles[0]) * (kHeads / L.group);
  const long long items_q = static_cast<long long>(L.max_tiles[1]) * kHeads;
  const int ctas_k = static_cast<int>(items_k < sms ? items_k : sms), ctas_q = static_cast<int>(items_q < sms ? items_q : sms);
  e = launch_kernel(backward_plan_kernel, dim3(1), dim3(1024), 0, stream, p, L, ctas_k, ctas_q);
  if (e == cudaSuccess && ctas_q)
    e = launch_kernel(backward_delta_kernel, dim3(L.max_tiles[1], kHeads / 8), dim3(256), 0, stream, p, L);
  if (e == cudaSuccess && ctas_q)
    e = launch_kernel(backward_kernel<false>, dim3(ctas_q), dim3(kThreads), kSmem, stream, maps, p, L);
  if (e == cudaSuccess && ctas_k)
    e = launch_kernel(backward_kernel<true>, dim3(ctas_k), dim3(kThreads), kSmem, stream, maps, p, L);
  if (e == cudaSuccess && ctas_k)
    e = launch_kernel(backward_rope_kernel, dim3(L.max_tiles[0], kTile / 16), dim3(256), 0, stream, p, L);
  return e;
}

}  // namespace mla
