// Expanded-form MLA attention over ragged sequences (prefill).
//
// For query row i of a sequence with nq queries and nk keys, and head h:
//     s_j = scale (q_nope_i . k_nope_j + q_rope_i . k_rope_j)
//     out_i = sum_j softmax_j(s) v_j,   lse_i = ln sum_j exp(s_j)
// over the keys j it sees: all nk, or with the causal mask j <= i + nk - nq
// (the queries are the sequence's last nq tokens).  A row that sees no key
// gets out = 0, lse = -inf.  The RoPE part of a key is shared by all heads
// and read as it is, never copied into a per-head key.
//
// Bound: 2 * 128 * (192 + 128) operations per visible (query, key) pair
// against 512 bytes of K and V per key and head, so with 256 query rows per
// K/V read the tensor cores bound it.  One pass over the keys with a running
// maximum and sum; S, P and O never leave the SM.
//
// One persistent CTA per SM, work items (head, 256 query rows) handed out by
// a counter, head by head (a head's K and V are then in L2 while its tiles
// run) and within a head the longest tiles first; the last heads, about five
// items a CTA, are taken together, so that the longest tiles of the last one do
// not start when everything else is done (4096 causal tokens 499 and 456 us,
// 2048 155 and 134, 8 x up to 256 over up to 4096 290 and 235).  Not where all
// tiles are about as long: there is nothing to balance, and the tiles of a head
// that run together share its K and V in L2.  There the last round's items go
// out in halves if it would leave half of the SMs idle (2 x 512 queries over
// 15,000 keys 879 and 815 us).  An item's rows are two
// M = 128 tiles that share each K/V tile of 80 keys:
//   tensor memory (512 columns): O0 | O1 (128 fp32 columns each), S0 | S1 (80
//       each), P0 | P1 (bf16, 40 each);
//   shared memory: Q0 | Q1 (48 KiB each), two K tiles (three 10-KiB chunks of 80
//       keys x 64 values each) and three V tiles (two chunks each);
//   warp 0 fetches the items and issues the TMA loads, warps 1 and 2 the
//   scores' MMAs of tile 0 and tile 1, warp 3 the P.V MMAs of both, warps
//   4..7 and 8..11 are the softmax of tile 0 and tile 1 (thread = row), warps
//   12..15 write the output of both.
//
// Why 80 keys.  With P beside S instead of in its place, S of the next step
// can be computed as soon as the softmax has read this one into registers,
// so the tensor cores never wait for a softmax; 2 (128 + N + N/2) columns fit
// the 512 up to N = 80.  An S MMA with N = 80 costs 52 cycles instead of the
// 40 its size would take, so a step of two tiles costs 23.2 cycles a key
// against 20 with N = 128 (1852 and 2566 cycles a step, measured alone); but
// with N = 128 P must replace S, the chain S, softmax, P.V is then serial
// for each tile and took 29 cycles a key (8192 causal 2.01 ms).
//
// Three warps issue MMAs because one cannot keep the pipe busy: a wait costs it
// 100 cycles or more even when its phase is complete, the pipe queues only a
// few MMAs, and one warp's waits and loop took about 1350 cycles of a step
// beside its MMAs (MMAs that several warps interleave run at full rate: 1871
// against 1852 cycles a step).  The step after an item's last is the next
// item's first, so items overlap, and the output warps drain O while the next
// item runs.
//
// The maximum is lazy: a row's reference moves only when a tile's maximum
// exceeds it by more than 2^kLazy, so O is rescaled rarely; its softmax warps
// do that themselves, after the previous P.V of the tile has completed.
//
// K and V have rings of their own: in one ring a K tile waited for the V tile
// whose slots it reused, which is read 600 cycles later (8192 causal 1.85 ms in
// a loop against 1.62; with two V tiles instead of three 1.95).
//
// Measured: 8192 causal tokens 1.47 to 1.52 ms (1815 to 1870 TFLOP/s; 1.6 to 1.7 in a
// loop of seconds, under the power cap), eight prompts of 54 to 1523 tokens 227 to
// 250 us by machine (1000 to 1100; HBM alone takes 130), 2 x 512 queries over 15,000
// keys 785 to 870 us (1630 to 1470), five prompts of up to 33 tokens 18.6 us.  An
// item's queries land about 1900 cycles after the last item's scores: a second
// copy of 256 of them does not fit beside K and V.  (An item of 128 rows or fewer
// uses query tile 0 alone, and waits for it although tile 1's half idles.)  Tried
// and no faster: K and V ahead of the queries (0 to 3 % either way), prefetches of
// K and V into L2 (3 % slower on ragged prompts).
//
// Every wait is bounded: after a timeout all roles of the CTA leave, and it ends
// through its teardown, which records MLA_STATUS_TIMEOUT.
#include <climits>

#include "prefill.cuh"
#include "waits.cuh"

namespace mla {

namespace {

constexpr int kThreads = 512;
constexpr int kKeys = 80;                          // keys per K/V tile
constexpr uint32_t kQChunk = 128u * 128u;          // 16 KiB: 128 query rows x 64 values
constexpr uint32_t kQTile = 3 * kQChunk;           // 128 query rows x 192
constexpr uint32_t kChunk = kKeys * 128u;          // 10 KiB: 80 keys x 64 values
constexpr uint32_t kKTiles = 2, kVTiles = 3;       // K and V tiles held
constexpr uint32_t kKTile = 3 * kChunk, kVTile = 2 * kChunk;
constexpr uint32_t kOffK = 2 * kQTile;
constexpr uint32_t kOffV = kOffK + kKTiles * kKTile;
constexpr uint32_t kOffBar = kOffV + kVTiles * kVTile;    // 216 KiB
constexpr int kItemSlots = 2;
constexpr int kHalvesFrom = 8;                     // K tiles from which a last round's items are halved
constexpr int kTailItems = 5;                      // items per CTA of the heads that are taken together at the end
enum Bar {
  QFULL = 0, QEMPTY = QFULL + 2, KFULL = QEMPTY + 2, KEMPTY = KFULL + kKTiles, VFULL = KEMPTY + kKTiles,
  VEMPTY = VFULL + kVTiles, SFULL = VEMPTY + kVTiles, SREAD = SFULL + 2,
  PREADY = SREAD + 2, PVDONE = PREADY + 2, LFULL = PVDONE + 2, LEMPTY = LFULL + 2, OFREE = LEMPTY + 2,
  IFULL = OFREE + 2, IEMPTY = IFULL + kItemSlots, DRAIN = IEMPTY + kItemSlots, VASK = DRAIN + 3,
  NBAR = VASK + 2 * kVTiles
};
constexpr uint32_t kOffTmem = kOffBar + 8 * NBAR;
constexpr uint32_t kOffItems = (kOffTmem + 16 + 15) & ~15u;     // kItemSlots x 32 bytes
constexpr uint32_t kOffInv = kOffItems + 32 * kItemSlots;       // fp32 1/l [2 tiles][128 rows]
constexpr uint32_t kOffQuit = kOffInv + 2 * 128 * 4;            // uint32: a wait gave up
// the second pass (see clean): the number of an item with values that were taken
// out, and the first key of each column with +inf and with -inf; for three items,
// because a role is at most two ahead of another
constexpr uint32_t kOffFound = kOffQuit + 16;                   // uint32 [3], padded
constexpr uint32_t kOffFirst = kOffFound + 16;                  // uint64 [3][2 signs][128 columns]
constexpr uint32_t kSmem = kOffFirst + 3 * 2 * 128 * 8;
static_assert(kOffFirst % 8 == 0, "alignment");
static_assert(kSmem <= 232448, "shared memory budget");

constexpr uint32_t kOCol = 0, kSCol = 256, kPCol = kSCol + 2 * kKeys;   // + 128 t, kKeys t, kKeys / 2 t
static_assert(kPCol + kKeys <= 512, "tensor memory columns");
constexpr uint32_t kIdescS = ptx::idesc_bf16(128, kKeys, 0, 0);  // Q, K: K-major
constexpr uint32_t kIdescPV = ptx::idesc_bf16(128, 128, 0, 1);   // P in tensor memory, V: MN-major
// log2 units: P <= 2^12, exact in relative terms, and far from fp32 overflow in O and l
constexpr float kLazy = 12.0f;
constexpr float kLn2 = 0.69314718055994530942f;

// The header's n_tiles are the tiles in the list, chunk the next work item after
// each CTA's first.
struct Tile {
  int q0, rows;   // first packed query row, query rows (1..256)
  int k0, nk;     // first packed key, keys of the sequence
  int lim;        // keys that row 0 sees before clamping to nk (row r: lim + r if causal)
  int head;       // filled in for a fetched item; -1: no more items
  int index;      // of the tile in the list, filled in too
  int pad;
};
static_assert(sizeof(Tile) == 32, "tile record");

__device__ __forceinline__ int visible(const Tile& t, int r, int causal) {
  return max(0, min(t.nk, t.lim + (causal ? r : 0)));
}
// K/V tiles that query tile t of the item visits (the last of its rows sees the most)
__device__ __forceinline__ int kv_tiles(const Tile& t, int half, int causal) {
  if (t.rows <= 128 * half) return 0;
  return (visible(t, min(t.rows, 128 * (half + 1)) - 1, causal) + kKeys - 1) / kKeys;
}

// ---------------------------------------------------------------- plan
// One CTA: the list of 256-row tiles of all sequences, the ones with most K/V
// tiles first (counting sort over the clipped tile count; the order within a
// class does not matter, every item is computed on its own).
constexpr int kClasses = 1024;

__global__ void __launch_bounds__(1024) prefill_plan_kernel(const int32_t* __restrict__ cu_q,
                                                            const int32_t* __restrict__ cu_k, int batch, int nq, int nk,
                                                            int causal, int first, uint8_t* __restrict__ ws, PrefillWs L) {
  __shared__ int s_count[kClasses];
  __shared__ int s_warp[32];
  __shared__ int s_longest, s_shortest;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(ws);
  Tile* tiles = reinterpret_cast<Tile*>(ws + L.tiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  s_count[tid] = 0;
  if (tid == 0) {
    s_longest = 0;
    s_shortest = kClasses;
  }
  ptx::grid_dep_launch();   // the attention kernel may set itself up; it waits for this grid before it reads the list
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int b = warp; b < batch; b += 32) {
      const int q0 = __ldg(cu_q + b), q1 = __ldg(cu_q + b + 1), k0 = __ldg(cu_k + b), k1 = __ldg(cu_k + b + 1);
      if (q0 < 0 || q1 < q0 || q1 > nq || k0 < 0 || k1 < k0 || k1 > nk) {
        if (lane == 0 && pass == 0) set_status(&hdr->status, MLA_STATUS_BAD_SEQ_LEN);
        continue;
      }
      const int n_q = q1 - q0, n_k = k1 - k0;
      for (int i = lane; i * kPrefillTile < n_q; i += 32) {
        Tile t;
        t.q0 = q0 + i * kPrefillTile;
        t.rows = min(kPrefillTile, n_q - i * kPrefillTile);
        t.k0 = k0;
        t.nk = n_k;
        t.lim = causal ? i * kPrefillTile + 1 + (n_k - n_q) : n_k;
        t.head = t.index = t.pad = 0;
        const int steps = min(kClasses - 1, max(kv_tiles(t, 0, causal), kv_tiles(t, 1, causal)));
        const int c = kClasses - 1 - steps;
        if (pass == 0) {
          atomicMax(&s_longest, steps);
          atomicMin(&s_shortest, steps);
        }
        const int pos = atomicAdd(&s_count[c], 1);
        if (pass == 1) {
          if (pos < L.max_tiles) {
            tiles[pos] = t;
            reinterpret_cast<uint4*>(ws + L.again)[pos] = make_uint4(0, 0, 0, 0);
          }
          else set_status(&hdr->status, MLA_STATUS_BAD_SEQ_LEN);   // overlapping sequences: cu_q decreased somewhere
        }
      }
    }
    __syncthreads();
    if (pass == 0) {
      // exclusive scan: s_count[c] becomes the first position of class c
      const int v = s_count[tid];
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_warp[warp] = x;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < warp; ++w) before += s_warp[w];
      s_count[tid] = before + x - v;
      if (tid == 1023) {
        const int n_tiles = min(before + x, L.max_tiles);
        hdr->n_tiles = n_tiles;
        hdr->chunk = first;
        // heads taken together at the end: one where all tiles are about as long.
        // There, if the last round would leave half of the CTAs idle and its items
        // are not short, they go out as two halves of 128 rows.
        const bool even = 2 * s_longest <= 3 * s_shortest;
        const int items = n_tiles * kHeads, rest = items % first;
        hdr->prefill_tail = even ? 1 : min(kHeads, (kTailItems * first + n_tiles - 1) / max(n_tiles, 1));
        hdr->prefill_halves = even && s_longest >= kHalvesFrom && 2 * rest <= first ? items - rest : INT_MAX;
        hdr->prefill_again = 0;
        hdr->abort_flag = 0;
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- attention
struct Maps {
  CUtensorMap qn, qr, kn, kr, v;
};

// Registers (128 a thread at launch): 72 for warps 0..3, 104 for the output
// warps, 168 for the softmax warps (4 * 72 + 4 * 104 + 8 * 168 = 16 * 128),
// each role's branch setting its own.
__device__ __forceinline__ void regs_issue() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
__device__ __forceinline__ void regs_output() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }
__device__ __forceinline__ void regs_softmax() { asm volatile("setmaxnreg.inc.sync.aligned.u32 168;"); }

// 32 lanes x 8 columns to tensor memory.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Maximum of a row's scores.
__device__ __forceinline__ float row_max(const uint32_t* s) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
  for (int e = 8; e < kKeys; e += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max3(m[i], __uint_as_float(s[e + 2 * i]), __uint_as_float(s[e + 2 * i + 1]));
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// sum += a b in bf16 pairs: not finite once a value was not.  (In its place behind
// the stores, which the compiler delays for it otherwise.)
__device__ __forceinline__ void add_product(uint32_t& sum, uint32_t a, uint32_t b) {
  asm volatile("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(a), "r"(b));
}

// A key that a row does not see has P = 0 there, which an infinity or a NaN in
// its V turns into NaN.  Looking for such values in every V tile at the mask's
// diagonal took up to half of a short item's time (64 prompts of up to 512 tokens
// 474 and 690 us), so they are looked for in the results: a tile and head with a
// row whose sum of weights is finite and whose output is not is marked, and done
// once more by a second launch of the kernel, which returns at once if there is
// none.  It runs this function over each V tile before its P.V.
//
// Rows [lo, hi) of a V tile, keys k0 + row of the sequence, by the 128 threads of
// a query tile's softmax: values that are not finite become 0, and `first` takes
// the smallest key of each column with +inf and with -inf (a NaN counts as both)
// under the item's number: `tag` has its complement in the high half, so that an
// entry of a later item is smaller and none needs a reset.  The output gives them
// back to the rows that see the key.  True if this thread found any.  (The other
// query tile's threads may do the same at the same time.)
__device__ __forceinline__ bool clean(uint8_t* tile, int lo, int hi, int k0, int tid, uint64_t tag,
                                      unsigned long long* first) {
  bool found = false;
#pragma unroll 1
  for (int i = 0; i < kKeys / 16 * 2 * 8; ++i) {     // (row, chunk, value) of this thread's share
    const int r = lo + (tid >> 3) + 16 * (i >> 4), c = (i >> 3) & 1, e = i & 7;
    if (r >= hi) break;
    volatile uint16_t* at = reinterpret_cast<volatile uint16_t*>(tile + c * kChunk + r * 128 + (tid & 7) * 16) + e;
    const uint32_t v = *at;
    if ((v & 0x7F80u) != 0x7F80u) continue;
    const bool nan = (v & 0x7Fu) != 0;
    unsigned long long* entry = first + 64 * c + 8 * ((tid & 7) ^ (r & 7)) + e;   // 128-byte swizzle
    if (nan || v < 0x8000u) atomicMin(entry, tag | static_cast<uint32_t>(k0 + r));
    if (nan || v >= 0x8000u) atomicMin(entry + 128, tag | static_cast<uint32_t>(k0 + r));
    *at = 0;
    found = true;
  }
  return found;
}

// kAgain: the second pass, over the items that the first one marked.
template <bool kAgain>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ Maps maps, const PrefillParams p, const PrefillWs L) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  // (through a shuffle, so that it counts as warp-uniform: an MMA whose operands
  // depend on it otherwise takes about 90 cycles to issue instead of 24)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  if constexpr (kAgain) {
    ptx::grid_dep_wait();
    if (*reinterpret_cast<const volatile int*>(&hdr->prefill_again) == 0) return;   // nothing was marked
  }
  volatile uint32_t* const quit = reinterpret_cast<volatile uint32_t*>(smem + kOffQuit);
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  if (threadIdx.x == 0) {
    *quit = 0;
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(BAR(QFULL + t), 1);
      ptx::mbar_init(BAR(QEMPTY + t), 1);
      ptx::mbar_init(BAR(SFULL + t), 1);
      ptx::mbar_init(BAR(SREAD + t), 4);           // one arrival a warp: softmax
      ptx::mbar_init(BAR(PREADY + t), 4);
      ptx::mbar_init(BAR(PVDONE + t), 1);
      ptx::mbar_init(BAR(LFULL + t), 4);
      ptx::mbar_init(BAR(LEMPTY + t), 4);          // output warps
      ptx::mbar_init(BAR(OFREE + t), 4);
      ptx::mbar_init(BAR(DRAIN + t), 1);
    }
    ptx::mbar_init(BAR(DRAIN + 2), 1);
    for (uint32_t s = 0; s < kKTiles; ++s) { ptx::mbar_init(BAR(KFULL + s), 1); ptx::mbar_init(BAR(KEMPTY + s), 2); }
    for (uint32_t s = 0; s < kVTiles; ++s) { ptx::mbar_init(BAR(VFULL + s), 1); ptx::mbar_init(BAR(VEMPTY + s), 1); }
    for (uint32_t s = 0; s < 2 * kVTiles; ++s) ptx::mbar_init(BAR(VASK + s), 1);
    for (int s = 0; s < kItemSlots; ++s) {
      ptx::mbar_init(BAR(IFULL + s), 1);
      ptx::mbar_init(BAR(IEMPTY + s), 15);         // three MMA, eight softmax, four output warps
    }
    ptx::fence_barrier_init();
  }
  if (kAgain && warp == 1) {                         // (items are numbered from 1)
    for (int i = lane; i < 3 * 2 * 128; i += 32) reinterpret_cast<unsigned long long*>(smem + kOffFirst)[i] = ~0ull;
    if (lane < 3) reinterpret_cast<uint32_t*>(smem + kOffFound)[lane] = 0;
  }
  if (warp == 2) {
    ptx::tmem_alloc(sbase + kOffTmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem), 0);
  // everything above overlaps the plan kernel, whose list is read from here on
  if constexpr (!kAgain) {
    ptx::grid_dep_wait();
    if (p.causal) ptx::grid_dep_launch();   // the second pass may be launched where a CTA has left
  }
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  const int causal = p.causal;

  // The next item of this role's walk: false when there is none (or a wait
  // gave up).  Each consumer reads the record and then releases its slot.
  struct Walk { int slot = 0; uint32_t phase = 0; };
  auto read_item = [&](Walk& w, Tile& t) {
    const volatile int* src = reinterpret_cast<const volatile int*>(smem + kOffItems + 32 * w.slot);
    t.q0 = src[0]; t.rows = src[1]; t.k0 = src[2]; t.nk = src[3]; t.lim = src[4]; t.head = src[5]; t.index = src[6];
  };
  auto next_warp = [&](Walk& w, Tile& t) {
    if (!wait_cta_warp(BAR(IFULL + w.slot), w.phase, quit)) { t.head = -1; t.nk = 0; return false; }
    read_item(w, t);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(IEMPTY + w.slot));
    if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
    return t.head >= 0;
  };

  if (smem_ok && warp == 0) {
    // ------------------------------------------------------------ items and TMA loads
    regs_issue();
    if (lane == 0) {
      const uint64_t pol = ptx::policy_evict_normal();
      Walk w;
      uint32_t kb = 0, k_phase = 0, vb = 0, v_phase = 0;   // next K and V buffer
      uint32_t k_tiles = 0, v_tiles = 0;       // tiles queued so far
      uint32_t nq0 = 0, nq1 = 0;               // Q tiles queued so far
      bool ok = true;
      auto query = [&](int t, uint32_t n, const Tile& it) {
        ok = wait_cta(BAR(QEMPTY + t), (n & 1u) ^ 1u, quit);
        if (!ok) return;
        ptx::mbar_arrive_expect_tx(BAR(QFULL + t), kQTile);
        const uint32_t dst = sbase + static_cast<uint32_t>(t) * kQTile;
        const int row = it.q0 + 128 * t;
        ptx::tma_load_4d(dst, &maps.qn, BAR(QFULL + t), 0, it.head, row, 0, pol);
        ptx::tma_load_4d(dst + kQChunk, &maps.qn, BAR(QFULL + t), 64, it.head, row, 0, pol);
        ptx::tma_load_4d(dst + 2 * kQChunk, &maps.qr, BAR(QFULL + t), 0, it.head, row, 0, pol);
      };
      const Tile* tiles = reinterpret_cast<const Tile*>(p.ws + L.tiles);
      const int n_tiles = *reinterpret_cast<const volatile int*>(&hdr->n_tiles);
      const int tail = *reinterpret_cast<const volatile int*>(&hdr->prefill_tail);
      const int first_half = *reinterpret_cast<const volatile int*>(&hdr->prefill_halves);
      const int items = n_tiles * kHeads, first_late = items - n_tiles * tail;
      auto record = [&](int item) {
        Tile t;
        t.q0 = t.rows = t.k0 = t.nk = t.lim = t.index = 0;
        t.head = -1;
        if constexpr (kAgain) {
          // `item` and every gridDim.x'th behind it, as far as it is not marked
          const uint32_t* again = reinterpret_cast<const uint32_t*>(p.ws + L.again);
          while (item < items && ((again[item >> 5] >> (item & 31)) & 1u) == 0) item += static_cast<int>(gridDim.x);
          if (item < items) {
            t = tiles[item / kHeads];
            t.head = item % kHeads;
            t.index = item;                    // (its number in the second pass: where the next search begins)
          }
          return t;
        }
        const int half = item >= first_half ? (item - first_half) & 1 : -1;
        if (half >= 0) item = first_half + ((item - first_half) >> 1);
        if (item < items) {
          const bool late = item >= first_late;
          const int left = late ? item - first_late : item, by = late ? tail : n_tiles;
          const int q = left / by, r = left - q * by;
          t = tiles[late ? q : r];
          t.head = late ? kHeads - tail + r : q;
          t.index = late ? q : r;
          if (half == 0) t.rows = min(t.rows, 128);
          if (half == 1) {                     // (none of a tile of 128 rows or fewer)
            t.q0 += 128;
            t.rows = max(t.rows - 128, 0);
            t.lim += causal ? 128 : 0;
          }
        }
        return t;
      };
      // The first item is the CTA's own number; the next one is claimed at the last
      // tile but one of the one before, early enough that its latency is not waited
      // for and no earlier: an item held in advance leaves other CTAs idle, and goes
      // to the CTA that asked first, not to the one that is done first (one held all
      // along: 8 x up to 700 over up to 4000 tokens 390 us instead of 379, 16 x up
      // to 200 55 instead of 53; two: 256 items of 1.7 ms 4.7 ms instead of 3.5).
      Tile it = record(static_cast<int>(blockIdx.x));
      while (ok) {
        ok = wait_cta(BAR(IEMPTY + w.slot), w.phase ^ 1u, quit);
        if (!ok) break;
        volatile int* dst = reinterpret_cast<volatile int*>(smem + kOffItems + 32 * w.slot);
        dst[0] = it.q0; dst[1] = it.rows; dst[2] = it.k0; dst[3] = it.nk; dst[4] = it.lim; dst[5] = it.head; dst[6] = it.index;
        ptx::mbar_arrive(BAR(IFULL + w.slot));
        if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
        if (it.head < 0) break;
        int item = 0;
        const int n0 = kv_tiles(it, 0, causal), n1 = kv_tiles(it, 1, causal), n = max(n0, n1);
        if (n0 > 0) {
          query(0, nq0, it);
          if (ok) ++nq0;
        }
        for (int j = 0; j < n && ok; ++j) {
          const int k = it.k0 + j * kKeys;
          if (!kAgain && j == max(n - 2, 0)) item = atomicAdd(&hdr->chunk, 1);
          ok = wait_cta(BAR(KEMPTY + kb), k_phase ^ 1u, quit);
          if (!ok) break;
          ptx::mbar_arrive_expect_tx(BAR(KFULL + kb), kKTile);
          const uint32_t k_dst = sbase + kOffK + kb * kKTile;
          ptx::tma_load_4d(k_dst, &maps.kn, BAR(KFULL + kb), 0, it.head, k, 0, pol);
          ptx::tma_load_4d(k_dst + kChunk, &maps.kn, BAR(KFULL + kb), 64, it.head, k, 0, pol);
          ptx::tma_load_4d(k_dst + 2 * kChunk, &maps.kr, BAR(KFULL + kb), 0, 0, k, 0, pol);
          if (++kb == kKTiles) { kb = 0; k_phase ^= 1u; }
          if (j == 0 && n1 > 0) {
            query(1, nq1, it);
            if (ok) ++nq1;
          }
          // (a K tile without its V is waited for all the same)
          ++k_tiles;
          if (ok) ok = wait_cta(BAR(VEMPTY + vb), v_phase ^ 1u, quit);
          if (!ok) break;
          ptx::mbar_arrive_expect_tx(BAR(VFULL + vb), kVTile);
          const uint32_t v_dst = sbase + kOffV + vb * kVTile;
          ptx::tma_load_4d(v_dst, &maps.v, BAR(VFULL + vb), 0, it.head, k, 0, pol);
          ptx::tma_load_4d(v_dst + kChunk, &maps.v, BAR(VFULL + vb), 64, it.head, k, 0, pol);
          if constexpr (kAgain) {   // tells a query tile's softmax that the phase of VFULL in progress is this V tile's
            if (j < n0) ptx::mbar_arrive(BAR(VASK + vb));
            if (j < n1) ptx::mbar_arrive(BAR(VASK + kVTiles + vb));
          }
          if (++vb == kVTiles) { vb = 0; v_phase ^= 1u; }
          ++v_tiles;
        }
        if (!kAgain && n == 0) item = atomicAdd(&hdr->chunk, 1);
        it = record(kAgain ? it.index + static_cast<int>(gridDim.x) : item);
      }
      // no copy may land after the CTA has left: wait for the last phase armed on each barrier
#pragma unroll 1
      for (uint32_t i = 0; i < 2 + kKTiles + kVTiles; ++i) {
        const uint32_t s = i < 2 ? i : i < 2 + kKTiles ? i - 2 : i - 2 - kKTiles;
        const uint32_t n = i < 2 ? (i == 0 ? nq0 : nq1)
                         : i < 2 + kKTiles ? (k_tiles + kKTiles - 1 - s) / kKTiles : (v_tiles + kVTiles - 1 - s) / kVTiles;
        const int bar = (i < 2 ? QFULL : i < 2 + kKTiles ? KFULL : VFULL) + static_cast<int>(s);
        if (n > 0) wait_issued(BAR(bar), (n - 1) & 1u, quit);
      }
    }
  } else if (smem_ok && warp < 3) {
    // ------------------------------------------------------------ S = Q K^T: warp 1 tile 0, warp 2 tile 1
    // The warp walks the steps together and an elected lane issues.  On a step
    // that its tile does not take part in, it releases K at once.
    regs_issue();
    const int t = warp - 1;
    Walk w;
    Tile it;
    const uint32_t s_col = tmem + kSCol + kKeys * t;
    const uint64_t desc_q = ptx::sdesc_sw128(sbase + static_cast<uint32_t>(t) * kQTile, 16, 1024);   // + chunks, K-steps
    const uint64_t desc_k = ptx::sdesc_sw128(sbase + kOffK, 16, 1024);
    constexpr uint64_t kQChunkD = kQChunk >> 4, kChunkD = kChunk >> 4;           // in descriptor units
    uint32_t kb = 0, k_phase = 0;
    uint32_t q_phase = 0, n_s = 0;           // S tiles issued so far
    bool ok = true;
#ifdef MLA_TEST_STALL_WAIT
    // Test builds only: a wait on a barrier that nothing arrives on before the end
    // of the kernel, so that its limit runs out and every role leaves through the
    // abort path.
    if (t == 0) ok = wait_cta_warp(BAR(DRAIN), 0u, quit);
#endif
    while (ok && next_warp(w, it)) {
      const int n0 = kv_tiles(it, 0, causal), n1 = kv_tiles(it, 1, causal);
      const int n_all = __shfl_sync(0xffffffffu, max(n0, n1), 0), n_mine = __shfl_sync(0xffffffffu, t ? n1 : n0, 0);
      for (int j = 0; j < n_all && ok; ++j) {
        ok = wait_cta_warp(BAR(KFULL + kb), k_phase, quit);
        if (ok && j < n_mine) {
          if (j == 0) {
            ok = wait_cta_warp(BAR(QFULL + t), q_phase, quit);
            q_phase ^= 1u;
          }
          // the softmax has the scores before these in its registers
          if (ok && n_s > 0) ok = wait_cta_warp(BAR(SREAD + t), (n_s - 1) & 1u, quit);
          if (!ok) break;
          ++n_s;
          ptx::tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              const uint64_t da = desc_q + c * kQChunkD;
              const uint64_t db = desc_k + (3u * kb + c) * kChunkD;
#pragma unroll
              for (int k = 0; k < 4; ++k) ptx::mma_ss(s_col, da + 2u * k, db + 2u * k, kIdescS, (c > 0 || k > 0) ? 1u : 0u);
            }
            ptx::mma_commit(BAR(SFULL + t));
            ptx::mma_commit(BAR(KEMPTY + kb));
            if (j == n_mine - 1) ptx::mma_commit(BAR(QEMPTY + t));
          }
          __syncwarp();
        } else if (ok && elect_one()) {
          ptx::mbar_arrive(BAR(KEMPTY + kb));
        }
        if (++kb == kKTiles) { kb = 0; k_phase ^= 1u; }
      }
    }
    // every MMA this warp issued completes before the CTA may leave
    if (n_s > 0 && elect_one()) {   // the lane that issued them
      ptx::mma_commit(BAR(DRAIN + t));
      wait_issued(BAR(DRAIN + t), 0u, quit);
    }
    __syncwarp();
  } else if (smem_ok && warp == 3) {
    // ------------------------------------------------------------ O += P V, both tiles
    regs_issue();
    Walk w;
    Tile it;
    const uint64_t desc_v = ptx::sdesc_sw128(sbase + kOffV, kChunk, 1024);
    constexpr uint64_t kChunkD = kChunk >> 4;
    uint32_t vb = 0, v_phase = 0;
    uint32_t p_phase = 0, o_phase = 3;       // bit t: parity to wait for on PREADY, OFREE (the first item waits for none)
    bool ok = true, issued = false;
    while (ok && next_warp(w, it)) {
      const int n0 = __shfl_sync(0xffffffffu, kv_tiles(it, 0, causal), 0);
      const int n1 = __shfl_sync(0xffffffffu, kv_tiles(it, 1, causal), 0);
      const int n_all = max(n0, n1), nk = __shfl_sync(0xffffffffu, it.nk, 0);
      for (int j = 0; j < n_all && ok; ++j) {
        ok = wait_cta_warp(BAR(VFULL + vb), v_phase, quit);
        const int valid = nk - j * kKeys;
        if (ok && valid < kKeys) {
          // keys past the sequence's end have P = 0; make their V rows 0 too
          // (they may be another sequence's, and hold NaN)
#pragma unroll 1
          for (uint32_t c = 0; c < 2; ++c) {
            uint4* dst = reinterpret_cast<uint4*>(smem + kOffV + vb * kVTile + c * kChunk);
            for (int i = valid * 8 + lane; i < kKeys * 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_cta();
          __syncwarp();
        }
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t) {
          if (j >= (t ? n1 : n0)) continue;
          // an item's first P.V overwrites O: the output warps must have read the last one's
          if (j == 0) {
            ok = wait_cta_warp(BAR(OFREE + t), (o_phase >> t) & 1u, quit);
            o_phase ^= 1u << t;
          }
          if (ok) ok = wait_cta_warp(BAR(PREADY + t), (p_phase >> t) & 1u, quit);
          if (!ok) break;
          p_phase ^= 1u << t;
          ptx::tc_fence_after();
          issued = true;
          if (elect_one()) {
            const uint64_t db = desc_v + 2u * vb * kChunkD;
            const uint32_t o_col = tmem + kOCol + 128u * t, p_col = tmem + kPCol + kKeys / 2 * t;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              ptx::mma_ts(o_col, p_col + 8u * k, db + 128u * k, kIdescPV, (j > 0 || k > 0) ? 1u : 0u);
            ptx::mma_commit(BAR(PVDONE + t));
          }
          __syncwarp();
        }
        if (ok && elect_one()) ptx::mma_commit(BAR(VEMPTY + vb));
        __syncwarp();
        if (++vb == kVTiles) { vb = 0; v_phase ^= 1u; }
      }
    }
    if (issued && elect_one()) {
      ptx::mma_commit(BAR(DRAIN + 2));
      wait_issued(BAR(DRAIN + 2), 0u, quit);
    }
    __syncwarp();
  } else if (smem_ok && warp < 12) {
    // ------------------------------------------------------------ softmax (thread = query row)
    regs_softmax();
    const int t = (warp - 4) >> 2;
    const int rt = (warp & 3) * 32 + lane, r = 128 * t + rt;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kSCol + kKeys * t, p_addr = tmem + lane_base + kPCol + kKeys / 2 * t;
    const uint32_t o_addr = tmem + lane_base + kOCol + 128u * t;
    volatile float* inv_l = reinterpret_cast<volatile float*>(smem + kOffInv) + 128 * t + rt;
    const float c = p.scale_log2;
    Walk w;
    Tile it;
    uint32_t steps = 0, outs = 0;            // tiles turned into P so far (phase of SFULL, PVDONE), outputs handed over
    uint32_t number = 0, v_next = 0;         // second pass: items, and their V tiles, so far
    uint32_t ask_phase = 0;                  // second pass, bit s: parity to wait for on VASK + s
    bool ok = true;
    while (ok && next_warp(w, it)) {
      const uint32_t v_first = v_next;
      if constexpr (kAgain) {
        ++number;
        v_next += static_cast<uint32_t>(max(kv_tiles(it, 0, causal), kv_tiles(it, 1, causal)));
      }
      if (it.rows <= 128 * t) continue;
      const int n = kv_tiles(it, t, causal);
      const int vis = visible(it, r, causal);
      const size_t orow = (static_cast<size_t>(it.q0) + r) * kHeads + it.head;
      if (n == 0) {                          // no row of the tile sees a key
        if (r < it.rows) {
          const uint32_t z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
          for (int q = 0; q < 8; ++q) ptx::st_global_v8(p.out + orow * 128 + 16 * q, z);
          p.lse[orow] = -INFINITY;
        }
        continue;
      }
      float mc = 0.f;                        // reference maximum * c (0 while nothing was seen)
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        if constexpr (kAgain) {
          const uint32_t at = v_first + static_cast<uint32_t>(j), vb = at % kVTiles;
          if (!wait_cta_warp(BAR(VASK + kVTiles * t + vb), (ask_phase >> vb) & 1u, quit) ||
              !wait_cta_warp(BAR(VFULL + vb), (at / kVTiles) & 1u, quit)) { ok = false; break; }
          ask_phase ^= 1u << vb;
          // the keys that a row of the tile does not see: row 0 sees the fewest
          if (clean(smem + kOffV + vb * kVTile, max(visible(it, 128 * t, causal) - j * kKeys, 0),
                    min(it.nk - j * kKeys, kKeys), j * kKeys, rt, static_cast<uint64_t>(~number) << 32,
                    reinterpret_cast<unsigned long long*>(smem + kOffFirst) + number % 3u * 256u)) {
            reinterpret_cast<volatile uint32_t*>(smem + kOffFound)[number % 3u] = number;
            ptx::fence_proxy_async_cta();
          }
          __syncwarp();
        }
        if (!wait_cta_warp(BAR(SFULL + t), steps & 1u, quit)) { ok = false; break; }
        ptx::tc_fence_after();
        uint32_t s[kKeys];
        ptx::tmem_ld32(s_addr, s);
        ptx::tmem_ld32(s_addr + 32u, s + 32);
        ptx::tmem_ld16(s_addr + 64u, s + 64);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(BAR(SREAD + t));
        const int valid = vis - j * kKeys;
        if (!__all_sync(0xffffffffu, valid >= kKeys)) {
#pragma unroll
          for (int e = 0; e < kKeys; ++e)
            if (e >= valid) s[e] = 0xFF800000u;   // -inf
        }
        const float mx = row_max(s);
        float alpha = 1.f;
        if (m_ref == -INFINITY) {
          m_ref = mx;                        // nothing accumulated so far: l = 0, O = 0
          mc = mx == -INFINITY ? 0.f : mx * c;
        } else if ((mx - m_ref) * c > kLazy) {
          m_ref = mx;
          const float nmc = mx * c;
          alpha = fast_exp2(mc - nmc);
          mc = nmc;
          l *= alpha;
        }
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        uint32_t pk[kKeys / 2];
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e) {
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
        if (steps > 0 && !wait_cta_warp(BAR(PVDONE + t), (steps - 1) & 1u, quit)) { ok = false; break; }
        ptx::tc_fence_after();
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            ptx::tmem_ld32(o_addr + 32u * q, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            ptx::tmem_st32(o_addr + 32u * q, o);
          }
        }
        ptx::tmem_st32(p_addr, pk);
        tmem_st8(p_addr + 32u, pk + 32);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(BAR(PREADY + t));
        ++steps;
      }
      if (!ok) break;
      // hand 1/l to the output warps
      if (!wait_cta_warp(BAR(LEMPTY + t), (outs & 1u) ^ 1u, quit)) break;
      ++outs;
      *inv_l = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // a NaN sum stays NaN
      __syncwarp();
      if (elect_one()) ptx::mbar_arrive(BAR(LFULL + t));
      if (r < it.rows) p.lse[orow] = l == 0.f ? -INFINITY : (mc + log2f(l)) * kLn2;
    }
  } else if (smem_ok) {
    // ------------------------------------------------------------ output (thread = row of both tiles)
    // O is read and packed, then freed for the next item before its rows are stored.
    regs_output();
    const int rt = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Walk w;
    Tile it;
    uint32_t outs = 0, steps = 0;            // bit t / half-words t: outputs and P.V steps of tile t so far, mod 2
    uint32_t number = 0;                     // second pass: items so far
    bool ok = true;
    while (ok && next_warp(w, it)) {
      ++number;
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int n = kv_tiles(it, t, causal);
        if (n == 0) continue;
        if (!wait_cta_warp(BAR(LFULL + t), (outs >> t) & 1u, quit)) { ok = false; break; }
        outs ^= 1u << t;
        const float inv = reinterpret_cast<const volatile float*>(smem + kOffInv)[128 * t + rt];
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(BAR(LEMPTY + t));
        steps ^= (static_cast<uint32_t>(n) & 1u) << t;
        // its last P.V: number steps - 1 of the tile's
        if (!wait_cta_warp(BAR(PVDONE + t), ((steps >> t) & 1u) ^ 1u, quit)) { ok = false; break; }
        ptx::tc_fence_after();
        uint32_t o16[64];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[32];
          ptx::tmem_ld32(tmem + lane_base + kOCol + 128u * t + 32u * q, o);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            o16[16 * q + e] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(BAR(OFREE + t));
        const int r = 128 * t + rt;
        if (r < it.rows) {
          __nv_bfloat16* dst = p.out + ((static_cast<size_t>(it.q0) + r) * kHeads + it.head) * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q) ptx::st_global_v8(dst + 16 * q, o16 + 8 * q);
          if constexpr (!kAgain) {
            // a result that is not finite, of weights that are (1/l is not NaN): once more
            uint32_t sum[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 64; e += 2) add_product(sum[(e >> 1) & 1], o16[e], o16[e + 1]);
            const uint32_t bad = ((sum[0] & 0x7F807F80u) + 0x00800080u) | ((sum[1] & 0x7F807F80u) + 0x00800080u);
            if (causal && inv >= 0.f && (bad & 0x80008000u)) {   // an exponent of ones carries into the sign's place
              atomicOr(reinterpret_cast<uint32_t*>(p.ws + L.again) + 4 * it.index + (it.head >> 5), 1u << (it.head & 31));
              *reinterpret_cast<volatile int*>(&hdr->prefill_again) = 1;
            }
          } else if (reinterpret_cast<const volatile uint32_t*>(smem + kOffFound)[number % 3u] == number) {
            // values that were taken out, of keys that the row sees (an entry of
            // another item is larger than any of this one)
            const volatile unsigned long long* first =
                reinterpret_cast<const volatile unsigned long long*>(smem + kOffFirst) + number % 3u * 256u;
            const unsigned long long end = static_cast<uint64_t>(~number) << 32 | static_cast<uint32_t>(visible(it, r, causal));
#pragma unroll 1
            for (int d = 0; d < 128; ++d) {
              const float up = first[d] < end ? INFINITY : 0.f, down = first[128 + d] < end ? -INFINITY : 0.f;
              if (up != down) dst[d] = __float2bfloat16(__bfloat162float(dst[d]) + up + down);
            }
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

}  // namespace

cudaError_t launch_prefill(PFN_cuTensorMapEncodeTiled_v12000 encode, const PrefillParams& p, int sms,
                           cudaStream_t stream) {
  const PrefillWs L = prefill_ws(p.batch, p.nq);
  if (L.max_tiles <= 0) return cudaSuccess;
  Maps maps;
  // with no key at all nothing is loaded; the maps still need one row
  const int nk = p.nk > 0 ? p.nk : 1;
  if (!encode_map(encode, &maps.qn, p.q_nope, 128, kHeads, p.nq, p.qn_t, p.qn_h, 128) ||
      !encode_map(encode, &maps.qr, p.q_rope, 64, kHeads, p.nq, p.qr_t, p.qr_h, 128) ||
      !encode_map(encode, &maps.kn, p.k_nope, 128, kHeads, nk, p.kn_t, p.kn_h, kKeys) ||
      !encode_map(encode, &maps.kr, p.k_rope, 64, 1, nk, p.kr_t, 64, kKeys) ||
      !encode_map(encode, &maps.v, p.v, 128, kHeads, nk, p.v_t, p.v_h, kKeys))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> configured{0}, configured_again{0};
  cudaError_t e = allow_smem(prefill_kernel<false>, kSmem, configured);
  if (e == cudaSuccess) e = allow_smem(prefill_kernel<true>, kSmem, configured_again);
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(L.max_tiles) * kHeads;
  const int ctas = static_cast<int>(items < sms ? items : sms);
  e = launch_kernel(prefill_plan_kernel, dim3(1), dim3(1024), 0, stream, p.cu_q, p.cu_k, p.batch, p.nq, p.nk, p.causal,
                    ctas, p.ws, L);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_kernel<false>, maps, p, L);
  // (without the mask a row sees every key)
  return e != cudaSuccess || !p.causal ? e : cudaLaunchKernelEx(&cfg, prefill_kernel<true>, maps, p, L);
}

}  // namespace mla
