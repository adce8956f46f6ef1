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
// run) and within a head the longest tiles first.  An item's rows are two
// M = 128 tiles that share each K/V tile of 128 keys:
//   tensor memory (512 columns): S0 | S1 | O0 | O1, 128 fp32 columns each; P
//       (bf16, 64 columns) takes the place of the S it was made from;
//   shared memory: Q0 | Q1 (48 KiB each), and a ring of eight 16-KiB chunks
//       (128 keys x 64 values), three per K tile and two per V tile, so K
//       and V are prefetched chunk by chunk as chunks are released;
//   warp 0 issues the TMA loads, warps 1 and 3 the MMAs of tile 0 and tile 1,
//   warp 2 fetches the items, warps 4..7 and 8..11 are the softmax of tile 0
//   and tile 1 (thread = row).
// An MMA warp issues P.V of step j and then S of step j + 1 (which overwrites
// that P: the tensor pipe runs in order), so while one tile's softmax runs the
// tensor cores work on the other's.  The step after an item's last is the next
// item's first, so items overlap.
//
// The maximum is lazy: a row's reference moves only when a tile's maximum
// exceeds it by more than 2^kLazy, so O is rescaled rarely; its softmax warps
// do that themselves, after the previous PV of the tile has completed.
//
// Every wait is bounded: a timeout records MLA_STATUS_TIMEOUT and raises the
// abort flag, all roles leave, and the kernel ends through its teardown.
#include <climits>

#include "prefill.cuh"
#include "waits.cuh"

namespace mla {

namespace {

constexpr int kThreads = 640;
constexpr int kKeys = 128;                         // keys per K/V tile
constexpr uint32_t kChunk = 128u * 128u;           // 16 KiB: 128 rows x 64 values
constexpr uint32_t kQTile = 3 * kChunk;            // 128 query rows x 192
constexpr int kRing = 8;
constexpr uint32_t kOffRing = 2 * kQTile;
constexpr uint32_t kOffBar = kOffRing + kRing * kChunk;   // 224 KiB
constexpr int kItemSlots = 2;
constexpr int kTiles = 4;                          // K or V tiles in flight at most (barriers)
enum Bar {
  QFULL = 0, QEMPTY = QFULL + 2, FULL = QEMPTY + 2, EMPTY = FULL + kTiles, SFULL = EMPTY + kTiles, PREADY = SFULL + 2,
  PVDONE = PREADY + 2, IFULL = PVDONE + 2, IEMPTY = IFULL + kItemSlots, DRAIN = IEMPTY + kItemSlots,
  NBAR = DRAIN + 2
};
constexpr uint32_t kOffTmem = kOffBar + 8 * NBAR;
constexpr uint32_t kOffItems = (kOffTmem + 16 + 15) & ~15u;     // kItemSlots x 32 bytes
constexpr uint32_t kOffPair = kOffItems + 32 * kItemSlots;      // fp32 [2 tiles][2 halves][128 rows]
constexpr uint32_t kSmem = kOffPair + 2 * 2 * 128 * 4;
static_assert(kSmem <= 232448, "shared memory budget");

constexpr uint32_t kSCol = 0, kOCol = 256;         // + 128 t
constexpr uint32_t kIdescS = ptx::idesc_bf16(128, 128, 0, 0);    // Q, K: K-major
constexpr uint32_t kIdescPV = ptx::idesc_bf16(128, 128, 0, 1);   // P in tensor memory, V: MN-major
constexpr uint32_t kIdescPVHalf = ptx::idesc_bf16(128, 64, 0, 1);
// log2 units: P <= 2^12, exact in relative terms, and far from fp32 overflow in O and l
constexpr float kLazy = 12.0f;
constexpr float kLn2 = 0.69314718055994530942f;

// Header fields this operator uses: n_tiles (tiles in the list) and chunk
// (the next work item).
struct Tile {
  int q0, rows;   // first packed query row, query rows (1..256)
  int k0, nk;     // first packed key, keys of the sequence
  int lim;        // keys that row 0 sees before clamping to nk (row r: lim + r if causal)
  int head;       // filled in for a fetched item; -1: no more items
  int pad[2];
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
                                                            int causal, uint8_t* __restrict__ ws, PrefillWs L) {
  __shared__ int s_count[kClasses];
  __shared__ int s_warp[32];
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(ws);
  Tile* tiles = reinterpret_cast<Tile*>(ws + L.tiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  s_count[tid] = 0;
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
        t.head = 0;
        t.pad[0] = t.pad[1] = 0;
        const int c = kClasses - 1 - min(kClasses - 1, max(kv_tiles(t, 0, causal), kv_tiles(t, 1, causal)));
        const int pos = atomicAdd(&s_count[c], 1);
        if (pass == 1) {
          if (pos < L.max_tiles) tiles[pos] = t;
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
        hdr->n_tiles = min(before + x, L.max_tiles);
        hdr->chunk = 0;
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

// 32 lanes x 16 columns to tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32"
               " [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                  "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
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

__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 104;"); }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Maximum of 64 scores.
__device__ __forceinline__ float row_max(const uint32_t* s) {
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
  for (int e = 16; e < 64; e += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = max3(m[i], __uint_as_float(s[e + 2 * i]), __uint_as_float(s[e + 2 * i + 1]));
  return fmaxf(max3(max3(m[0], m[1], m[2]), m[3], m[4]), max3(m[5], m[6], m[7]));
}

// Named barrier of two warps, and the same with an OR over their 64 threads.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" :: "r"(id) : "memory"); }
__device__ __forceinline__ bool any_of_pair(int id, bool v) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\tbar.red.or.pred p, %1, 64, q;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(r) : "r"(id), "r"(static_cast<uint32_t>(v)) : "memory");
  return r != 0;
}

// P = exp2(s c - mc) of 64 scores, as bf16 into 32 columns of tensor memory;
// the unrounded sum is added to `sum`.
__device__ __forceinline__ void p_half(const uint32_t* s, float c, float mc, float& sum, uint32_t addr) {
  float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t* v = s + 32 * q + 2 * e;
      const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), make_float2(c, c),
                                  make_float2(-mc, -mc));
      const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      if (e & 1) acc1 = __fadd2_rn(acc1, p);
      else acc0 = __fadd2_rn(acc0, p);
      const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
      pk[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    tmem_st16(addr + 16u * q, pk);
  }
  acc0 = __fadd2_rn(acc0, acc1);
  sum += acc0.x + acc0.y;
}

__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ Maps maps, const PrefillParams p, const PrefillWs L) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws);
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(BAR(QFULL + t), 1);
      ptx::mbar_init(BAR(QEMPTY + t), 1);
      ptx::mbar_init(BAR(SFULL + t), 1);
      ptx::mbar_init(BAR(PREADY + t), 8);           // one arrival a softmax warp
      ptx::mbar_init(BAR(PVDONE + t), 1);
    }
    for (int s = 0; s < kTiles; ++s) { ptx::mbar_init(BAR(FULL + s), 1); ptx::mbar_init(BAR(EMPTY + s), 2); }
    for (int s = 0; s < kItemSlots; ++s) {
      ptx::mbar_init(BAR(IFULL + s), 1);
      ptx::mbar_init(BAR(IEMPTY + s), 19);     // producer, two MMA warps, sixteen softmax warps
    }
    ptx::mbar_init(BAR(DRAIN), 1);
    ptx::mbar_init(BAR(DRAIN + 1), 1);
    ptx::fence_barrier_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc(sbase + kOffTmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  const int causal = p.causal;

  // The next item of this role's walk: false when there is none (or a wait
  // gave up).  Each consumer reads the record and then releases its slot.
  struct Walk { int slot = 0; uint32_t phase = 0; };
  auto read_item = [&](Walk& w, Tile& t) {
    const volatile int* src = reinterpret_cast<const volatile int*>(smem + kOffItems + 32 * w.slot);
    t.q0 = src[0]; t.rows = src[1]; t.k0 = src[2]; t.nk = src[3]; t.lim = src[4]; t.head = src[5];
  };
  auto next_warp = [&](Walk& w, Tile& t) {
    if (!wait_short_warp(BAR(IFULL + w.slot), w.phase, hdr)) { t.head = -1; t.nk = 0; return false; }
    read_item(w, t);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(IEMPTY + w.slot));
    if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
    return t.head >= 0;
  };

  // Registers (96 a thread at launch) are split 64 to warps 0..3, 104 to the
  // softmax warps (4 * 64 + 16 * 104 = 20 * 96), each role's branch setting
  // its own.
  if (smem_ok && warp == 2) {
    // ------------------------------------------------------------ items
    reg_dec();
    if (lane == 0) {
      const Tile* tiles = reinterpret_cast<const Tile*>(p.ws + L.tiles);
      const int n = *reinterpret_cast<const volatile int*>(&hdr->n_tiles);
      Walk w;
      while (true) {
        const int item = atomicAdd(&hdr->chunk, 1);
        const bool more = item < n * kHeads;
        Tile t;
        t.q0 = t.rows = t.k0 = t.nk = t.lim = 0;
        t.head = -1;
        if (more) {
          t = tiles[item % n];
          t.head = item / n;
        }
        if (!wait_short(BAR(IEMPTY + w.slot), w.phase ^ 1u, hdr)) break;
        volatile int* dst = reinterpret_cast<volatile int*>(smem + kOffItems + 32 * w.slot);
        dst[0] = t.q0; dst[1] = t.rows; dst[2] = t.k0; dst[3] = t.nk; dst[4] = t.lim; dst[5] = t.head;
        ptx::mbar_arrive(BAR(IFULL + w.slot));
        if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
        if (!more) break;
      }
    }
  } else if (smem_ok && warp == 0) {
    // ------------------------------------------------------------ TMA producer
    reg_dec();
    if (lane == 0) {
      const uint64_t pol = ptx::policy_evict_normal();
      Walk w;
      uint32_t pos = 0, seq = 0;               // chunks and tiles queued so far
      uint32_t nq0 = 0, nq1 = 0;               // Q tiles queued so far
      bool ok = true;
      // The ring holds eight chunks, so a tile's slots were last used by the
      // third and fourth tiles before it (K 3 + V 2 + K 3, or V 2 + K 3 + V 2
      // and one chunk of a K).
      auto slot_free = [&]() {
        if (seq >= 4) ok = wait_short(BAR(EMPTY + (seq & 3u)), ((seq - 4) >> 2) & 1u, hdr);
        if (ok && seq >= 3) ok = wait_short(BAR(EMPTY + ((seq - 3) & 3u)), ((seq - 3) >> 2) & 1u, hdr);
        return ok;
      };
      auto chunk = [&](const CUtensorMap* map, int x, int y, int z) {
        ptx::tma_load_3d(sbase + kOffRing + (pos & (kRing - 1)) * kChunk, map, BAR(FULL + (seq & 3u)), x, y, z, pol);
        ++pos;
      };
      auto query = [&](int t, uint32_t n, const Tile& it) {
        ok = wait_short(BAR(QEMPTY + t), (n & 1u) ^ 1u, hdr);
        if (!ok) return;
        ptx::mbar_arrive_expect_tx(BAR(QFULL + t), kQTile);
        const uint32_t dst = sbase + static_cast<uint32_t>(t) * kQTile;
        const int row = it.q0 + 128 * t;
        ptx::tma_load_3d(dst, &maps.qn, BAR(QFULL + t), 0, it.head, row, pol);
        ptx::tma_load_3d(dst + kChunk, &maps.qn, BAR(QFULL + t), 64, it.head, row, pol);
        ptx::tma_load_3d(dst + 2 * kChunk, &maps.qr, BAR(QFULL + t), 0, it.head, row, pol);
      };
      while (ok) {
        if (!wait_short(BAR(IFULL + w.slot), w.phase, hdr)) break;
        Tile it;
        read_item(w, it);
        ptx::mbar_arrive(BAR(IEMPTY + w.slot));
        if (++w.slot == kItemSlots) { w.slot = 0; w.phase ^= 1u; }
        if (it.head < 0) break;
        const int n0 = kv_tiles(it, 0, causal), n1 = kv_tiles(it, 1, causal), n = max(n0, n1);
        if (n0 > 0) {
          query(0, nq0, it);
          if (ok) ++nq0;
        }
        for (int j = 0; j < n && ok; ++j) {
          const int k = it.k0 + j * kKeys;
          if (!slot_free()) break;
          ptx::mbar_arrive_expect_tx(BAR(FULL + (seq & 3u)), 3 * kChunk);
          chunk(&maps.kn, 0, it.head, k);
          chunk(&maps.kn, 64, it.head, k);
          chunk(&maps.kr, 0, 0, k);
          ++seq;
          if (j == 0 && n1 > 0) {
            query(1, nq1, it);
            if (ok) ++nq1;
          }
          if (!ok || !slot_free()) break;
          ptx::mbar_arrive_expect_tx(BAR(FULL + (seq & 3u)), 2 * kChunk);
          chunk(&maps.v, 0, it.head, k);
          chunk(&maps.v, 64, it.head, k);
          ++seq;
        }
      }
      // no copy may land after the CTA has left: wait for the last phase armed on each barrier
      if (nq0 > 0) wait_drain(BAR(QFULL), (nq0 - 1) & 1u, hdr);
      if (nq1 > 0) wait_drain(BAR(QFULL + 1), (nq1 - 1) & 1u, hdr);
      for (uint32_t s = 0; s < kTiles; ++s) {
        const uint32_t n = (seq + kTiles - 1 - s) / kTiles;
        if (n > 0) wait_drain(BAR(FULL + s), (n - 1) & 1u, hdr);
      }
    }
  } else if (smem_ok && warp < 4) {
    // ------------------------------------------------------------ MMA issuers: warp 1 tile 0, warp 3 tile 1
    // The warp walks the steps together and an elected lane issues.  A wait
    // costs about 100 cycles even when its phase is complete, and the tensor
    // pipe queues only a few MMAs, so each query tile has a warp of its own:
    // one's waits pass while the other's MMAs run.  K and V are waited for
    // before P.  Everything that steers the loop comes through a shuffle or a
    // vote, so positions and descriptors stay warp-uniform.  On a step that
    // its tile does not take part in, a warp releases K and V at once.
    reg_dec();
    const int t = warp >> 1;
    Walk w;
    Tile it;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t sb = __shfl_sync(0xffffffffu, sbase, 0);
    const uint32_t d = tm + kOCol + 128u * t, a = tm + kSCol + 128u * t;
    const uint64_t desc_q = ptx::sdesc_sw128(sb + static_cast<uint32_t>(t) * kQTile, 16, 1024);   // + chunks, K-steps
    const uint64_t desc_k = ptx::sdesc_sw128(sb + kOffRing, 16, 1024);
    const uint64_t desc_v = ptx::sdesc_sw128(sb + kOffRing, kChunk, 1024);
    constexpr uint64_t kChunkD = kChunk >> 4;                                    // a chunk in descriptor units
    uint32_t kpos = 0, kseq = 0;             // ring position and tile number of the K tile to be scored next
    uint32_t q_phase = 0, p_phase = 0;
    bool ok = true, issued = false;
    // the next (item, K/V tile) step jn: the item's steps, this tile's share of them, the sequence's keys
    int jn = 0, n_all = 0, n_mine = 0, nkn = 0;
    // One item at a time, even one without keys: the softmax warps read an item
    // only after this one's last P.V, so waiting for more than the next item
    // before that P.V would wait for ever.
    auto fetch = [&]() -> bool {
      const bool have = next_warp(w, it);
      const int n0 = have ? kv_tiles(it, 0, causal) : 0, n1 = have ? kv_tiles(it, 1, causal) : 0;
      n_all = __shfl_sync(0xffffffffu, max(n0, n1), 0);
      n_mine = __shfl_sync(0xffffffffu, t ? n1 : n0, 0);
      nkn = __shfl_sync(0xffffffffu, it.nk, 0);
      jn = 0;
      return __shfl_sync(0xffffffffu, have ? 1 : 0, 0) != 0;
    };
    bool more = fetch();
    // step state: the step whose P.V comes next (its S was issued); jc < 0: none
    int jc = -1, n_cur = 0, nkc = 0;
    uint32_t vpos = 0, vseq = 0;
    while (ok && (jc >= 0 || more)) {
      const bool pv = jc >= 0 && jc < n_cur;
      if (jc >= 0) {
        ok = wait_short_warp(BAR(FULL + (vseq & 3u)), (vseq >> 2) & 1u, hdr);
        const int valid = nkc - jc * kKeys;
        if (ok && pv && valid < kKeys) {
          // keys past the sequence's end have P = 0; make their V rows 0 too
          // (they may be another sequence's, and hold NaN); both tiles' warps
          // write the same zeros before their own MMAs
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint4* dst = reinterpret_cast<uint4*>(smem + kOffRing + ((vpos + c) & (kRing - 1)) * kChunk);
            for (int i = valid * 8 + lane; i < kKeys * 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_cta();
          __syncwarp();
        }
        if (ok && !pv && elect_one()) ptx::mbar_arrive(BAR(EMPTY + (vseq & 3u)));
      }
      const bool step = more && n_all > 0, sc = step && jn < n_mine;
      if (ok && step) {
        ok = wait_short_warp(BAR(FULL + (kseq & 3u)), (kseq >> 2) & 1u, hdr);
        if (ok && !sc && elect_one()) ptx::mbar_arrive(BAR(EMPTY + (kseq & 3u)));
      }
      if (ok && sc && jn == 0) {
        ok = wait_short_warp(BAR(QFULL + t), q_phase, hdr);
        q_phase ^= 1u;
      }
      if (ok && pv) {
        ok = wait_short_warp(BAR(PREADY + t), p_phase, hdr);
        p_phase ^= 1u;
      }
      if (!ok) break;
      ptx::tc_fence_after();
      if (pv) {
        const uint32_t s0 = vpos & (kRing - 1);
        const uint64_t db = desc_v + s0 * kChunkD;
        if (elect_one()) {
          if (s0 != kRing - 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              ptx::mma_ts(d, a + 64u * (k >> 2) + 8u * (k & 3), db + 128u * k, kIdescPV, (jc > 0 || k > 0) ? 1u : 0u);
          } else {
            // the tile's second chunk wrapped to the ring's start: two halves
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const uint32_t acc = (jc > 0 || k > 0) ? 1u : 0u, ak = a + 64u * (k >> 2) + 8u * (k & 3);
              ptx::mma_ts(d, ak, db + 128u * k, kIdescPVHalf, acc);
              ptx::mma_ts(d + 64u, ak, desc_v + 128u * k, kIdescPVHalf, acc);
            }
          }
          ptx::mma_commit(BAR(EMPTY + (vseq & 3u)));
          ptx::mma_commit(BAR(PVDONE + t));
        }
        __syncwarp();
      }
      if (sc) {
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const uint64_t da = desc_q + c * kChunkD;
            const uint64_t db = desc_k + ((kpos + c) & (kRing - 1)) * kChunkD;
#pragma unroll
            for (int k = 0; k < 4; ++k) ptx::mma_ss(a, da + 2u * k, db + 2u * k, kIdescS, (c > 0 || k > 0) ? 1u : 0u);
          }
          ptx::mma_commit(BAR(SFULL + t));
          ptx::mma_commit(BAR(EMPTY + (kseq & 3u)));
          if (jn == n_mine - 1) ptx::mma_commit(BAR(QEMPTY + t));
        }
        __syncwarp();
        issued = true;
      }
      // advance: the step just scored becomes the one whose P.V comes next
      jc = -1;
      if (step) {
        jc = jn;
        n_cur = n_mine;
        nkc = nkn;
        vpos = kpos + 3;
        vseq = kseq + 1;
        kpos += 5;
        kseq += 2;
        ++jn;
      }
      if (more && jn >= n_all) more = fetch();   // (an item without keys has no step)
    }
    // every MMA this warp issued completes before the CTA may leave
    if (issued && elect_one()) {   // the lane that issued them
      ptx::mma_commit(BAR(DRAIN + t));
      wait_drain(BAR(DRAIN + t), 0u, hdr);
    }
    __syncwarp();
  } else if (smem_ok && warp >= 4) {
    // ------------------------------------------------------------ softmax and epilogue
    // Eight warps a tile: two threads share a row, each with 64 of a tile's
    // keys (and 64 of the output's columns).  Their warps meet at a named
    // barrier once a tile, which also tells whether any row's maximum passed
    // its reference by too much; only then (and on an item's first tile) do
    // they exchange maxima, so both always hold the same reference.
    reg_inc();
    const int t = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1;
    const int rt = (warp & 3) * 32 + lane;                 // row of the tile
    const int r = 128 * t + rt;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // S of keys 64 hf.. is in columns 64 hf.. of the tile's S; their P replaces its first 32 columns
    const uint32_t s_addr = tmem + lane_base + kSCol + 128u * t + 64u * hf;
    const uint32_t o_addr = tmem + lane_base + kOCol + 128u * t + 64u * hf;
    const int pair = 1 + 4 * t + (warp & 3);               // named barrier of the two warps that share rows
    volatile float* own = reinterpret_cast<volatile float*>(smem + kOffPair) + (2 * t + hf) * 128 + rt;
    const volatile float* other = reinterpret_cast<const volatile float*>(smem + kOffPair) + (2 * t + (hf ^ 1)) * 128 + rt;
    const float c = p.scale_log2;
    Walk w;
    Tile it;
    uint32_t steps = 0;                      // tiles turned into P so far (phase of SFULL, PVDONE)
    bool ok = true;
    // Both warps of a pair leave at the same place: what one of them knows alone
    // (a wait that gave up) takes effect only once the other has heard of it.
    while (true) {
      const bool have = next_warp(w, it);
      if (any_of_pair(pair, !have)) break;
      if (it.rows <= 128 * t) continue;
      const int n = kv_tiles(it, t, causal);
      const int vis = visible(it, r, causal) - 64 * hf;    // of this thread's keys
      float mc = 0.f;                        // reference maximum * c (0 while nothing was seen)
      float m_ref = -INFINITY, l = 0.f;      // l: this thread's keys
      bool quit = false;
      for (int j = 0; j < n; ++j) {
        if (!wait_short_warp(BAR(SFULL + t), steps & 1u, hdr)) ok = false;
        ptx::tc_fence_after();
        uint32_t s[64];
        ptx::tmem_ld32(s_addr, s);
        ptx::tmem_ld32(s_addr + 32u, s + 32);
        ptx::tmem_wait_ld();
        const int valid = vis - j * kKeys;
        if (!__all_sync(0xffffffffu, valid >= 64)) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= valid) s[e] = 0xFF800000u;   // -inf
        }
        float mx = row_max(s);
        const bool up = !ok || j == 0 || (m_ref == -INFINITY ? mx != -INFINITY : (mx - m_ref) * c > kLazy);
        if (any_of_pair(pair, up)) {
          // rare: agree on the rows' maxima and move the references that need it
          *own = mx;
          quit = any_of_pair(pair, !ok);
          mx = fmaxf(mx, *other);
          float alpha = 1.f;
          if (m_ref == -INFINITY ? mx != -INFINITY : (mx - m_ref) * c > kLazy) {
            const float nmc = mx * c;
            alpha = m_ref == -INFINITY ? 1.f : fast_exp2(mc - nmc);   // -inf: l = 0 and O = 0 so far
            m_ref = mx;
            mc = nmc;
            l *= alpha;
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            // O of the tiles so far is complete once the previous P.V is
            if (!wait_short_warp(BAR(PVDONE + t), (steps - 1) & 1u, hdr)) ok = false;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t o[16];
              ptx::tmem_ld16(o_addr + 16u * q, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(o_addr + 16u * q, o);
            }
          }
        }
        p_half(s, c, mc, l, s_addr);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(BAR(PREADY + t));
        ++steps;
        if (quit) break;
      }
      if (!quit && n > 0) {
        if (!wait_short_warp(BAR(PVDONE + t), (steps - 1) & 1u, hdr)) ok = false;
        ptx::tc_fence_after();
      }
      pair_sync(pair);                       // the partner has read what an exchange left here
      *own = l;
      if (any_of_pair(pair, !ok)) break;
      l += *other;
      const bool live = r < it.rows;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // a NaN sum stays NaN
      const size_t orow = (static_cast<size_t>(it.q0) + r) * kHeads + it.head;
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        uint32_t o[32], w16[16];
        if (n > 0) {
          ptx::tmem_ld32(o_addr + 32u * q, o);
          ptx::tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          w16[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (live) {
          ptx::st_global_v8(p.out + orow * 128 + 64 * hf + 32 * q, w16);
          ptx::st_global_v8(p.out + orow * 128 + 64 * hf + 32 * q + 16, w16 + 8);
        }
      }
      if (live && hf == 0) p.lse[orow] = l == 0.f ? -INFINITY : (mc + log2f(l)) * kLn2;
      ptx::tc_fence_before();
    }
  }
  // ------------------------------------------------------------ teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// (64 values, heads, tokens) boxes of 64 x 1 x 128; strides in values.
bool encode_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* base, int width, int heads,
                int tokens, long long stride_t, long long stride_h) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride_h) * 2, static_cast<cuuint64_t>(stride_t) * 2};
  cuuint32_t box[3] = {64, 1, 128};
  cuuint32_t es[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_prefill(PFN_cuTensorMapEncodeTiled_v12000 encode, const PrefillParams& p, int sms,
                           cudaStream_t stream) {
  const PrefillWs L = prefill_ws(p.batch, p.nq);
  if (L.max_tiles <= 0) return cudaSuccess;
  Maps maps;
  // with no key at all nothing is loaded; the maps still need one row
  const int nk = p.nk > 0 ? p.nk : 1;
  if (!encode_map(encode, &maps.qn, p.q_nope, 128, kHeads, p.nq, p.qn_t, p.qn_h) ||
      !encode_map(encode, &maps.qr, p.q_rope, 64, kHeads, p.nq, p.qr_t, p.qr_h) ||
      !encode_map(encode, &maps.kn, p.k_nope, 128, kHeads, nk, p.kn_t, p.kn_h) ||
      !encode_map(encode, &maps.kr, p.k_rope, 64, 1, nk, p.kr_t, 64) ||
      !encode_map(encode, &maps.v, p.v, 128, kHeads, nk, p.v_t, p.v_h))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = allow_smem(prefill_kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  e = launch_kernel(prefill_plan_kernel, dim3(1), dim3(1024), 0, stream, p.cu_q, p.cu_k, p.batch, p.nq, p.nk, p.causal,
                    p.ws, L);
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(L.max_tiles) * kHeads;
  return launch_kernel(prefill_kernel, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(kThreads), kSmem,
                       stream, maps, p, L);
}

}  // namespace mla
