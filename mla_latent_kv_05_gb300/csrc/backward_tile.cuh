// What the kernels of the backward pass share: work items, and a thread's quarter
// row of P and dS.
#pragma once
#include "backward.cuh"

namespace mla {
namespace bwd {

// Everything before it overlaps what precedes the pass in the stream.  The query pass,
// where there is one, waits for the statistics and then lets the key pass begin where
// one of its CTAs has left: that one needs the statistics too, which are complete by
// then, and nothing of the query pass.  It waits for it at its own end, so that the call
// is over when both are.
template <bool kKeys>
__device__ __forceinline__ void begin_pass(const BackwardParams& p) {
  if (!kKeys || p.key_waits) ptx::grid_dep_wait();   // (where no query pass lies between)
  ptx::grid_dep_launch();
}

// launch_kernel as a programmatic dependent of what precedes it.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

constexpr int kTile = kBackwardTile;
constexpr uint32_t kChunk = kTile * 128u;          // 16 KiB: 128 rows x 64 values
constexpr uint32_t kStatBytes = 2 * kTile * 4;     // lse and delta of a query tile
constexpr int kWarps = 16, kCols = 32;              // warps that compute P and dS, columns of a thread (a quarter row)
constexpr uint32_t kAcc1 = 0, kAcc2 = 192, kX = 320, kY = 448;   // tensor memory columns
constexpr float kLog2e = 1.4426950408889634f;

// Rows of one sequence: keys (key pass) or queries (query pass).
struct Tile {
  int r0, rows;   // first packed row, rows
  int c0, nc;     // first packed column of the sequence, its columns
  int lim;        // row r sees the columns from lim + r (keys), or those below lim + r (queries), where causal
  int first;      // first column tile
  int steps;      // column tiles
  int stat;       // query tile (of 128) of column tile 0 (keys), or of the rows' first (queries)
  int slot;       // place of the dS tile of column tile 0 (keys), or the sequence's first key tile (queries)
  int tile;       // of its sequence
  int unused[2];
};
static_assert(sizeof(Tile) == kTileBytes, "tile record");
// Keys, causal: the columns from here on are seen by all rows.
__device__ __forceinline__ int mask_end(const Tile& t) { return t.lim + t.rows - 1; }
constexpr uint32_t kItemBytes = 64;

}  // namespace bwd

// The maps of a pass: what is held (R) and what is streamed (C), as in backward.cu, the
// latter in the forms that the products need.
struct PassMaps {
  CUtensorMap r1n, r1r, r2;        // 128 rows: the 128 values, the RoPE values; V or d_out
  CUtensorMap c1n, c1r, c2;        // first products: 128 rows, or on pairs 64
  CUtensorMap c1n_d, c1r_d;        // dq on pairs: 128 rows of 64 values
};

namespace bwd {

// 128 (chunks = 2) or 64 values of tokens and heads; boxes of box_chunks x rows x 64
// values of a head, in that order, so that one copy brings both chunks of an operand
// (a copy costs its thread about 160 cycles, whatever its size).  Strides in values.
inline bool encode_chunks(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* base, int chunks, int heads,
                          int tokens, long long stride_t, long long stride_h, unsigned rows, unsigned box_chunks) {
  // (spans.cuh; 128 values of 128 heads span enough from the fourth token on)
  const uint64_t far = chunks > 1 ? 0 : tma_far(base, 2 * static_cast<uint64_t>((tokens - 1) * stride_t + (heads - 1) * stride_h + 64));
  cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(tokens), static_cast<cuuint64_t>(far ? 2 : chunks), static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride_t) * 2, far ? far : 128u, static_cast<cuuint64_t>(stride_h) * 2};
  cuuint32_t box[4] = {64, rows, box_chunks, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// keys: rows are keys.  col_rows: rows of the streamed boxes of the first products.
inline bool pass_maps(PFN_cuTensorMapEncodeTiled_v12000 encode, const BackwardParams& p, bool keys, unsigned col_rows, PassMaps* m) {
  // with no row at all nothing is loaded; the maps still need one
  const int nq = p.nq > 0 ? p.nq : 1, nk = p.nk > 0 ? p.nk : 1;
  auto qn = [&](CUtensorMap* t, unsigned rows, unsigned box) { return encode_chunks(encode, t, p.q_nope, 2, kHeads, nq, p.qn_t, p.qn_h, rows, box); };
  auto qr = [&](CUtensorMap* t, unsigned rows) { return encode_chunks(encode, t, p.q_rope, 1, kHeads, nq, p.qr_t, p.qr_h, rows, 1); };
  auto kn = [&](CUtensorMap* t, unsigned rows, unsigned box) { return encode_chunks(encode, t, p.k_nope, 2, kHeads, nk, p.kn_t, p.kn_h, rows, box); };
  auto kr = [&](CUtensorMap* t, unsigned rows) { return encode_chunks(encode, t, p.k_rope, 1, 1, nk, p.kr_t, 64, rows, 1); };
  auto v = [&](CUtensorMap* t, unsigned rows, unsigned box) { return encode_chunks(encode, t, p.v, 2, kHeads, nk, p.v_t, p.v_h, rows, box); };
  auto od = [&](CUtensorMap* t, unsigned rows, unsigned box) { return encode_chunks(encode, t, p.d_out, 2, kHeads, nq, p.do_t, p.do_h, rows, box); };
  // on pairs both chunks of a first product's operand in one copy, else a copy each
  const bool pairs = col_rows < kTile;
  const unsigned box = pairs ? 2 : 1;
  if (keys)
    return kn(&m->r1n, kTile, 2) && kr(&m->r1r, kTile) && v(&m->r2, kTile, 2) && qn(&m->c1n, kTile, 1) &&
           qr(&m->c1r, kTile) && od(&m->c2, kTile, 1);
  return qn(&m->r1n, kTile, 2) && qr(&m->r1r, kTile) && od(&m->r2, kTile, 2) && kn(&m->c1n, col_rows, box) &&
         kr(&m->c1r, col_rows) && v(&m->c2, col_rows, box) &&
         (!pairs || (kn(&m->c1n_d, kTile, 1) && kr(&m->c1r_d, kTile)));
}

// (Through L2: the key pass begins without waiting for the grids that wrote the list
// and the statistics, which are complete by then.)
__device__ __forceinline__ Tile read_tile(const Tile* at) {
  const int4 a = __ldcg(reinterpret_cast<const int4*>(at)), b = __ldcg(reinterpret_cast<const int4*>(at) + 1);
  const int2 c = __ldcg(reinterpret_cast<const int2*>(at) + 4);
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y};
}

// An item in shared memory: its tile, and its first head (-1: no more items).
__device__ __forceinline__ void write_item(uint8_t* at, const Tile& t, int head) {
  volatile int* dst = reinterpret_cast<volatile int*>(at);
  dst[0] = t.r0; dst[1] = t.rows; dst[2] = t.c0; dst[3] = t.nc; dst[4] = t.lim; dst[5] = t.first; dst[6] = t.steps;
  dst[7] = t.stat;
  dst[8] = head;
  dst[9] = t.slot;
  dst[10] = t.tile;
}
__device__ __forceinline__ void read_item(const uint8_t* at, Tile& t, int& head) {
  const volatile int* src = reinterpret_cast<const volatile int*>(at);
  t.r0 = src[0]; t.rows = src[1]; t.c0 = src[2]; t.nc = src[3]; t.lim = src[4]; t.first = src[5]; t.steps = src[6];
  t.stat = src[7];
  head = src[8];
  t.slot = src[9];
  t.tile = src[10];
}

__device__ __forceinline__ bool stored(const BackwardPlan* plan) { return *reinterpret_cast<const volatile int*>(&plan->stored) != 0; }

// (Without a cache hint, with which concurrent copies of all SMs reached 110 GB/s an SM
// instead of 190.)
__device__ __forceinline__ void load_4d(uint32_t dst, const void* tmap, uint32_t bar, int x, int row, int chunk, int head) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
               :: "r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(row), "r"(chunk), "r"(head) : "memory");
}

// Items in the order in which they are handed out: head group by head group, and
// the last groups tile by tile (as in prefill).
struct Schedule {
  int n_tiles, tail, groups, items, first_late;
  __device__ Schedule(const BackwardPlan* plan, int side, int groups, bool off) : groups(groups) {
    n_tiles = *reinterpret_cast<const volatile int*>(&plan->tiles[side]);
    tail = *reinterpret_cast<const volatile int*>(&plan->tail[side]);
    items = off ? 0 : n_tiles * groups;
    first_late = items - n_tiles * tail;
  }
  __device__ bool find(int item, int& tile, int& head_group) const {
    if (item >= items) return false;
    const bool late = item >= first_late;
    const int left = late ? item - first_late : item, by = late ? tail : n_tiles;
    const int q = left / by, r = left - q * by;
    tile = late ? q : r;
    head_group = late ? groups - tail + r : q;
    return true;
  }
};

// Scores of 32 columns to probabilities, in place: exp2(s c - lse log2(e)), 0 outside
// [lo, hi) unless `all` are inside.  kKeys: the columns are queries, with their lse in
// lse4; else the row is one, with row_lse.
template <bool kKeys>
__device__ __forceinline__ void probabilities(uint32_t* s, const float4* lse4, float row_lse, float c, bool all, int lo, int hi) {
#pragma unroll
  for (int e = 0; e < kCols; e += 4) {
    float4 l = make_float4(row_lse, row_lse, row_lse, row_lse);
    if constexpr (kKeys) l = lse4[e / 4];
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(c, c), make_float2(-l.x, -l.y));
    const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), make_float2(c, c), make_float2(-l.z, -l.w));
    s[e] = __float_as_uint(fast_exp2(x.x));
    s[e + 1] = __float_as_uint(fast_exp2(x.y));
    s[e + 2] = __float_as_uint(fast_exp2(y.x));
    s[e + 3] = __float_as_uint(fast_exp2(y.y));
  }
  if (!all) {
#pragma unroll
    for (int e = 0; e < kCols; ++e)
      if (e < lo || e >= hi) s[e] = 0u;
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// P and dS as the bf16 operands of the second products: half a step, 2^-8 of each.  The
// MMAs that take fp32 values (tf32) run at half the rate; two bf16 terms for each of P and
// dS would be another 320 (dk, dv) and 192 (dq) units beside the 832.  Against 64 bits the
// results' relative error is 2.3e-3, that of exact results rounded to bf16 1.7e-3
// (1000 causal, 777 full).
__device__ __forceinline__ void pack(const uint32_t* s, uint32_t* pk) {
#pragma unroll
  for (int e = 0; e < kCols / 2; ++e) pk[e] = bf16_pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
}

// dS / scale = p (dP - delta) of 32 columns, as bf16.
template <bool kKeys>
__device__ __forceinline__ void gradients(const uint32_t* pr, const uint32_t* d, const float4* delta4, float row_delta, bool all,
                                          int lo, int hi, uint32_t* pk) {
#pragma unroll
  for (int e = 0; e < kCols; e += 4) {
    float4 m = make_float4(row_delta, row_delta, row_delta, row_delta);
    if constexpr (kKeys) m = delta4[e / 4];
    float y[4];
    const float2 a = __fadd2_rn(make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), make_float2(-m.x, -m.y));
    const float2 b = __fadd2_rn(make_float2(__uint_as_float(d[e + 2]), __uint_as_float(d[e + 3])), make_float2(-m.z, -m.w));
    y[0] = __uint_as_float(pr[e]) * a.x;
    y[1] = __uint_as_float(pr[e + 1]) * a.y;
    y[2] = __uint_as_float(pr[e + 2]) * b.x;
    y[3] = __uint_as_float(pr[e + 3]) * b.y;
    if (!all) {                              // (0 times what is not finite)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e + k < lo || e + k >= hi) y[k] = 0.f;
    }
    pk[e / 2] = bf16_pair(y[0], y[1]);
    pk[e / 2 + 1] = bf16_pair(y[2], y[3]);
  }
}

// 16 columns to tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32"
               " [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                  "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// 2 kPairs accumulator columns, read and waited for, as bf16.
template <int kPairs>
__device__ __forceinline__ void to_bf16(const uint32_t* a, float mul, uint32_t* out) {
#pragma unroll
  for (int e = 0; e < kPairs; ++e) out[e] = bf16_pair(__uint_as_float(a[2 * e]) * mul, __uint_as_float(a[2 * e + 1]) * mul);
}

// Registers (80 a thread at launch): 40 for the eight warps that load and
// issue, 96 for the sixteen others (8 * 40 + 16 * 96 <= 24 * 80), each role's branch
// setting its own.
__device__ __forceinline__ void regs_issue() { asm volatile("setmaxnreg.dec.sync.aligned.u32 40;"); }
__device__ __forceinline__ void regs_compute() { asm volatile("setmaxnreg.inc.sync.aligned.u32 96;"); }

// 16 bf16 values to 32 bytes at dst (16-byte aligned).
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const uint32_t* v) {
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
}

// A quarter row of dS, 32 columns of key r, to its place in the tile that the product with
// K reads: halves of 64 keys, of which each has 16 columns of 8 queries, a key's 16 bytes
// behind the last key's (MN-major without swizzle, so that a warp writes 512 bytes in a
// row: the key pass of 4096 tokens takes 1,017 us; as 128-byte rows in the swizzled order
// 1,080, without storing 890).  Written to leave L2 first: 1,660 us instead of 1,674 for
// 2 x 512 queries over 8,012 keys.
__device__ __forceinline__ void store_ds(uint8_t* tile, int r, int quarter, const uint32_t* pk) {
  uint4* at = reinterpret_cast<uint4*>(tile + (r >> 6) * 16384 + quarter * 4096 + (r & 63) * 16);
#pragma unroll
  for (int e = 0; e < 4; ++e) __stcs(at + 64 * e, make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]));
}

// A quarter row of a head's results: 32 values of dk (or dq) and of dv as bf16, 16 of
// the RoPE part, which of dk is fp32 and stored with the group's last head, for the sum.
template <bool kKeys>
__device__ __forceinline__ void store_results(const BackwardParams& p, const BackwardWs& L, size_t row, int head, int head_group,
                                              int quarter, bool last, const uint32_t* nope, const uint32_t* second,
                                              const uint32_t* rope) {
  if (!kKeys && p.causal) {
    // 0 times every value: not 0 where one is not finite (backward_last.cu)
    __nv_bfloat162 z[4];
    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int e = 0; e < 24; ++e) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(e < 16 ? nope + e : rope + e - 16);
      z[e & 3] = e < 4 ? __hmul2(x, zero) : __hfma2(x, zero, z[e & 3]);
    }
    z[0] = __hadd2(__hadd2(z[0], z[1]), __hadd2(z[2], z[3]));
    if ((*reinterpret_cast<const uint32_t*>(z) & 0x7FFF7FFFu) != 0) reinterpret_cast<BackwardPlan*>(p.ws + L.plan)->odd[1] = 1;
  }
  __nv_bfloat16* dst = (kKeys ? p.dk_nope + row * p.dkn_t + head * p.dkn_h : p.dq_nope + row * p.dqn_t + head * p.dqn_h) + 32 * quarter;
  store16(dst, nope);
  store16(dst + 16, nope + 8);
  if constexpr (kKeys) {
    dst = p.dv + row * p.dv_t + head * p.dv_h + 32 * quarter;
    store16(dst, second);
    store16(dst + 16, second + 8);
    if (last) {
      float* part = reinterpret_cast<float*>(p.ws + L.rope) + (static_cast<size_t>(head_group) * p.nk + row) * kDr + 16 * quarter;
      ptx::st_global_v8(part, rope);
      ptx::st_global_v8(part + 8, rope + 8);
    }
  } else {
    store16(p.dq_rope + row * p.dqr_t + head * p.dqr_h + 16 * quarter, rope);
  }
}

}  // namespace bwd
}  // namespace mla
