// C ABI of the MLA decode library: argument validation, workspace sizing,
// tensor-map creation and the launch sequence (planner -> paired decode
// kernel -> split merge), all on the caller's stream.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "backward.cuh"
#include "decode.cuh"
#include "expand.cuh"
#include "prefill.cuh"
#include "rope.cuh"
#include "rows.cuh"
#include "tree.cuh"

namespace {

using namespace mla;

thread_local cudaEvent_t g_prof_before = nullptr, g_prof_after = nullptr;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// The bf16 cache viewed as a 4-D tensor: (64 columns, 8 rows, 9 column
// chunks, num_pages*8 row groups) with strides 1152 B (row), 128 B (chunk)
// and 9216 B (row group).  A box of 64 x 8 x `chunks` x 4 is one half page
// (32 tokens), written to shared memory as 8-row x 128-byte swizzle atoms in
// (row group, chunk, row) order, so consecutive half-page slots form one
// K-major operand with a constant row-group stride.
// `groups` row groups per box: 4 for a half page, 8 for a whole page.
int make_cache_tmap(CUtensorMap* m, const void* cache, int num_pages, unsigned chunks, unsigned groups = 4) {
  auto fn = encode_fn();
  if (!fn) return MLA_ERR_CUDA;
  cuuint64_t dims[4] = {64, 8, static_cast<cuuint64_t>(kRow / 64), static_cast<cuuint64_t>(num_pages) * (kPage / 8)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(kRow) * 2, 128, static_cast<cuuint64_t>(kRow) * 2 * 8};
  cuuint32_t box[4] = {64, 8, chunks, groups};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(cache), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MLA_OK : MLA_ERR_CUDA;
}

int validate_common(const void* q_absorbed, const void* q_rope, const void* kv_cache, const int32_t* block_table,
                    const int32_t* seq_lens, int batch, int sq, int num_heads, int num_pages, int page_size,
                    int max_pages, float scale, const void* out, const float* lse, const void* workspace) {
  if (!q_absorbed || !q_rope || !kv_cache || !block_table || !seq_lens || !out || !lse || !workspace)
    return MLA_ERR_INVALID_ARG;
  if (batch < 0 || sq <= 0 || num_pages <= 0 || max_pages <= 0 || !std::isfinite(scale) || !(scale > 0.f))
    return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads || page_size != kPage || sq > kMaxSq) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(batch) * sq > kMaxRows) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * kPage >= INT_MAX / 2 ||
      static_cast<long long>(max_pages) * kPage >= INT_MAX / 2)
    return MLA_ERR_UNSUPPORTED;
  if (!aligned(q_absorbed, 16) || !aligned(q_rope, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

enum class CacheKind { kBf16, kFp8, kFp4, kFp8V41, kFp4V41 };

// CTA pairs a query index gets: all resident pairs, but no more than one per
// kPagesPerPair pages the call can hold (batch * max_pages, known on the host
// without reading seq_lens).  A small decode then runs on a few pairs, and a
// row of a few pages is not split (no partial write, nothing to merge).  The
// workspace stays sized for all resident pairs.
constexpr long long kPagesPerPair = 8;
int pairs_for(int max_pairs, long long page_bound, long long pages_per_pair = kPagesPerPair) {
  const long long want = (page_bound + pages_per_pair - 1) / pages_per_pair;
  return static_cast<int>(want < 1 ? 1 : (want < max_pairs ? want : max_pairs));
}

int run_decode(CacheKind kind, const uint16_t* q_absorbed, const uint16_t* q_rope, const void* kv_cache,
               const int32_t* block_table, const int32_t* seq_lens, int batch, int sq, int num_heads, int num_pages,
               int page_size, int max_pages, float softmax_scale, uint16_t* out, float* lse, void* workspace,
               size_t workspace_bytes, void* stream_ptr) {
  int st = validate_common(q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads, num_pages,
                           page_size, max_pages, softmax_scale, out, lse, workspace);
  if (st != MLA_OK) return st;
  if (batch == 0) return MLA_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const int pairs = decode_max_pairs();
  if (pairs <= 0) return MLA_ERR_CUDA;
  const int ppg = pairs_for(pairs / sq > 0 ? pairs / sq : 1, static_cast<long long>(batch) * max_pages);
  const WsLayout L = ws_layout(batch, sq, pairs);
  if (workspace_bytes < L.total) return MLA_ERR_WORKSPACE;

  // half and whole pages of chunks 0..4 and 5..8 (score SM), half pages of
  // the 8 latent chunks (value SM)
  CacheMaps maps;
  const bool quant = kind != CacheKind::kBf16;
  if (!quant) {
    st = make_cache_tmap(&maps.k, kv_cache, num_pages, 5);
    if (st == MLA_OK) st = make_cache_tmap(&maps.k8, kv_cache, num_pages, 5, 8);
    if (st == MLA_OK) st = make_cache_tmap(&maps.kb, kv_cache, num_pages, 4);
    if (st == MLA_OK) st = make_cache_tmap(&maps.kb8, kv_cache, num_pages, 4, 8);
    if (st == MLA_OK) st = make_cache_tmap(&maps.v, kv_cache, num_pages, 8);
    if (st != MLA_OK) return st;
  }

  if (launch_plan(seq_lens, batch, sq, max_pages, ppg, workspace, L, reinterpret_cast<__nv_bfloat16*>(out), lse,
                  stream) != cudaSuccess)
    return MLA_ERR_CUDA;
  DecodeParams p;
  p.q_abs = reinterpret_cast<const __nv_bfloat16*>(q_absorbed);
  p.q_rope = reinterpret_cast<const __nv_bfloat16*>(q_rope);
  p.kv_quant = quant ? static_cast<const uint8_t*>(kv_cache) : nullptr;
  p.kv_bf16 = quant ? nullptr : static_cast<const uint8_t*>(kv_cache);
  p.sp_slots = nullptr;
  p.topk = 0;
  p.tree_nodes = 0;
  p.skip_chunk7 = 0;
  p.block_table = block_table;
  p.batch = batch;
  p.sq = sq;
  p.pairs_per_group = ppg;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.fp8_fallback = 0;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ws = static_cast<uint8_t*>(workspace);
  p.L = L;
  // The three kernels are chained with programmatic dependent launch, so the
  // attention kernel's prologue overlaps the planner and the merge kernel's
  // launch overlaps the attention kernel's tail.  A call with the profiling
  // hook set records its events around the attention kernel and launches the
  // kernels without that overlap, so that the events bracket it alone.
  cudaEvent_t ev0 = g_prof_before, ev1 = g_prof_after;
  g_prof_before = g_prof_after = nullptr;
  const bool pdl = ev0 == nullptr;
  if (ev0 && cudaEventRecord(ev0, stream) != cudaSuccess) return MLA_ERR_CUDA;
  cudaError_t le;
  if (kind == CacheKind::kFp8) le = launch_decode_fp8(p, ppg * sq, pdl, stream);
  else if (kind == CacheKind::kFp4) le = launch_decode_fp4(p, ppg * sq, pdl, stream);
  else if (kind == CacheKind::kFp8V41) le = launch_decode_fp8_v41(p, ppg * sq, pdl, stream);
  else if (kind == CacheKind::kFp4V41) le = launch_decode_fp4_v41(p, ppg * sq, pdl, stream);
  else le = launch_decode_bf16(maps, p, ppg * sq, pdl, stream);
  if (le != cudaSuccess) return MLA_ERR_CUDA;
  if (ev1 && cudaEventRecord(ev1, stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (launch_combine_plan(workspace, L, batch, sq, p.out, lse, pdl, stream) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

// Library-owned scratch of mla_decode_bf16_noalloc: the plan header, the
// split-KV plan and the fp32 partial outputs, for callers that cannot hand
// the library device memory.  40 MiB holds the partials of 76 CTA pairs (the
// 152 SMs of a GB300: 152 slots x 128 heads x 512 bf16 = 19 MiB) plus the
// plan of up to kStaticMaxRows query rows, with room to spare.  One copy per
// device, shared by every call on that device.
constexpr size_t kStaticScratchBytes = size_t{40} << 20;
constexpr int kStaticMaxRows = 8192;
constexpr int kStaticMaxDevices = 64;
static __device__ __align__(256) uint8_t g_static_scratch[kStaticScratchBytes];

std::mutex g_static_mu;
void* g_static_ptr[kStaticMaxDevices] = {};

// Device address of this device's copy of the scratch, looked up once per
// device (with that device current) and cached.
int static_scratch(void** ptr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  if (dev < 0 || dev >= kStaticMaxDevices) return MLA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_static_mu);
  if (!g_static_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_static_scratch) != cudaSuccess || !p) {
      cudaGetLastError();
      return MLA_ERR_CUDA;
    }
    g_static_ptr[dev] = p;
  }
  *ptr = g_static_ptr[dev];
  return MLA_OK;
}

constexpr int kMaxTopk = 16384;
constexpr int kMaxExpandRows = 1 << 24;    // tokens of one expansion (work items stay below 2^31)
constexpr int kMaxPrefillRows = 1 << 24;   // packed queries or keys of one prefill

// Sparse top-k decode: compact the slot lists, plan the B*Sq query rows as a
// batch of rows with one query each, gather-attend, merge.
int run_sparse(const uint16_t* q_absorbed, const uint16_t* q_rope, const void* kv_cache, const int32_t* token_slots,
               int batch, int sq, int topk, int num_heads, int num_pages, int page_size, float softmax_scale,
               uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream_ptr) {
  if (!q_absorbed || !q_rope || !kv_cache || !token_slots || !out || !lse || !workspace) return MLA_ERR_INVALID_ARG;
  if (batch < 0 || sq <= 0 || topk <= 0 || num_pages <= 0 || !std::isfinite(softmax_scale) || !(softmax_scale > 0.f))
    return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads || page_size != kPage || topk > kMaxTopk) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(batch) * sq > kMaxRows) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * kPage >= INT_MAX / 2) return MLA_ERR_UNSUPPORTED;
  if (!aligned(q_absorbed, 16) || !aligned(q_rope, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(token_slots, 4) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const int pairs = decode_max_pairs();
  if (pairs <= 0) return MLA_ERR_CUDA;
  const int rows = batch * sq;
  const WsLayout L = ws_layout(rows, 1, pairs, topk);
  if (workspace_bytes < L.total) return MLA_ERR_WORKSPACE;
  const int max_pages = (topk + kPage - 1) / kPage;
  const int ppg = pairs_for(pairs, static_cast<long long>(rows) * max_pages);
  if (launch_sparse_prep(token_slots, rows, topk, num_pages * kPage, workspace, L, stream) != cudaSuccess)
    return MLA_ERR_CUDA;
  const int32_t* counts = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(workspace) + L.sp_lens);
  if (launch_plan(counts, rows, 1, max_pages, ppg, workspace, L, reinterpret_cast<__nv_bfloat16*>(out), lse,
                  stream) != cudaSuccess)
    return MLA_ERR_CUDA;
  DecodeParams p;
  memset(&p, 0, sizeof(p));
  p.q_abs = reinterpret_cast<const __nv_bfloat16*>(q_absorbed);
  p.q_rope = reinterpret_cast<const __nv_bfloat16*>(q_rope);
  p.kv_bf16 = static_cast<const uint8_t*>(kv_cache);
  p.block_table = nullptr;
  p.batch = rows;
  p.sq = 1;
  p.pairs_per_group = ppg;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.sp_slots = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(workspace) + L.sp_slots);
  p.topk = topk;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ws = static_cast<uint8_t*>(workspace);
  p.L = L;
  cudaEvent_t ev0 = g_prof_before, ev1 = g_prof_after;
  g_prof_before = g_prof_after = nullptr;
  const bool pdl = ev0 == nullptr;
  if (ev0 && cudaEventRecord(ev0, stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (launch_decode_sparse(p, ppg, pdl, stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (ev1 && cudaEventRecord(ev1, stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (launch_combine_plan(workspace, L, rows, 1, p.out, lse, pdl, stream) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

// Pages per pair of a small tree decode, at eight, four and two: eight nodes over
// 200 tokens 22.7, 16.6 and 16.6 us, over 1008 24.7, 18.7 and 20.8, over 4096 24.8,
// 26.7 and 25.3; 4 x 8 over 500 20.7, 20.7 and 24.7, over 1008 28.7, 27.0 and 27.6.
constexpr long long kTreePagesPerPair = 4;

// A quantised cache's tree decode first widens the live pages to bf16 rows, once
// for all nodes, when the workspace has room for them: the attention then runs
// at the bf16 rate.  Two nodes pay for it already: 64 x 2 nodes over 4096 fp8
// tokens take 205 us so and 322 over the codes (fp4: 182 and 298), 64 x 4 272 and
// 583, 8 x 16 over 16,384 361 and 1070; small calls gain too (1 x 2 over 500: 21 and
// 45).  The weights P are rounded to bf16 so, and to f16 over the codes (to bf16
// where f16 does not hold an input), as in the decode.
constexpr int kWidenNodes = 2;
size_t widened_bytes(int batch, int max_pages) {
  return static_cast<size_t>(batch) * max_pages * kPage * kRow * 2;
}

// Tree decode: the drafted nodes' masks and lengths, then the split planner
// over the batch * nodes rows with one query each, the attention, the merge.
int run_tree(CacheKind kind, const uint16_t* q_absorbed, const uint16_t* q_rope, const void* kv_cache,
             const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents, const int32_t* n_nodes,
             int batch, int nodes, int num_heads, int num_pages, int page_size, int max_pages, float softmax_scale,
             uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream_ptr) {
  if (!parents || nodes <= 0) return MLA_ERR_INVALID_ARG;
  int st = validate_common(q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, 1, num_heads, num_pages,
                           page_size, max_pages, softmax_scale, out, lse, workspace);
  if (st != MLA_OK) return st;
  if (nodes > kMaxNodes || static_cast<long long>(batch) * nodes > kMaxRows) return MLA_ERR_UNSUPPORTED;
  // the planner's page totals over the rows are 32-bit
  if (static_cast<long long>(batch) * nodes * max_pages >= (1ll << 30)) return MLA_ERR_UNSUPPORTED;
  // query rows are read and output rows written 32 bytes at a time
  if (!aligned(q_absorbed, 32) || !aligned(q_rope, 32) || !aligned(out, 32) || !aligned(parents, 4) ||
      !aligned(n_nodes, 4))
    return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const int pairs = decode_max_pairs();
  if (pairs <= 0) return MLA_ERR_CUDA;
  const int rows = batch * nodes;
  const WsLayout L = ws_layout(rows, 1, pairs, 0, true);
  if (workspace_bytes < L.total) return MLA_ERR_WORKSPACE;
  const int ppg = pairs_for(pairs, static_cast<long long>(rows) * max_pages, kTreePagesPerPair);
  const bool quant = kind != CacheKind::kBf16;
  const bool widen = quant && nodes >= kWidenNodes && workspace_bytes >= L.total + widened_bytes(batch, max_pages) &&
                     static_cast<long long>(batch) * max_pages * kPage < INT_MAX / 2;
  // The bf16 kernel's rows are planned node by node: pairs that work on
  // different nodes of a sequence then read its rows at about the same time,
  // and from L2, when the batch's rows together exceed it.
  const bool by_node = widen || !quant;
  auto encode = encode_fn();
  if (!encode) return MLA_ERR_CUDA;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(out);
  if (launch_tree_prep(parents, n_nodes, seq_lens, batch, nodes, max_pages, by_node, workspace, L, stream) != cudaSuccess)
    return MLA_ERR_CUDA;
  uint8_t* rows16 = static_cast<uint8_t*>(workspace) + L.total;
  if (widen) {
    RowsParams r;
    memset(&r, 0, sizeof(r));
    r.cache = static_cast<uint8_t*>(const_cast<void*>(kv_cache));
    r.block_table = block_table;
    r.seq_lens = seq_lens;
    r.batch = batch;
    r.num_pages = num_pages;
    r.max_pages = max_pages;
    r.out = reinterpret_cast<__nv_bfloat16*>(rows16);
    r.status = &static_cast<PlanHeader*>(workspace)->status;
    const RowFormat fmt = kind == CacheKind::kFp8 ? RowFormat::kFp8 : kind == CacheKind::kFp4 ? RowFormat::kFp4
                        : kind == CacheKind::kFp8V41 ? RowFormat::kFp8V41 : RowFormat::kFp4V41;
    if (launch_widen(fmt, r, stream) != cudaSuccess) return MLA_ERR_CUDA;
  }
  const int32_t* row_lens = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(workspace) + L.sp_lens);
  // A small call whose rows are cut into three or more parts anyway is cut into
  // even ones: with a cost on starting a row, some pairs got no page and others
  // seven (8 nodes over 1000 tokens 20.6 and 18.6 us; where all pairs are in
  // use, even cuts fall across rows: 8 over 4096 25.7 and 29.1).
  const bool even = ppg < pairs && 3 * rows <= ppg;
  if (launch_plan(row_lens, rows, 1, max_pages, ppg, workspace, L, nullptr, nullptr, stream,
                  even ? 0 : -1) != cudaSuccess)
    return MLA_ERR_CUDA;
  DecodeParams p;
  memset(&p, 0, sizeof(p));
  p.q_abs = reinterpret_cast<const __nv_bfloat16*>(q_absorbed);
  p.q_rope = reinterpret_cast<const __nv_bfloat16*>(q_rope);
  p.kv_quant = quant ? static_cast<const uint8_t*>(kv_cache) : nullptr;
  p.kv_bf16 = widen ? rows16 : quant ? nullptr : static_cast<const uint8_t*>(kv_cache);
  p.block_table = widen ? nullptr : block_table;
  p.skip_chunk7 = widen && (kind == CacheKind::kFp8V41 || kind == CacheKind::kFp4V41);
  p.batch = rows;
  p.sq = 1;
  p.pairs_per_group = ppg;
  p.num_pages = widen ? batch * max_pages : num_pages;
  p.max_pages = max_pages;
  p.tree_nodes = nodes;
  p.tree_seqs = batch;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = o;
  p.lse = lse;
  p.ws = static_cast<uint8_t*>(workspace);
  p.L = L;
  cudaEvent_t ev0 = g_prof_before, ev1 = g_prof_after;
  g_prof_before = g_prof_after = nullptr;
  const bool pdl = ev0 == nullptr;
  if (ev0 && cudaEventRecord(ev0, stream) != cudaSuccess) return MLA_ERR_CUDA;
  cudaError_t le;
  if (by_node) le = launch_tree(encode, p, ppg, pdl, stream);
  else if (kind == CacheKind::kFp8) le = launch_tree_fp8(p, ppg, pdl, stream);
  else if (kind == CacheKind::kFp4) le = launch_tree_fp4(p, ppg, pdl, stream);
  else if (kind == CacheKind::kFp8V41) le = launch_tree_fp8_v41(p, ppg, pdl, stream);
  else le = launch_tree_fp4_v41(p, ppg, pdl, stream);
  if (le != cudaSuccess) return MLA_ERR_CUDA;
  if (ev1 && cudaEventRecord(ev1, stream) != cudaSuccess) return MLA_ERR_CUDA;
  le = by_node ? launch_combine_tree(workspace, L, rows, batch, o, lse, pdl, stream)
               : launch_combine_plan(workspace, L, rows, 1, o, lse, pdl, stream, true);
  if (le != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

// Row strides (values) a 16-byte access or a TMA map takes.
constexpr int kMaxRopeRows = 1 << 24, kMaxRopeHeads = 4096;

bool stride_ok(size_t s) { return s > 0 && s % 8 == 0 && s < (size_t{1} << 38); }

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Append (c_kv non-null) or gather (out non-null) of packed rows.
int run_rows(RowFormat fmt, const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
             const void* cache, const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_rows, int batch,
             int rows, int num_pages, int page_size, int max_pages, uint16_t* out, bool append, void* workspace,
             size_t workspace_bytes, void* stream, const RowsRope* rope = nullptr) {
  if (!cache || !block_table || !seq_lens || !cu_rows || !workspace || (append ? !c_kv || !k_rope : !out))
    return MLA_ERR_INVALID_ARG;
  if (batch < 0 || rows < 0 || num_pages <= 0 || max_pages <= 0) return MLA_ERR_INVALID_ARG;
  if (page_size != kPage || batch > kMaxRows) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * kPage >= INT_MAX / 2 ||
      static_cast<long long>(max_pages) * kPage >= INT_MAX / 2 || rows >= INT_MAX / 2)
    return MLA_ERR_UNSUPPORTED;
  if (!aligned(cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_rows, 4) ||
      !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (append) {
    if (!aligned(c_kv, 16) || !aligned(k_rope, 16) || !stride_ok(c_stride) || !stride_ok(r_stride))
      return MLA_ERR_INVALID_ARG;
  } else if (!aligned(out, 16)) {
    return MLA_ERR_INVALID_ARG;
  }
  if (workspace_bytes < sizeof(PlanHeader)) return MLA_ERR_WORKSPACE;
  if (batch == 0 || rows == 0) return MLA_OK;
  RowsParams p;
  p.c_kv = reinterpret_cast<const __nv_bfloat16*>(c_kv);
  p.k_rope = reinterpret_cast<const __nv_bfloat16*>(k_rope);
  p.c_stride = static_cast<long long>(c_stride);
  p.r_stride = static_cast<long long>(r_stride);
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_rows = cu_rows;
  p.batch = batch;
  p.rows = rows;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.status = &static_cast<PlanHeader*>(workspace)->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = rope ? launch_append_rope(fmt, p, *rope, st) : launch_rows(fmt, p, append, st);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

bool rope_ok(const mla_rope* rope) { return rope && std::isfinite(rope->scale); }

int run_append_rope(RowFormat fmt, const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                    const int32_t* positions, const mla_rope* rope, void* cache, const int32_t* block_table,
                    const int32_t* seq_lens, const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size,
                    int max_pages, void* workspace, size_t workspace_bytes, void* stream) {
  if (!rope_ok(rope) || !aligned(positions, 4)) return MLA_ERR_INVALID_ARG;
  const RowsRope r = {positions, *rope};
  return run_rows(fmt, c_kv, c_stride, k_rope, r_stride, cache, block_table, seq_lens, cu_rows, batch, rows, num_pages,
                  page_size, max_pages, nullptr, true, workspace, workspace_bytes, stream, &r);
}

}  // namespace

// Only the C ABI below is exported (the library is built with hidden
// visibility), so a process may load several copies without their internals
// binding to each other.
#pragma GCC visibility push(default)
extern "C" {

int mla_up_project_wuv(const uint16_t* latent, const uint16_t* w_uv, int rows, int num_heads, int d_v,
                       uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!latent || !w_uv || !out || !workspace || rows < 0) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads || d_v != 128) return MLA_ERR_UNSUPPORTED;
  if (rows > kMaxRows) return MLA_ERR_UNSUPPORTED;
  if (!aligned(latent, 16) || !aligned(w_uv, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(PlanHeader)) return MLA_ERR_WORKSPACE;
  if (rows == 0) return MLA_OK;
  auto fn = encode_fn();
  if (!fn) return MLA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(static_cast<uint8_t*>(workspace) + offsetof(PlanHeader, abort_flag), 0, sizeof(int), st) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  return launch_wuv(fn, latent, w_uv, rows, out, workspace, st) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_cache_append_bf16(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                          uint16_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kBf16, c_kv, c_stride, k_rope, r_stride, kv_cache, block_table, seq_lens, cu_rows, batch,
                  rows, num_pages, page_size, max_pages, nullptr, true, workspace, workspace_bytes, stream);
}

int mla_cache_gather_bf16(const uint16_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kBf16, nullptr, 0, nullptr, 0, kv_cache, block_table, seq_lens, cu_rows, batch, rows,
                  num_pages, page_size, max_pages, out, false, workspace, workspace_bytes, stream);
}

int mla_cache_append_fp8(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                          uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp8, c_kv, c_stride, k_rope, r_stride, kv_cache, block_table, seq_lens, cu_rows, batch,
                  rows, num_pages, page_size, max_pages, nullptr, true, workspace, workspace_bytes, stream);
}

int mla_cache_gather_fp8(const uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp8, nullptr, 0, nullptr, 0, kv_cache, block_table, seq_lens, cu_rows, batch, rows,
                  num_pages, page_size, max_pages, out, false, workspace, workspace_bytes, stream);
}

int mla_cache_append_fp4(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                          uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp4, c_kv, c_stride, k_rope, r_stride, kv_cache, block_table, seq_lens, cu_rows, batch,
                  rows, num_pages, page_size, max_pages, nullptr, true, workspace, workspace_bytes, stream);
}

int mla_cache_gather_fp4(const uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp4, nullptr, 0, nullptr, 0, kv_cache, block_table, seq_lens, cu_rows, batch, rows,
                  num_pages, page_size, max_pages, out, false, workspace, workspace_bytes, stream);
}

int mla_cache_append_fp8_v41(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                          uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp8V41, c_kv, c_stride, k_rope, r_stride, kv_cache, block_table, seq_lens, cu_rows, batch,
                  rows, num_pages, page_size, max_pages, nullptr, true, workspace, workspace_bytes, stream);
}

int mla_cache_gather_fp8_v41(const uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp8V41, nullptr, 0, nullptr, 0, kv_cache, block_table, seq_lens, cu_rows, batch, rows,
                  num_pages, page_size, max_pages, out, false, workspace, workspace_bytes, stream);
}

int mla_cache_append_fp4_v41(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                          uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp4V41, c_kv, c_stride, k_rope, r_stride, kv_cache, block_table, seq_lens, cu_rows, batch,
                  rows, num_pages, page_size, max_pages, nullptr, true, workspace, workspace_bytes, stream);
}

int mla_cache_gather_fp4_v41(const uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* cu_rows, int batch, int rows, int num_pages, int page_size, int max_pages,
                          uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return run_rows(RowFormat::kFp4V41, nullptr, 0, nullptr, 0, kv_cache, block_table, seq_lens, cu_rows, batch, rows,
                  num_pages, page_size, max_pages, out, false, workspace, workspace_bytes, stream);
}

int mla_cache_append_rope_bf16(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                               const int32_t* positions, const mla_rope* rope, uint16_t* kv_cache,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_rows, int batch,
                               int rows, int num_pages, int page_size, int max_pages, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return run_append_rope(RowFormat::kBf16, c_kv, c_stride, k_rope, r_stride, positions, rope, kv_cache, block_table,
                         seq_lens, cu_rows, batch, rows, num_pages, page_size, max_pages, workspace, workspace_bytes,
                         stream);
}

int mla_cache_append_rope_fp8(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                               const int32_t* positions, const mla_rope* rope, uint8_t* kv_cache,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_rows, int batch,
                               int rows, int num_pages, int page_size, int max_pages, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return run_append_rope(RowFormat::kFp8, c_kv, c_stride, k_rope, r_stride, positions, rope, kv_cache, block_table,
                         seq_lens, cu_rows, batch, rows, num_pages, page_size, max_pages, workspace, workspace_bytes,
                         stream);
}

int mla_cache_append_rope_fp4(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                               const int32_t* positions, const mla_rope* rope, uint8_t* kv_cache,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_rows, int batch,
                               int rows, int num_pages, int page_size, int max_pages, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return run_append_rope(RowFormat::kFp4, c_kv, c_stride, k_rope, r_stride, positions, rope, kv_cache, block_table,
                         seq_lens, cu_rows, batch, rows, num_pages, page_size, max_pages, workspace, workspace_bytes,
                         stream);
}

int mla_cache_append_rope_fp8_v41(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                               const int32_t* positions, const mla_rope* rope, uint8_t* kv_cache,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_rows, int batch,
                               int rows, int num_pages, int page_size, int max_pages, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return run_append_rope(RowFormat::kFp8V41, c_kv, c_stride, k_rope, r_stride, positions, rope, kv_cache, block_table,
                         seq_lens, cu_rows, batch, rows, num_pages, page_size, max_pages, workspace, workspace_bytes,
                         stream);
}

int mla_cache_append_rope_fp4_v41(const uint16_t* c_kv, size_t c_stride, const uint16_t* k_rope, size_t r_stride,
                               const int32_t* positions, const mla_rope* rope, uint8_t* kv_cache,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_rows, int batch,
                               int rows, int num_pages, int page_size, int max_pages, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return run_append_rope(RowFormat::kFp4V41, c_kv, c_stride, k_rope, r_stride, positions, rope, kv_cache, block_table,
                         seq_lens, cu_rows, batch, rows, num_pages, page_size, max_pages, workspace, workspace_bytes,
                         stream);
}

int mla_rope_init(mla_rope* rope, const double* inv_freq, float scale, int interleaved) {
  if (!rope || !inv_freq || !std::isfinite(scale)) return MLA_ERR_INVALID_ARG;
  for (int i = 0; i < kRopePairs; ++i)
    if (!(std::fabs(inv_freq[i]) <= 1024.0)) return MLA_ERR_INVALID_ARG;
  // 1 / (2 pi) in two parts; the turns a token, modulo one, in units of 2^-64
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  for (int i = 0; i < kRopePairs; ++i) {
    const double p = inv_freq[i] * kHi, rest = std::fma(inv_freq[i], kLo, std::fma(inv_freq[i], kHi, -p));
    double whole;
    const double turn = std::ldexp(std::modf(p, &whole), 32), upper = std::floor(turn);
    const double lower = std::nearbyint(std::ldexp(turn - upper, 32) + std::ldexp(rest, 64));
    rope->turns[i] = (static_cast<uint64_t>(static_cast<int64_t>(upper)) << 32) +
                     static_cast<uint64_t>(static_cast<int64_t>(lower));
  }
  rope->scale = scale;
  rope->interleaved = interleaved != 0;
  return MLA_OK;
}

int mla_rope_frequencies(float base, float factor, int original_tokens, float beta_fast, float beta_slow,
                         double* inv_freq) {
  const double scaling[4] = {base, factor, beta_fast, beta_slow};
  return mla_rope_frequencies_f64(scaling, original_tokens, inv_freq);
}

int mla_rope_frequencies_f64(const double* scaling, int original_tokens, double* inv_freq) {
  if (!scaling || !inv_freq) return MLA_ERR_INVALID_ARG;
  const double base = scaling[0], factor = scaling[1], beta_fast = scaling[2], beta_slow = scaling[3];
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) ||
      original_tokens <= 0 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
    return MLA_ERR_INVALID_ARG;
  const double ln_base = std::log(base);
  // the pair that turns `n` times over the original length
  auto pair = [&](double n) { return kDr * std::log(original_tokens / (n * 6.283185307179586)) / (2 * ln_base); };
  const double low = std::fmax(std::floor(pair(beta_fast)), 0.0);
  const double high = std::fmin(std::ceil(pair(beta_slow)), kDr - 1.0);
  for (int i = 0; i < kRopePairs; ++i) {
    const double f = std::exp(-ln_base * i / kRopePairs);
    const double ramp = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
    inv_freq[i] = f / factor * ramp + f * (1.0 - ramp);
  }
  return MLA_OK;
}

int mla_rope_bf16(const uint16_t* x, const size_t* strides, const int32_t* positions, int rows, int heads,
                  const mla_rope* rope, int inverse, uint16_t* out, void* stream) {
  if (!x || !strides || !positions || !out || !rope_ok(rope) || rows < 0 || heads < 0) return MLA_ERR_INVALID_ARG;
  if (rows > kMaxRopeRows || heads > kMaxRopeHeads) return MLA_ERR_UNSUPPORTED;
  for (int i = 0; i < 4; ++i)
    if (!stride_ok(strides[i])) return MLA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4)) return MLA_ERR_INVALID_ARG;
  if (rows == 0 || heads == 0) return MLA_OK;
  // in place every vector stays where it is
  if (x == out && ((rows > 1 && strides[0] != strides[2]) || (heads > 1 && strides[1] != strides[3]))) return MLA_ERR_INVALID_ARG;
  RopeParams p;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.x_t = static_cast<long long>(strides[0]);
  p.x_h = static_cast<long long>(strides[1]);
  p.out_t = static_cast<long long>(strides[2]);
  p.out_h = static_cast<long long>(strides[3]);
  p.positions = positions;
  p.rows = rows;
  p.heads = heads;
  p.inverse = inverse != 0;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.rope = *rope;
  return launch_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_expand_kv(const uint16_t* latent, size_t row_stride, const uint16_t* w_uk, const uint16_t* w_uv, int rows,
                  int num_heads, int d_v, uint16_t* k_nope, uint16_t* v, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (!latent || !w_uk || !w_uv || !k_nope || !v || !workspace || rows < 0) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads || d_v != 128) return MLA_ERR_UNSUPPORTED;
  if (rows > kMaxExpandRows) return MLA_ERR_UNSUPPORTED;
  if (!stride_ok(row_stride) || row_stride < static_cast<size_t>(kDc)) return MLA_ERR_INVALID_ARG;
  if (!aligned(latent, 16) || !aligned(w_uk, 16) || !aligned(w_uv, 16) || !aligned(k_nope, 32) || !aligned(v, 32) ||
      !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(PlanHeader)) return MLA_ERR_WORKSPACE;
  if (rows == 0) return MLA_OK;
  auto fn = encode_fn();
  const int sms = sm_count();
  if (!fn || sms <= 0) return MLA_ERR_CUDA;
  return launch_expand(fn, latent, static_cast<long long>(row_stride), w_uk, w_uv, rows, k_nope, v, workspace, sms,
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

int mla_workspace_size_prefill(int batch, int num_q, size_t* bytes) {
  if (!bytes || batch < 0 || num_q < 0) return MLA_ERR_INVALID_ARG;
  if (batch > kMaxRows || num_q > kMaxPrefillRows) return MLA_ERR_UNSUPPORTED;
  *bytes = prefill_ws(batch, num_q).total;
  return MLA_OK;
}

int mla_prefill_bf16(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* k_nope, const uint16_t* k_rope,
                     const uint16_t* v, const size_t* strides, const int32_t* cu_q, const int32_t* cu_k, int batch,
                     int num_q, int num_k, int num_heads, int causal, float softmax_scale, uint16_t* out, float* lse,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!q_nope || !q_rope || !strides || !cu_q || !cu_k || !out || !lse || !workspace) return MLA_ERR_INVALID_ARG;
  if (batch < 0 || num_q < 0 || num_k < 0 || !std::isfinite(softmax_scale) || !(softmax_scale > 0.f))
    return MLA_ERR_INVALID_ARG;
  if (num_k > 0 && (!k_nope || !k_rope || !v)) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads) return MLA_ERR_UNSUPPORTED;
  if (batch > kMaxRows || num_q > kMaxPrefillRows || num_k > kMaxPrefillRows) return MLA_ERR_UNSUPPORTED;
  for (int i = 0; i < 9; ++i)
    if (!stride_ok(strides[i])) return MLA_ERR_INVALID_ARG;
  if (!aligned(q_nope, 16) || !aligned(q_rope, 16) || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16) ||
      !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(out, 32) || !aligned(lse, 4) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < prefill_ws(batch, num_q).total) return MLA_ERR_WORKSPACE;
  if (batch == 0 || num_q == 0) return MLA_OK;
  auto fn = encode_fn();
  const int sms = sm_count();
  if (!fn || sms <= 0) return MLA_ERR_CUDA;
  PrefillParams p;
  // with no key nothing is read through the key pointers; the maps need valid addresses all the same
  const uint16_t* any = q_nope;
  p.q_nope = reinterpret_cast<const __nv_bfloat16*>(q_nope);
  p.q_rope = reinterpret_cast<const __nv_bfloat16*>(q_rope);
  p.k_nope = reinterpret_cast<const __nv_bfloat16*>(num_k > 0 ? k_nope : any);
  p.k_rope = reinterpret_cast<const __nv_bfloat16*>(num_k > 0 ? k_rope : any);
  p.v = reinterpret_cast<const __nv_bfloat16*>(num_k > 0 ? v : any);
  long long* s[9] = {&p.qn_t, &p.qn_h, &p.qr_t, &p.qr_h, &p.kn_t, &p.kn_h, &p.kr_t, &p.v_t, &p.v_h};
  for (int i = 0; i < 9; ++i) *s[i] = static_cast<long long>(strides[i]);
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.batch = batch;
  p.nq = num_q;
  p.nk = num_k;
  p.causal = causal != 0;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ws = static_cast<uint8_t*>(workspace);
  return launch_prefill(fn, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_workspace_size_prefill_backward(int batch, int num_q, int num_k, size_t* bytes) {
  if (!bytes || batch < 0 || num_q < 0 || num_k < 0) return MLA_ERR_INVALID_ARG;
  if (batch > kMaxRows || num_q > kMaxPrefillRows || num_k > kMaxPrefillRows) return MLA_ERR_UNSUPPORTED;
  *bytes = backward_ws(batch, num_q, num_k).total;
  return MLA_OK;
}

int mla_prefill_backward_bf16(const uint16_t* d_out, const float* d_lse, const uint16_t* q_nope, const uint16_t* q_rope,
                              const uint16_t* k_nope, const uint16_t* k_rope, const uint16_t* v, const uint16_t* out,
                              const float* lse, const size_t* strides, const int32_t* cu_q, const int32_t* cu_k,
                              int batch, int num_q, int num_k, int num_heads, int causal, float softmax_scale,
                              uint16_t* dq_nope, uint16_t* dq_rope, uint16_t* dk_nope, uint16_t* dk_rope, uint16_t* dv,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!strides || !cu_q || !cu_k || !workspace) return MLA_ERR_INVALID_ARG;
  if (batch < 0 || num_q < 0 || num_k < 0 || !std::isfinite(softmax_scale) || !(softmax_scale > 0.f))
    return MLA_ERR_INVALID_ARG;
  if (num_q > 0 && (!d_out || !q_nope || !q_rope || !out || !lse || !dq_nope || !dq_rope)) return MLA_ERR_INVALID_ARG;
  if (num_k > 0 && (!k_nope || !k_rope || !v || !dk_nope || !dk_rope || !dv)) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads) return MLA_ERR_UNSUPPORTED;
  if (batch > kMaxRows || num_q > kMaxPrefillRows || num_k > kMaxPrefillRows) return MLA_ERR_UNSUPPORTED;
  for (int i = 0; i < 20; ++i)
    if (!stride_ok(strides[i])) return MLA_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(d_out), static_cast<const void*>(q_nope), static_cast<const void*>(q_rope),
                          static_cast<const void*>(k_nope), static_cast<const void*>(k_rope), static_cast<const void*>(v),
                          static_cast<const void*>(out), static_cast<const void*>(dq_nope), static_cast<const void*>(dq_rope),
                          static_cast<const void*>(dk_nope), static_cast<const void*>(dk_rope), static_cast<const void*>(dv)})
    if (!aligned(ptr, 16)) return MLA_ERR_INVALID_ARG;
  if (!aligned(d_lse, 4) || !aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < backward_ws(batch, num_q, num_k).total) return MLA_ERR_WORKSPACE;
  if (batch == 0 || (num_q == 0 && num_k == 0)) return MLA_OK;
  // in place, or two results in one place (other overlaps of views are the caller's to avoid)
  const uint16_t* const tensors[12] = {dq_nope, dq_rope, dk_nope, dk_rope, dv, d_out, q_nope, q_rope, k_nope, k_rope, v, out};
  const int rows_of[12] = {num_q, num_q, num_k, num_k, num_k, num_q, num_q, num_q, num_k, num_k, num_k, num_q};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 12; ++j)
      if (rows_of[i] > 0 && rows_of[j] > 0 && tensors[i] == tensors[j]) return MLA_ERR_INVALID_ARG;
  auto fn = encode_fn();
  const int sms = sm_count();
  if (!fn || sms <= 0) return MLA_ERR_CUDA;
  BackwardParams p;
  // with no query or no key nothing is read through those pointers; the maps need valid addresses all the same
  const uint16_t* any = num_q > 0 ? q_nope : k_nope;
  auto in = [&](const uint16_t* ptr, int n) { return reinterpret_cast<const __nv_bfloat16*>(n > 0 ? ptr : any); };
  p.d_out = in(d_out, num_q);
  p.q_nope = in(q_nope, num_q);
  p.q_rope = in(q_rope, num_q);
  p.k_nope = in(k_nope, num_k);
  p.k_rope = in(k_rope, num_k);
  p.v = in(v, num_k);
  p.out = in(out, num_q);
  p.d_lse = d_lse;
  p.lse = lse;
  long long* s[20] = {&p.qn_t, &p.qn_h, &p.qr_t, &p.qr_h, &p.kn_t, &p.kn_h, &p.kr_t, &p.v_t, &p.v_h, &p.do_t, &p.do_h,
                      &p.dqn_t, &p.dqn_h, &p.dqr_t, &p.dqr_h, &p.dkn_t, &p.dkn_h, &p.dkr_t, &p.dv_t, &p.dv_h};
  for (int i = 0; i < 20; ++i) *s[i] = static_cast<long long>(strides[i]);
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.batch = batch;
  p.nq = num_q;
  p.nk = num_k;
  p.causal = causal != 0;
  p.scale = softmax_scale;
  p.dq_nope = reinterpret_cast<__nv_bfloat16*>(dq_nope);
  p.dq_rope = reinterpret_cast<__nv_bfloat16*>(dq_rope);
  p.dk_nope = reinterpret_cast<__nv_bfloat16*>(dk_nope);
  p.dk_rope = reinterpret_cast<__nv_bfloat16*>(dk_rope);
  p.dv = reinterpret_cast<__nv_bfloat16*>(dv);
  p.ws = static_cast<uint8_t*>(workspace);
  return launch_backward(fn, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_workspace_size_sparse(int batch, int sq, int topk, int num_heads, int page_size, size_t* bytes) {
  if (!bytes || batch < 0 || sq <= 0 || topk <= 0) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads || page_size != kPage || topk > kMaxTopk) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(batch) * sq > kMaxRows) return MLA_ERR_UNSUPPORTED;
  const int pairs = decode_max_pairs();
  if (pairs <= 0) return MLA_ERR_CUDA;
  *bytes = ws_layout(batch > 0 ? batch * sq : 1, 1, pairs, topk).total;
  return MLA_OK;
}

int mla_decode_sparse_bf16(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint16_t* kv_cache,
                           const int32_t* token_slots, int batch, int sq, int topk, int num_heads, int num_pages,
                           int page_size, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return run_sparse(q_absorbed, q_rope, kv_cache, token_slots, batch, sq, topk, num_heads, num_pages, page_size,
                    softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

int mla_workspace_size(int batch, int sq, int num_heads, int page_size, size_t* bytes) {
  if (!bytes || batch < 0 || sq <= 0) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads || page_size != kPage || sq > kMaxSq) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(batch) * sq > kMaxRows) return MLA_ERR_UNSUPPORTED;
  const int pairs = decode_max_pairs();
  if (pairs <= 0) return MLA_ERR_CUDA;
  *bytes = ws_layout(batch > 0 ? batch : 1, sq, pairs).total;
  return MLA_OK;
}

int mla_decode_bf16(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint16_t* kv_cache,
                    const int32_t* block_table, const int32_t* seq_lens, int batch, int sq, int num_heads,
                    int num_pages, int page_size, int max_pages, float softmax_scale, uint16_t* out, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return run_decode(CacheKind::kBf16, q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads,
                    num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

int mla_decode_bf16_noalloc(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint16_t* kv_cache,
                            const int32_t* block_table, const int32_t* seq_lens, int batch, int sq, int num_heads,
                            int num_pages, int page_size, int max_pages, float softmax_scale, uint16_t* out,
                            float* lse, int* device_status, void* stream) {
  void* scratch = nullptr;
  int st = static_scratch(&scratch);
  if (st != MLA_OK) return st;
  st = validate_common(q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads, num_pages,
                       page_size, max_pages, softmax_scale, out, lse, scratch);
  if (st != MLA_OK) return st;
  if (device_status && !aligned(device_status, 4)) return MLA_ERR_INVALID_ARG;
  if (static_cast<long long>(batch) * sq > kStaticMaxRows) return MLA_ERR_WORKSPACE;
  const int pairs = decode_max_pairs();
  if (pairs <= 0) return MLA_ERR_CUDA;
  if (ws_layout(batch, sq, pairs).total > kStaticScratchBytes) return MLA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the status word and the abort flag must start at zero for this call
  if (cudaMemsetAsync(scratch, 0, sizeof(PlanHeader), s) != cudaSuccess) return MLA_ERR_CUDA;
  st = run_decode(CacheKind::kBf16, q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads,
                  num_pages, page_size, max_pages, softmax_scale, out, lse, scratch, kStaticScratchBytes, stream);
  if (st != MLA_OK) return st;
  if (device_status &&
      cudaMemcpyAsync(device_status, scratch, sizeof(int), cudaMemcpyDeviceToDevice, s) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

int mla_decode_fp8(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                   const int32_t* block_table, const int32_t* seq_lens, int batch, int sq, int num_heads,
                   int num_pages, int page_size, int max_pages, float softmax_scale, uint16_t* out, float* lse,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return run_decode(CacheKind::kFp8, q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads,
                    num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

int mla_decode_fp4(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                   const int32_t* block_table, const int32_t* seq_lens, int batch, int sq, int num_heads,
                   int num_pages, int page_size, int max_pages, float softmax_scale, uint16_t* out, float* lse,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return run_decode(CacheKind::kFp4, q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads,
                    num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

int mla_decode_fp8_v41(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                       const int32_t* block_table, const int32_t* seq_lens, int batch, int sq, int num_heads,
                       int num_pages, int page_size, int max_pages, float softmax_scale, uint16_t* out, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream) {
  return run_decode(CacheKind::kFp8V41, q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads,
                    num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

int mla_decode_fp4_v41(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                       const int32_t* block_table, const int32_t* seq_lens, int batch, int sq, int num_heads,
                       int num_pages, int page_size, int max_pages, float softmax_scale, uint16_t* out, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream) {
  return run_decode(CacheKind::kFp4V41, q_absorbed, q_rope, kv_cache, block_table, seq_lens, batch, sq, num_heads,
                    num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

int mla_workspace_size_tree(int batch, int nodes, int num_heads, int page_size, size_t* bytes) {
  if (!bytes || batch < 0 || nodes <= 0) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads || page_size != kPage || nodes > kMaxNodes) return MLA_ERR_UNSUPPORTED;
  if (static_cast<long long>(batch) * nodes > kMaxRows) return MLA_ERR_UNSUPPORTED;
  const int pairs = decode_max_pairs();
  if (pairs <= 0) return MLA_ERR_CUDA;
  *bytes = ws_layout(batch > 0 ? batch * nodes : 1, 1, pairs, 0, true).total;
  return MLA_OK;
}

int mla_workspace_size_tree_widened(int batch, int nodes, int num_heads, int page_size, int max_pages, size_t* bytes) {
  if (max_pages <= 0) return MLA_ERR_INVALID_ARG;
  const int rc = mla_workspace_size_tree(batch, nodes, num_heads, page_size, bytes);
  if (rc == MLA_OK) *bytes += widened_bytes(batch, max_pages);
  return rc;
}

int mla_decode_tree_bf16(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint16_t* kv_cache,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* n_nodes, int batch, int nodes, int num_heads, int num_pages, int page_size,
                         int max_pages, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return run_tree(CacheKind::kBf16, q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, n_nodes, batch, nodes,
                  num_heads, num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes,
                  stream);
}

int mla_decode_tree_fp8(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* n_nodes, int batch, int nodes, int num_heads, int num_pages, int page_size,
                         int max_pages, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return run_tree(CacheKind::kFp8, q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, n_nodes, batch, nodes,
                  num_heads, num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes,
                  stream);
}

int mla_decode_tree_fp4(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* n_nodes, int batch, int nodes, int num_heads, int num_pages, int page_size,
                         int max_pages, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return run_tree(CacheKind::kFp4, q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, n_nodes, batch, nodes,
                  num_heads, num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes,
                  stream);
}

int mla_decode_tree_fp8_v41(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* n_nodes, int batch, int nodes, int num_heads, int num_pages, int page_size,
                         int max_pages, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return run_tree(CacheKind::kFp8V41, q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, n_nodes, batch, nodes,
                  num_heads, num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes,
                  stream);
}

int mla_decode_tree_fp4_v41(const uint16_t* q_absorbed, const uint16_t* q_rope, const uint8_t* kv_cache,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* n_nodes, int batch, int nodes, int num_heads, int num_pages, int page_size,
                         int max_pages, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return run_tree(CacheKind::kFp4V41, q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, n_nodes, batch, nodes,
                  num_heads, num_pages, page_size, max_pages, softmax_scale, out, lse, workspace, workspace_bytes,
                  stream);
}

int mla_combine_splits(const float* partial_out, const float* partial_lse, const int32_t* split_indptr, int rows,
                       int num_heads, uint16_t* out, float* lse, void* stream) {
  if (rows < 0 || !split_indptr || !out || !lse) return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads) return MLA_ERR_UNSUPPORTED;
  if (rows == 0) return MLA_OK;
  if (!partial_out || !partial_lse) return MLA_ERR_INVALID_ARG;
  if (!aligned(partial_out, 16) || !aligned(out, 8)) return MLA_ERR_INVALID_ARG;
  if (launch_combine_indptr(partial_out, partial_lse, split_indptr, rows, reinterpret_cast<__nv_bfloat16*>(out), lse,
                            static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

int mla_profile_next_decode(void* before, void* after) {
  if ((before == nullptr) != (after == nullptr)) return MLA_ERR_INVALID_ARG;
  g_prof_before = static_cast<cudaEvent_t>(before);
  g_prof_after = static_cast<cudaEvent_t>(after);
  return MLA_OK;
}

int mla_get_status(void* workspace, void* stream) {
  if (!workspace) return MLA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return MLA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, workspace, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return MLA_ERR_CUDA;
  // a reported timeout also leaves the abort flag set; both are cleared
  if (v != 0 && (cudaMemset(workspace, 0, sizeof(int)) != cudaSuccess ||
                 cudaMemset(static_cast<uint8_t*>(workspace) + offsetof(PlanHeader, abort_flag), 0, sizeof(int)) !=
                     cudaSuccess))
    return MLA_ERR_CUDA;
  return v;
}

const char* mla_status_string(int code) {
  switch (code) {
    case MLA_OK: return "MLA_OK";
    case MLA_ERR_INVALID_ARG: return "MLA_ERR_INVALID_ARG";
    case MLA_ERR_UNSUPPORTED: return "MLA_ERR_UNSUPPORTED";
    case MLA_ERR_WORKSPACE: return "MLA_ERR_WORKSPACE";
    case MLA_ERR_CUDA: return "MLA_ERR_CUDA";
    case MLA_STATUS_BAD_PAGE: return "MLA_STATUS_BAD_PAGE";
    case MLA_STATUS_TIMEOUT: return "MLA_STATUS_TIMEOUT";
    case MLA_STATUS_BAD_SEQ_LEN: return "MLA_STATUS_BAD_SEQ_LEN";
    case MLA_STATUS_BAD_INDEX: return "MLA_STATUS_BAD_INDEX";
    default: return "MLA_UNKNOWN_STATUS";
  }
}

}  // extern "C"
#pragma GCC visibility pop
