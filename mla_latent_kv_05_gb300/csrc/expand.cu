// Expansion of latent rows into per-head keys and values (the expanded form
// of latent attention): for every token t and head h
//     k_nope[t, h, :] = W_h^UK c_t,     v[t, h, :] = W_h^UV c_t,
// c_t the 512 latent values, W_h^UK and W_h^UV of 128 x 512.  Over n tokens
// this is one product of M = n, K = 512, N = 128 heads x 256.
//
// Bound: 2 n 512 32768 operations against 64 KiB of bf16 written per token,
// so at 8192 tokens the tensor cores need about as long as HBM does for the
// output, and what has to be kept off their path is traffic through L2.
//
// A pair of CTAs computes 256 tokens x 256 columns with cta_group::2 MMAs (M =
// 256, N = 256): each CTA holds half of the weights' rows (rank 0 W^UK, rank 1
// W^UV) and half of the tokens, so an operand crosses L2 once for the pair.
// One head's weights stay in shared memory (128 KiB a CTA) while latent tiles
// stream past them, not the other way round: streaming the 33.5 MB of weights
// past a resident latent tile moves as many bytes, but with the output
// streaming out beside it the two did not overlap in L2 (8192 tokens: 203 us;
// with every pair reading one head's weights, for timing only, 154 us), while
// the latent rows in use are few enough (8 MB) to be served beside it.  The
// output leaves as TMA stores of whole 128-byte lines from a staging buffer,
// and the fp32 accumulators (256 columns of each SM's tensor memory) are
// double-buffered, so writing an item overlaps the next one's products.
//
// Persistent pairs; a work item is (head h, token tile m), and a pair takes a
// contiguous run of items ordered by (block of 32 token tiles, head, tile).
// Per item: 32 K-steps of tcgen05.mma, both operands K-major with 128-byte
// swizzle, in K blocks of 64: the latent through a four-block ring, the
// weights' eight blocks each reloaded as soon as their last use is over.  Warp
// 0 of each rank issues its loads (all counted on rank 0's barriers), warp 1
// of rank 0 the MMAs, warps 4..11 of each rank write (4..7 the keys, 8..11 the
// values; thread = token).  Rows past n are read as zeros and not written.
//
// Measured: 8192 tokens 165 us (1660 TFLOP/s, 3.5 TB/s of HBM), 2048 48, 1000 26.5,
// 130 and fewer 12 (the 33.5 MB of weights alone take 5 us from HBM: 128 heads
// over 76 pairs are two rounds, and the second head's weights are asked for only
// as the first one's products end; with one token tile the roles could swap,
// latents resident and weights streaming, which is not built).  Alone and cold, at
// 4096 tokens, the tensor pipe is active 71 % of the time and HBM at 43 % of its
// rate.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "expand.cuh"
#include "waits.cuh"

namespace mla {

namespace {

constexpr int kThreads = 384;
constexpr int kKBlock = 64;                             // K values per block (128-byte rows)
constexpr int kKBlocks = kDc / kKBlock;                 // 8
constexpr uint32_t kBlock = 128u * 128u;                // 16 KiB: 128 tokens, or weight rows, x 64 values
constexpr int kStages = 4;
constexpr uint32_t kStageOut = 32u * 128u;              // 4 KiB per writer warp: 32 tokens x 64 values
constexpr uint32_t kOffRing = kKBlocks * kBlock;        // after the weights
constexpr uint32_t kOffOut = kOffRing + kStages * kBlock;
constexpr uint32_t kOffBar = kOffOut + 8 * kStageOut;   // 224 KiB
constexpr uint32_t kSmem = kOffBar + 512;
constexpr uint32_t kIdesc = ptx::idesc_bf16(256, 256, 0, 0);

enum Bar {
  WFULL = 0, WEMPTY = WFULL + kKBlocks, CFULL = WEMPTY + kKBlocks, CEMPTY = CFULL + kStages, DFULL = CEMPTY + kStages,
  DEMPTY = DFULL + 2, DRAIN = DEMPTY + 2, NBAR
};

// tiled store from shared memory, in this thread's bulk group
__device__ __forceinline__ void store_4d(const void* tmap, uint32_t src, int x, int y, int z, int w, uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3, %4, %5}], [%1], %6;"
               :: "l"(tmap), "r"(src), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

constexpr int kTileBlock = 32;   // token tiles of a block

// Item i of all: the blocks of kTileBlock token tiles in turn, in each the
// heads, in each head the block's tiles.
__device__ __forceinline__ void item_of(int i, int tiles, int& m, int& h) {
  const int block = i / (kTileBlock * kHeads), left = i - block * (kTileBlock * kHeads);
  const int size = min(kTileBlock, tiles - block * kTileBlock);
  h = left / size;
  m = block * kTileBlock + left - h * size;
}

struct ExpandMaps {
  CUtensorMap c, w[2], out[2];   // latent; W^UK, W^UV; keys, values
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expand_kernel(const __grid_constant__ ExpandMaps maps, int rows, int tiles, PlanHeader* hdr) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t rank = ptx::cluster_ctarank();
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  const uint32_t tmem_slot = sbase + kOffBar + 8u * NBAR;
  if (threadIdx.x == 0) {
    for (int b = 0; b < kKBlocks; ++b) { ptx::mbar_init(BAR(WFULL + b), 1); ptx::mbar_init(BAR(WEMPTY + b), 1); }
    for (int s = 0; s < kStages; ++s) { ptx::mbar_init(BAR(CFULL + s), 1); ptx::mbar_init(BAR(CEMPTY + s), 1); }
    for (int s = 0; s < 2; ++s) { ptx::mbar_init(BAR(DFULL + s), 1); ptx::mbar_init(BAR(DEMPTY + s), 16); }   // both ranks' writer warps
    ptx::mbar_init(BAR(DRAIN), 1);
    ptx::fence_barrier_init();
  }
  if (warp == 2) {
    ptx::pair_tmem_alloc(tmem_slot, 512);
    ptx::pair_tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::cluster_sync();   // both ranks' barriers are initialised before any load or commit of the pair
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 8u * NBAR), 0);
  const bool smem_ok = (sbase & 1023u) == 0;   // the same in both ranks
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  // this pair's items [lo, hi)
  const long long items = static_cast<long long>(tiles) * kHeads;
  const uint32_t pair = ptx::cluster_id_x(), pairs = gridDim.x >> 1;
  const int lo = static_cast<int>(items * pair / pairs);
  const int hi = smem_ok ? static_cast<int>(items * (pair + 1) / pairs) : lo;

  if (warp == 0) {
    // ------------------------------------------------------------ loads (each rank its own halves)
    if (lane == 0) {
      const uint64_t pol = ptx::policy_evict_normal();
      int s = 0, nw = 0, nc = 0;             // ring stage; heads' weights and latent blocks loaded so far
      uint32_t ph = 0;
      bool ok = true;
      int h_last = -1;
      for (int i = lo; i < hi && ok; ++i) {
        int m, h;
        item_of(i, tiles, m, h);
        const bool weights = h != h_last || i == lo;
        h_last = h;
        for (int kb = 0; kb < kKBlocks; ++kb) {
          if (weights) {
            ok = wait_short<true>(BAR(WEMPTY + kb), (nw & 1u) ^ 1u, hdr);
            if (!ok) break;
            if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(WFULL + kb), 2 * kBlock);
            ptx::pair_load_3d(sbase + kb * kBlock, &maps.w[rank], ptx::mapa(BAR(WFULL + kb), 0), kb * kKBlock, 0, h, pol);
          }
          ok = wait_short<true>(BAR(CEMPTY + s), ph ^ 1u, hdr);
          if (!ok) break;
          if (rank == 0) ptx::mbar_arrive_expect_tx(BAR(CFULL + s), 2 * kBlock);
          ptx::pair_load_3d(sbase + kOffRing + static_cast<uint32_t>(s) * kBlock, &maps.c, ptx::mapa(BAR(CFULL + s), 0),
                       kb * kKBlock, m * 256 + static_cast<int>(rank) * 128, 0, pol);
          ++nc;
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
        if (weights) ++nw;
      }
      // no copy may land after the CTA has left: rank 0's barriers count both
      // ranks' bytes (after a wait that gave up, the pause at the end covers
      // what was not waited for here).  Nor any arrival: rank 0's commits arrive in
      // both ranks, and that it has seen its own says nothing about the other's;
      // the commit to DRAIN is the last one.
      if (ok && nc > 0) {
#pragma unroll 1
        for (int b = 0; b < kKBlocks; ++b) {
          if (rank == 0) wait_drain(BAR(WFULL + b), (nw - 1) & 1, hdr);
          wait_short<true>(BAR(WEMPTY + b), (nw - 1) & 1, hdr);
        }
#pragma unroll 1
        for (int b = 0; b < kStages; ++b) {
          const int n = (nc + kStages - 1 - b) / kStages;     // times stage b was armed
          if (rank == 0) wait_drain(BAR(CFULL + b), (n - 1) & 1, hdr);
          wait_short<true>(BAR(CEMPTY + b), (n - 1) & 1, hdr);
        }
        if (rank == 1) wait_short<true>(BAR(DRAIN), 0u, hdr);
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    int s = 0, d = 0;
    uint32_t ph = 0, wph = 0, dph = 0;
    bool ok = true;
#ifdef MLA_TEST_STALL_WAIT
    // Test builds only: a wait on a barrier that nothing arrives on before the end
    // of the kernel, so that its limit runs out and every role leaves through the
    // abort path.
    ok = wait_short_warp<true>(BAR(DRAIN), 0u, hdr);
#endif
    const uint64_t desc_w = ptx::sdesc_sw128(sbase, 16, 1024), desc_c = ptx::sdesc_sw128(sbase + kOffRing, 16, 1024);
    int m, h = -1, h_next = -1, h_last = -1;
    if (lo < hi) item_of(lo, tiles, m, h_next);
    for (int i = lo; i < hi && ok; ++i) {
      h = h_next;
      h_next = -1;
      if (i + 1 < hi) item_of(i + 1, tiles, m, h_next);
      const bool first = h != h_last, last = h_next != h;     // of this head's weights
      h_last = h;
      ok = wait_short_warp<true>(BAR(DEMPTY + d), dph ^ 1u, hdr);
      for (int kb = 0; kb < kKBlocks && ok; ++kb) {
        if (first) ok = wait_short_warp<true>(BAR(WFULL + kb), wph, hdr);
        if (ok) ok = wait_short_warp<true>(BAR(CFULL + s), ph, hdr);
        if (!ok) break;
        ptx::tc_fence_after();
        if (elect_one()) {
          const uint64_t da = desc_c + static_cast<uint64_t>(s) * (kBlock >> 4);
          const uint64_t db = desc_w + static_cast<uint64_t>(kb) * (kBlock >> 4);
#pragma unroll
          for (int k = 0; k < kKBlock / 16; ++k)
            ptx::pair_mma_ss(tmem + 256u * d, da + 2u * k, db + 2u * k, kIdesc, (kb > 0 || k > 0) ? 1u : 0u);
          ptx::pair_commit(BAR(CEMPTY + s));
          if (last) ptx::pair_commit(BAR(WEMPTY + kb));
          if (kb == kKBlocks - 1) ptx::pair_commit(BAR(DFULL + d));
        }
        __syncwarp();
        if (++s == kStages) { s = 0; ph ^= 1u; }
      }
      if (first) wph ^= 1u;
      d ^= 1;
      if (d == 0) dph ^= 1u;
    }
    // every MMA completes before the pair may leave (the commits to rank 1 are
    // waited for there, by its loader)
    if (lo < hi && elect_one()) {   // the lane that issued them
      ptx::pair_commit(BAR(DRAIN));
      wait_drain(BAR(DRAIN), 0u, hdr);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ writers
    const int half = (warp - 4) >> 2;                    // 0: keys, 1: values
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t stage = sbase + kOffOut + static_cast<uint32_t>(warp - 4) * kStageOut;
    uint8_t* stage_row = smem + kOffOut + static_cast<uint32_t>(warp - 4) * kStageOut + lane * 128;
    const uint64_t pol = ptx::policy_evict_first();      // the output leaves L2 first
    int d = 0;
    uint32_t dph = 0;
    for (int i = lo; i < hi; ++i) {
      int m, h;
      item_of(i, tiles, m, h);
      const int row0 = m * 256 + static_cast<int>(rank) * 128 + (warp & 3) * 32;     // the warp's first token
      if (!wait_short_warp(BAR(DFULL + d), dph, hdr)) break;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {                      // 64 columns at a time
        uint32_t r[64];
        ptx::tmem_ld32(tmem + lane_base + 256u * d + 128u * half + 64u * c, r);
        ptx::tmem_ld32(tmem + lane_base + 256u * d + 128u * half + 64u * c + 32u, r + 32);
        ptx::tmem_wait_ld();
        if (c == 1) {
          // this warp has read its part of D
          ptx::tc_fence_before();
          __syncwarp();
          if (elect_one()) ptx::arrive_leader(ptx::mapa(BAR(DEMPTY + d), 0));
        }
        if (row0 < rows) {
          // the last store must have read the staging rows
          if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {                  // 16-byte pieces, 128-byte swizzle
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b =
                  __floats2bfloat162_rn(__uint_as_float(r[8 * q + 2 * e]), __uint_as_float(r[8 * q + 2 * e + 1]));
              o[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(stage_row + ((q ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          ptx::fence_proxy_async_cta();
          __syncwarp();
          if (elect_one()) store_4d(&maps.out[half], stage, 64 * c, h, row0, 0, pol);   // rows past n are clipped
          __syncwarp();
        }
      }
      d ^= 1;
      if (d == 0) dph ^= 1u;
    }
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  // after a wait gave up, loads that rank 1 issued may be in flight uncounted:
  // give them time to land before either CTA leaves
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

cudaError_t launch_expand(PFN_cuTensorMapEncodeTiled_v12000 encode, const void* latent, long long row_stride,
                          const void* w_uk, const void* w_uv, int rows, void* k_nope, void* v, void* hdr, int sms,
                          cudaStream_t stream) {
  if (rows <= 0) return cudaSuccess;
  ExpandMaps maps;
  auto map = [&](CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t n = static_cast<cuuint64_t>(rows);
  {
    const cuuint64_t dims[3] = {kDc, n, 2}, strides[2] = {static_cast<cuuint64_t>(row_stride) * 2, kTmaFar};
    const cuuint32_t box[3] = {kKBlock, 128, 1};
    if (!map(&maps.c, latent, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[3] = {kDc, 128, kHeads}, strides[2] = {kDc * 2, 128 * kDc * 2};
    const cuuint32_t box[3] = {kKBlock, 128, 1};
    if (!map(&maps.w[0], w_uk, 3, dims, strides, box) || !map(&maps.w[1], w_uv, 3, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[4] = {128, kHeads, n, 2}, strides[3] = {256, kHeads * 256, kTmaFar};
    const cuuint32_t box[4] = {64, 1, 32, 1};
    if (!map(&maps.out[0], k_nope, 4, dims, strides, box) || !map(&maps.out[1], v, 4, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = allow_smem(expand_kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  const int tiles = (rows + 255) / 256, pairs = sms / 2 > 0 ? sms / 2 : 1;
  return launch_kernel(expand_kernel, dim3(2 * (pairs < kHeads ? pairs : kHeads)), dim3(kThreads), kSmem, stream, maps,
                       rows, tiles, static_cast<PlanHeader*>(hdr));
}

}  // namespace mla
