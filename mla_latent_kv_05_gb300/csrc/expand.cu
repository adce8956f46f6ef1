// Expansion of latent rows into per-head keys and values (the expanded form
// of latent attention): for every token t and head h
//     k_nope[t, h, :] = W_h^UK c_t,     v[t, h, :] = W_h^UV c_t,
// c_t the 512 latent values, W_h^UK and W_h^UV of 128 x 512.  Over n tokens
// this is one product of M = n, K = 512, N = 128 heads x 256.
//
// Bound: 2 n 512 32768 operations against 64 KiB of bf16 written per token,
// so at 8192 tokens the tensor cores need about twice HBM's time.  The
// latent tile (128 tokens x 512, 128 KiB) therefore stays in shared memory
// while the heads' weights stream past it from L2 (33.5 MB, resident there),
// and the fp32 accumulators are double-buffered in tensor memory so that
// writing a tile overlaps the next one's products.
//
// One persistent CTA per SM.  A work item is (token tile m, head h); a CTA
// takes a contiguous run of items in m-major order, so it loads a latent tile
// once per m it touches.  Per item: D[128 x 256] = C[128 x 512] . [W^UK_h;
// W^UV_h]^T, 32 K-steps of tcgen05.mma M = 128, N = 256, K = 16, both
// operands K-major with 128-byte swizzle.  Warp 0 issues the TMA loads, warp
// 1 the MMAs, warps 4..11 write (4..7 the keys, 8..11 the values; thread =
// token).  Rows past n are read as zeros and not written.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "expand.cuh"

namespace mla {

namespace {

constexpr int kThreads = 384;
constexpr int kKBlock = 64;                             // K values per block (128-byte rows)
constexpr int kKBlocks = kDc / kKBlock;                 // 8
constexpr uint32_t kABlock = 128u * 128u;               // 16 KiB: 128 tokens x 64 values
constexpr uint32_t kBBlock = 2 * kABlock;               // 32 KiB: 128 key rows, then 128 value rows
constexpr int kStages = 3;
constexpr uint32_t kOffB = kKBlocks * kABlock;          // after the latent tile
constexpr uint32_t kOffBar = kOffB + kStages * kBBlock; // 224 KiB
constexpr uint32_t kSmem = kOffBar + 256;
constexpr uint32_t kIdesc = ptx::idesc_bf16(128, 256, 0, 0);

enum Bar {
  AFULL = 0, AEMPTY, BFULL, BEMPTY = BFULL + kStages, DFULL = BEMPTY + kStages, DEMPTY = DFULL + 2, DRAIN = DEMPTY + 2,
  NBAR
};

__global__ void __launch_bounds__(kThreads, 1)
expand_kernel(const __grid_constant__ CUtensorMap tmap_c, const __grid_constant__ CUtensorMap tmap_uk,
              const __grid_constant__ CUtensorMap tmap_uv, int rows, int items, __nv_bfloat16* __restrict__ k_out,
              __nv_bfloat16* __restrict__ v_out, PlanHeader* hdr) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto BAR = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  const uint32_t tmem_slot = sbase + kOffBar + 8u * NBAR;
  if (threadIdx.x == 0) {
    ptx::mbar_init(BAR(AFULL), 1);
    ptx::mbar_init(BAR(AEMPTY), 1);
    for (int s = 0; s < kStages; ++s) { ptx::mbar_init(BAR(BFULL + s), 1); ptx::mbar_init(BAR(BEMPTY + s), 1); }
    for (int s = 0; s < 2; ++s) { ptx::mbar_init(BAR(DFULL + s), 1); ptx::mbar_init(BAR(DEMPTY + s), 256); }
    ptx::mbar_init(BAR(DRAIN), 1);
    ptx::fence_barrier_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 8u * NBAR);
  const bool smem_ok = (sbase & 1023u) == 0;
  if (threadIdx.x == 0 && !smem_ok) set_status(&hdr->status, MLA_ERR_UNSUPPORTED);
  // this CTA's items [lo, hi): item = m * 128 + h
  const int lo = static_cast<int>(static_cast<long long>(items) * blockIdx.x / gridDim.x);
  const int hi = smem_ok ? static_cast<int>(static_cast<long long>(items) * (blockIdx.x + 1) / gridDim.x) : lo;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol = ptx::policy_evict_normal();
      int s = 0, na = 0, nb = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int it = lo; it < hi && ok; ++it) {
        const int m = it / kHeads, h = it - m * kHeads;
        if (it == lo || h == 0) {
          if (!wait_bounded<false>(BAR(AEMPTY), aph ^ 1u, hdr)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(BAR(AFULL), kKBlocks * kABlock);
          for (int kb = 0; kb < kKBlocks; ++kb)
            ptx::tma_load_2d(sbase + kb * kABlock, &tmap_c, BAR(AFULL), kb * kKBlock, m * 128, pol);
          aph ^= 1u;
          ++na;
        }
        for (int kb = 0; kb < kKBlocks; ++kb) {
          if (!wait_bounded<false>(BAR(BEMPTY + s), ph ^ 1u, hdr)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(BAR(BFULL + s), kBBlock);
          const uint32_t dst = sbase + kOffB + static_cast<uint32_t>(s) * kBBlock;
          ptx::tma_load_3d(dst, &tmap_uk, BAR(BFULL + s), kb * kKBlock, 0, h, pol);
          ptx::tma_load_3d(dst + kABlock, &tmap_uv, BAR(BFULL + s), kb * kKBlock, 0, h, pol);
          ++nb;
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
      // no copy may land after the CTA has left: wait for the last phases armed
      if (na > 0) wait_drain(BAR(AFULL), (na - 1) & 1, hdr);
      for (int i = 0; i < kStages; ++i) {
        const int n = (nb + kStages - 1 - i) / kStages;     // times stage i was armed
        if (n > 0) wait_drain(BAR(BFULL + i), (n - 1) & 1, hdr);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int s = 0, d = 0;
    uint32_t ph = 0, aph = 0, dph = 0;
    bool ok = true;
    for (int it = lo; it < hi && ok; ++it) {
      const int h = it % kHeads;
      if (it == lo || h == 0) {
        if (!wait_warp<false>(BAR(AFULL), aph, hdr)) { ok = false; break; }
        aph ^= 1u;
      }
      if (!wait_warp<false>(BAR(DEMPTY + d), dph ^ 1u, hdr)) { ok = false; break; }
      ptx::tc_fence_after();
      for (int kb = 0; kb < kKBlocks; ++kb) {
        if (!wait_warp<false>(BAR(BFULL + s), ph, hdr)) { ok = false; break; }
        ptx::tc_fence_after();
        if (lane == 0) {
          const uint64_t da = ptx::sdesc_sw128(sbase + kb * kABlock, 16, 1024);
          const uint64_t db = ptx::sdesc_sw128(sbase + kOffB + static_cast<uint32_t>(s) * kBBlock, 16, 1024);
#pragma unroll
          for (int k = 0; k < kKBlock / 16; ++k)
            ptx::mma_ss(tmem + 256u * d, da + static_cast<uint64_t>((k * 32) >> 4),
                        db + static_cast<uint64_t>((k * 32) >> 4), kIdesc, (kb > 0 || k > 0) ? 1u : 0u);
          ptx::mma_commit(BAR(BEMPTY + s));
          if (kb == kKBlocks - 1) {
            ptx::mma_commit(BAR(DFULL + d));
            if (h == kHeads - 1) ptx::mma_commit(BAR(AEMPTY));   // the latent tile is done with
          }
        }
        __syncwarp();
        if (++s == kStages) { s = 0; ph ^= 1u; }
      }
      d ^= 1;
      if (d == 0) dph ^= 1u;
    }
    // every MMA this thread issued completes before the CTA may leave
    if (lo < hi && lane == 0) {
      ptx::mma_commit(BAR(DRAIN));
      wait_drain(BAR(DRAIN), 0u, hdr);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ writers
    const int half = (warp - 4) >> 2;                    // 0: keys, 1: values
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int tr = (warp & 3) * 32 + lane;               // token of the tile
    __nv_bfloat16* base = half == 0 ? k_out : v_out;
    int d = 0;
    uint32_t dph = 0;
    for (int it = lo; it < hi; ++it) {
      const int m = it / kHeads, h = it - m * kHeads;
      if (!wait_warp<false>(BAR(DFULL + d), dph, hdr)) break;
      ptx::tc_fence_after();
      const int row = m * 128 + tr;
      __nv_bfloat16* dst = base + (static_cast<size_t>(row) * kHeads + h) * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        ptx::tmem_ld32(tmem + lane_base + 256u * d + 128u * half + 32u * c, r);
        ptx::tmem_wait_ld();
        if (row < rows) {
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
            o[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          ptx::st_global_v8(dst + 32 * c, o);
          ptx::st_global_v8(dst + 32 * c + 16, o + 8);
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(BAR(DEMPTY + d));
      d ^= 1;
      if (d == 0) dph ^= 1u;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_expand(PFN_cuTensorMapEncodeTiled_v12000 encode, const void* latent, long long row_stride,
                          const void* w_uk, const void* w_uv, int rows, void* k_nope, void* v, void* hdr, int sms,
                          cudaStream_t stream) {
  if (rows <= 0) return cudaSuccess;
  CUtensorMap tm_c, tm_uk, tm_uv;
  {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(kDc), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_stride) * 2};
    cuuint32_t box[2] = {kKBlock, 128};
    cuuint32_t es[2] = {1, 1};
    if (encode(&tm_c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(latent), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const void* w[2] = {w_uk, w_uv};
  CUtensorMap* tw[2] = {&tm_uk, &tm_uv};
  for (int i = 0; i < 2; ++i) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(kDc), 128, static_cast<cuuint64_t>(kHeads)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(kDc) * 2, static_cast<cuuint64_t>(128) * kDc * 2};
    cuuint32_t box[3] = {kKBlock, 128, 1};
    cuuint32_t es[3] = {1, 1, 1};
    if (encode(tw[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(w[i]), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = allow_smem(expand_kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  const int items = (rows + 127) / 128 * kHeads;
  return launch_kernel(expand_kernel, dim3(items < sms ? items : sms), dim3(kThreads), kSmem, stream, tm_c, tm_uk,
                       tm_uv, rows, items, static_cast<__nv_bfloat16*>(k_nope), static_cast<__nv_bfloat16*>(v),
                       static_cast<PlanHeader*>(hdr));
}

}  // namespace mla
