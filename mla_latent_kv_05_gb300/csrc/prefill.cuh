// Expanded-form (prefill) attention: parameters, workspace and launcher.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace mla {

constexpr int kPrefillTile = 256;   // query rows of a work tile (two 128-row tiles)

struct PrefillParams {
  const __nv_bfloat16 *q_nope, *q_rope, *k_nope, *k_rope, *v;
  // strides in values: of a token, and of a head
  long long qn_t, qn_h, qr_t, qr_h, kn_t, kn_h, kr_t, v_t, v_h;
  const int32_t *cu_q, *cu_k;   // [batch + 1]
  int batch, nq, nk, causal;
  float scale_log2;             // softmax scale * log2(e)
  __nv_bfloat16* out;           // [nq, 128, 128]
  float* lse;                   // [nq, 128]
  uint8_t* ws;
};

// Workspace: the plan header, then the tile list, then 128 bits a tile: the heads
// whose results the second pass computes again.
struct PrefillWs {
  size_t tiles, again, total;
  int max_tiles;
};
__host__ __device__ inline PrefillWs prefill_ws(int batch, int nq) {
  PrefillWs w;
  w.max_tiles = nq / kPrefillTile + (batch < nq ? batch : nq);   // every sequence ends at most one tile early
  w.tiles = align256(sizeof(PlanHeader));
  w.again = align256(w.tiles + 32 * static_cast<size_t>(w.max_tiles));
  w.total = align256(w.again + 16 * static_cast<size_t>(w.max_tiles));
  return w;
}

cudaError_t launch_prefill(PFN_cuTensorMapEncodeTiled_v12000 encode, const PrefillParams& p, int sms,
                           cudaStream_t stream);

}  // namespace mla
