// Backward pass of the expanded-form (prefill) attention: parameters, workspace
// and launcher.
#pragma once
#include "prefill.cuh"

namespace mla {

constexpr int kBackwardTile = 128;   // columns of a step's tile of scores, and rows of a CTA's

struct BackwardParams {
  const __nv_bfloat16 *d_out, *q_nope, *q_rope, *k_nope, *k_rope, *v, *out;
  const float *d_lse, *lse;     // d_lse may be null
  long long do_t, do_h, qn_t, qn_h, qr_t, qr_h, kn_t, kn_h, kr_t, v_t, v_h;
  const int32_t *cu_q, *cu_k;
  int batch, nq, nk, causal;
  float scale;
  __nv_bfloat16 *dq_nope, *dq_rope, *dk_nope, *dk_rope, *dv;
  long long dqn_t, dqn_h, dqr_t, dqr_h, dkn_t, dkn_h, dkr_t, dv_t, dv_h;
  uint8_t* ws;
  int key_waits;   // the key pass follows a kernel of this call that it has to wait for (begin_pass)
};

// Behind the plan header.
struct BackwardPlan {
  int tiles[2], next[2], tail[2];   // [0] key tiles, [1] query tiles
  int stored, query_rows;           // dq comes from stored dS tiles; rows of a query tile
  int odd[2];                       // where causal, the pass may have results that are not finite
};

// Workspace: header and plan; the first query tile of each sequence; the key tiles
// and the query tiles; per query tile and head 128 values lse log2(e) and 128 values
// of sum(d_out out) - d_lse; the key-RoPE gradients of `group` heads each, fp32; the
// place of each key tile's first dS tile, and the dS tiles of all heads.
constexpr size_t kDsTile = 2 * kBackwardTile * kBackwardTile;   // bytes
constexpr long long kMaxDsTiles = 1024;                         // 4 GiB with all heads
constexpr size_t kTileBytes = 48;
constexpr int kCtas = 152;            // CTAs of the passes, one an SM; sizes do not depend on the device that is current
// Every part grows with each of the three counts, and so does the total.
struct BackwardWs {
  size_t plan, base[2], tiles[2], stats, rope, slots, ds, total;
  int max_tiles[2], group, ds_tiles;
  bool ds_always;   // there is room for all tiles, whatever the sequences' lengths
};
inline BackwardWs backward_ws(int batch, int nq, int nk) {
  BackwardWs w;
  // every sequence ends at most one tile early
  w.max_tiles[0] = nk / kBackwardTile + (batch < nk ? batch : nk);
  w.max_tiles[1] = nq / kBackwardTile + (batch < nq ? batch : nq);
  // eight heads where they still make eight items a CTA (a sixteenth of the keys' whole
  // gradients in the workspace instead of a quarter), two where they do not: one made
  // 8 x up to 1024 tokens 669 us instead of 646, four 654; 4096 tokens take the same
  // with one, two or eight
  constexpr int kEightFrom = 8 * kCtas / (kHeads / 8);   // key tiles
  w.group = w.max_tiles[0] >= kEightFrom ? 8 : 2;
  w.plan = align256(sizeof(PlanHeader));
  w.base[0] = align256(w.plan + sizeof(BackwardPlan));
  w.base[1] = align256(w.base[0] + sizeof(int) * static_cast<size_t>(batch));
  w.tiles[0] = align256(w.base[1] + sizeof(int) * static_cast<size_t>(batch));
  w.tiles[1] = align256(w.tiles[0] + kTileBytes * static_cast<size_t>(w.max_tiles[0]));
  w.stats = align256(w.tiles[1] + kTileBytes * static_cast<size_t>(w.max_tiles[1]));
  w.rope = align256(w.stats + sizeof(float) * 2 * kBackwardTile * kHeads * static_cast<size_t>(w.max_tiles[1]));
  // a call of fewer keys may take two heads, four times the sums a key: there is room for
  // those too, so that a workspace for a larger call serves every smaller one
  const size_t row = sizeof(float) * kDr, own = row * (kHeads / w.group) * static_cast<size_t>(nk),
               fewer = row * (kHeads / 2) * static_cast<size_t>(nk < kEightFrom * kBackwardTile ? nk : kEightFrom * kBackwardTile);
  w.slots = align256(w.rope + (own > fewer ? own : fewer));
  w.ds = align256(w.slots + sizeof(int) * static_cast<size_t>(w.max_tiles[0]));
  // Tiles of scores: sum over the sequences of ceil(q / 128) ceil(k / 128).  A sequence has
  // no more along one axis than all tokens would have together; and its tiles are at most
  // (q + 127) (k + 127) / 128^2, where the products q k sum to at most nq nk.
  constexpr long long kT = kBackwardTile;
  const long long q = nq, k = nk, some = batch < nq ? (batch < nk ? batch : nk) : (nq < nk ? nq : nk),   // sequences with both
                  by_q = (q + kT - 1) / kT * w.max_tiles[0], by_k = (k + kT - 1) / kT * w.max_tiles[1],
                  by_area = (q * k + (kT - 1) * (q + k) + (kT - 1) * (kT - 1) * some) / (kT * kT),
                  by_axis = by_q < by_k ? by_q : by_k, most = by_axis < by_area ? by_axis : by_area;
  w.ds_always = most <= kMaxDsTiles;
  w.ds_tiles = static_cast<int>(w.ds_always ? most : kMaxDsTiles);
  w.total = align256(w.ds + kDsTile * kHeads * static_cast<size_t>(w.ds_tiles));
  return w;
}

// The query pass on CTA pairs, whose row tiles are 256.
struct PassMaps;
cudaError_t launch_backward_pairs(const PassMaps& maps, const BackwardParams& p, const BackwardWs& L, int pairs,
                                  cudaStream_t stream);
// dq from stored dS tiles.
cudaError_t launch_backward_dq(PFN_cuTensorMapEncodeTiled_v12000 encode, const BackwardParams& p, const BackwardWs& L, int ctas,
                               cudaStream_t stream);
// The sums of the RoPE part of dk, and what values outside the mask would spoil.
cudaError_t launch_backward_last(const BackwardParams& p, const BackwardWs& L, cudaStream_t stream);
cudaError_t launch_backward(PFN_cuTensorMapEncodeTiled_v12000 encode, BackwardParams p, int sms, cudaStream_t stream);

}  // namespace mla
