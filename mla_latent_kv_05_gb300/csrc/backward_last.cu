// The last kernel of the backward pass (backward.cu): the RoPE part of dk, summed over
// the groups of heads, and what values outside the mask would spoil.
//
// A pair outside the causal mask has P = dS = 0 in its tile, which an infinity or a NaN
// in its streamed row (the key's K for dq, the query's Q and d_out for dk and dv) turns
// into NaN.  Looking for such values in every tile at the mask's edge would cost every
// call.  A query's show in its lse or its delta, which are formed anyway, and a key's in
// results of the query pass, 24 multiply-adds a thread and item.  (The same in the key
// pass, 48, cost 2 x 512 queries over 8,012 keys another 9 us.)
//
// Where a query's has been noted, the key pass takes such values of its tiles at the edge
// as 0 in the sums.  For dk that is all: a query whose Q is not finite has a NaN for p and
// ds of every key that it sees (its lse is NaN, or it is -inf as every score of it).  For
// dv the terms p d_out of seen pairs of those tiles are missing, each an infinity or a
// NaN; this kernel adds them to the results, over the at most 255 columns of these tiles.
// (With every sum that was not finite computed again over all its columns, a column of
// d_out that is +inf in all of 4096 rows took 420 ms a call instead of 11.)
//
// Where a key's has been noted, it looks for results of dq that are not finite.  Where a
// hidden column of their edge tiles is not either, their rows are computed again on the
// CUDA cores, over the pairs that are seen alone; a value that is NaN by rights is so
// again, and once all that matter are, the row is left.
//
// Bound: without such rows the reading of the groups' fp32 sums, 64 (or 16) times 256
// bytes a key, which the key pass has left in L2.  (The second half's code must not cost
// the first its occupancy: with 112 registers a thread 2 x 512 queries over 8,012 keys
// took 1,738 us, with 40, and spills in the second half alone, 1,677.)
#include "backward_tile.cuh"

namespace mla {

namespace {

using namespace bwd;

constexpr int kUnits = 64;   // CTAs a tile

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float bf16_value(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// A lane's share of a row of a head: values 4 lane .. of 128, and 2 lane .. of 64.
__device__ __forceinline__ void load4(const __nv_bfloat16* row, int lane, float* x) {
  const uint2 w = *reinterpret_cast<const uint2*>(row + 4 * lane);
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load2(const __nv_bfloat16* row, int lane, float* x) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(row + 2 * lane);
  x[0] = __uint_as_float(w << 16);
  x[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void save4(__nv_bfloat16* row, int lane, const float* x) {
  *reinterpret_cast<uint2*>(row + 4 * lane) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
}
// A bit for each of a lane's values that is not finite.
template <int kN>
__device__ __forceinline__ uint32_t odd_values(const float* x) {
  uint32_t odd = 0;
#pragma unroll
  for (int e = 0; e < kN; ++e) odd |= isfinite(x[e]) ? 0u : 1u << e;
  return odd;
}
// The values of the bits from the first, times mul, into those of the second.
template <int kN>
__device__ __forceinline__ void replace(uint32_t bits, const float* from, float mul, float* to) {
#pragma unroll
  for (int e = 0; e < kN; ++e)
    if (bits >> e & 1u) to[e] = from[e] * mul;
}

// A lane's share of a query's and of a key's 192 values.
__device__ __forceinline__ void load_q(const BackwardParams& p, size_t i, int head, int lane, float* x) {
  load4(p.q_nope + i * p.qn_t + head * p.qn_h, lane, x);
  load2(p.q_rope + i * p.qr_t + head * p.qr_h, lane, x + 4);
}
__device__ __forceinline__ void load_k(const BackwardParams& p, size_t j, int head, int lane, float* x) {
  load4(p.k_nope + j * p.kn_t + head * p.kn_h, lane, x);
  load2(p.k_rope + j * p.kr_t, lane, x + 4);
}
// lse log2(e) of a sequence's query i, and kTile values on its delta.
__device__ __forceinline__ const float* stats_of(const BackwardParams& p, const BackwardWs& L, const Tile& t, int i, int head) {
  return reinterpret_cast<const float*>(p.ws + L.stats) + (static_cast<size_t>(t.stat + i / kTile) * kHeads + head) * 2 * kTile + i % kTile;
}
__device__ __forceinline__ float probability(const BackwardParams& p, const float* a, const float* x, float lse) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 6; ++e) s += a[e] * x[e];
  return fast_exp2(warp_sum(s) * (p.scale * kLog2e) - lse);
}

// dq of a row of a head before scaling once more, over its seen columns, one warp.  need:
// the values that matter; when all of them are NaN, the rest of the row cannot change that.
__device__ void row_again(const BackwardParams& p, const BackwardWs& L, const Tile& t, int r, int head, int lane, uint32_t need, float* dq) {
  const size_t row = static_cast<size_t>(t.r0) + r;
  const float* st = stats_of(p, L, t, r, head);
  const float lse = __ldcg(st), delta = __ldcg(st + kTile);
  float a[6], b[4], x[6], y[4];
#pragma unroll
  for (int e = 0; e < 6; ++e) dq[e] = 0.f;
  load_q(p, row, head, lane, a);
  load4(p.d_out + row * p.do_t + head * p.do_h, lane, b);
  const int to = min(t.nc, t.lim + r);
  for (int i = 0; i < to; ++i) {
    const size_t col = static_cast<size_t>(t.c0) + i;
    load_k(p, col, head, lane, x);
    load4(p.v + col * p.v_t + head * p.v_h, lane, y);
    float dp = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) dp += b[e] * y[e];
    const float ds = bf16_value(probability(p, a, x, lse) * (warp_sum(dp) - delta));
    bool open = false;
#pragma unroll
    for (int e = 0; e < 6; ++e) {
      dq[e] += ds * x[e];
      open |= (need >> e & 1u) && !isnan(dq[e]);
    }
    if (!__any_sync(0xffffffffu, open)) break;
  }
}

// Whether a key that the row does not see, in a tile that the pass has computed, has a
// value that is not finite; without one the row's results are what the formula gives.
__device__ bool hidden_odd(const BackwardParams& p, const Tile& t, int r, int head, int lane) {
  const int from = max(0, t.lim + r), to = min(t.nc, t.steps * kTile);
  uint32_t odd = 0;
  for (int i = from; i < to; ++i) {
    float x[6];
    load_k(p, static_cast<size_t>(t.c0) + i, head, lane, x);
    odd |= odd_values<6>(x);
  }
  return __any_sync(0xffffffffu, odd != 0);
}

// The rows [r, end) of a query tile whose dq is not finite, one warp a row and head.
__device__ __noinline__ void queries_again(const BackwardParams& p, const BackwardWs& L, const Tile t, int r, int end) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (; r < end; ++r)
    for (int head = warp; head < kHeads; head += 8) {
      const size_t row = static_cast<size_t>(t.r0) + r;
      __nv_bfloat16 *dn = p.dq_nope + row * p.dqn_t + head * p.dqn_h, *dr = p.dq_rope + row * p.dqr_t + head * p.dqr_h;
      float x[6], again[6];
      load4(dn, lane, x);
      load2(dr, lane, x + 4);
      const uint32_t need = odd_values<6>(x);
      if (!__any_sync(0xffffffffu, need != 0) || !hidden_odd(p, t, r, head, lane)) continue;
      row_again(p, L, t, r, head, lane, need, again);
      replace<6>(need, again, p.scale, x);
      save4(dn, lane, x);
      *reinterpret_cast<uint32_t*>(dr + 2 * lane) = bf16_pair(x[4], x[5]);
    }
}

// dv of the keys [r, end) of a tile: the terms of seen pairs whose d_out the key pass has
// taken as 0, one warp a row and head.  Such a query's delta is not finite.
__device__ __noinline__ void keys_again(const BackwardParams& p, const BackwardWs& L, const Tile t, int r, int end) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int to = min(t.nc, (max(0, mask_end(t)) + kTile - 1) / kTile * kTile);   // the last tile with hidden pairs
  for (; r < end; ++r)
    for (int head = warp; head < kHeads; head += 8) {
      const size_t row = static_cast<size_t>(t.r0) + r;
      __nv_bfloat16* dv = p.dv + row * p.dv_t + head * p.dv_h;
      float a[6], sum[4];
      bool some = false;
      for (int i0 = max(0, t.lim + r); i0 < to; i0 += 32) {
        const int mine = i0 + lane;
        uint32_t columns = __ballot_sync(0xffffffffu, mine < to && !isfinite(__ldcg(stats_of(p, L, t, mine, head) + kTile)));
        for (; columns != 0; columns &= columns - 1) {
          const int i = i0 + __ffs(static_cast<int>(columns)) - 1;
          const size_t col = static_cast<size_t>(t.c0) + i;
          float x[6], y[4];
          load4(p.d_out + col * p.do_t + head * p.do_h, lane, y);
          const uint32_t odd = odd_values<4>(y);
          if (!__any_sync(0xffffffffu, odd != 0)) continue;
          if (!some) {
            load_k(p, row, head, lane, a);
            load4(dv, lane, sum);
            some = true;
          }
          load_q(p, col, head, lane, x);
          const float pr = bf16_value(probability(p, a, x, __ldcg(stats_of(p, L, t, i, head))));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (odd >> e & 1u) sum[e] += pr * y[e];
        }
      }
      if (some) save4(dv, lane, sum);
    }
}

// CTAs [0, kUnits key_tiles): two keys of a tile, whose sums 16 threads a key and run of
// groups with four values each form, then over the eight runs, in their order.  Those
// behind them, where causal: a 64th of a query tile.
__global__ void __launch_bounds__(256, 6) backward_last_kernel(const __grid_constant__ BackwardParams p, const __grid_constant__ BackwardWs L, int key_tiles) {
  __shared__ float4 s_sum[2][8][16];
  const BackwardPlan* plan = reinterpret_cast<const BackwardPlan*>(p.ws + L.plan);
  const int i_tile = static_cast<int>(blockIdx.x) / kUnits, unit = static_cast<int>(blockIdx.x) % kUnits;
  ptx::grid_dep_wait();
  if (i_tile >= key_tiles) {
    if (plan->odd[1] == 0 || i_tile - key_tiles >= plan->tiles[1]) return;
    const Tile t = read_tile(reinterpret_cast<const Tile*>(p.ws + L.tiles[1]) + (i_tile - key_tiles));
    const int per = plan->query_rows / kUnits;
    queries_again(p, L, t, per * unit, min(per * unit + per, t.rows));
    return;
  }
  if (i_tile >= plan->tiles[0]) return;
  const Tile t = read_tile(reinterpret_cast<const Tile*>(p.ws + L.tiles[0]) + i_tile);
  const int k = threadIdx.x >> 7, run = (threadIdx.x >> 4) & 7, lane = threadIdx.x & 15, r = 2 * unit + k;
  if (2 * unit >= t.rows) return;
  if (plan->odd[0] != 0) keys_again(p, L, t, 2 * unit, min(2 * unit + 2, t.rows));
  const size_t row = static_cast<size_t>(t.r0) + r;
  const int per = kHeads / L.group / 8;   // 2 or 8 groups a run
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < t.rows) {
    const float4* part = reinterpret_cast<const float4*>(p.ws + L.rope) + (static_cast<size_t>(run * per) * p.nk + row) * (kDr / 4) + lane;
#pragma unroll 8
    for (int g = 0; g < per; ++g) {
      const float4 x = __ldcs(part + static_cast<size_t>(g) * p.nk * (kDr / 4));
      sum.x += x.x;
      sum.y += x.y;
      sum.z += x.z;
      sum.w += x.w;
    }
  }
  s_sum[k][run][lane] = sum;
  __syncthreads();
  if (run != 0 || r >= t.rows) return;
#pragma unroll
  for (int q = 1; q < 8; ++q) {
    const float4 x = s_sum[k][q][lane];
    sum.x += x.x;
    sum.y += x.y;
    sum.z += x.z;
    sum.w += x.w;
  }
  *reinterpret_cast<uint2*>(p.dk_rope + row * p.dkr_t + 4 * lane) =
      make_uint2(bf16_pair(sum.x * p.scale, sum.y * p.scale), bf16_pair(sum.z * p.scale, sum.w * p.scale));
}

}  // namespace

cudaError_t launch_backward_last(const BackwardParams& p, const BackwardWs& L, cudaStream_t stream) {
  // (no more query tiles of 256 rows than of 128)
  const unsigned tiles = static_cast<unsigned>(L.max_tiles[0] + (p.causal ? L.max_tiles[1] : 0));
  return launch_dependent(backward_last_kernel, dim3(tiles * kUnits), dim3(256), 0, stream, p, L, L.max_tiles[0]);
}

}  // namespace mla
