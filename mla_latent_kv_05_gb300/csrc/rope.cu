// Rotary positions of packed vectors: y = scale R(position) x for the 64 values
// of each row and head, where R turns pair i by position f_i.  A pair is (2i, 2i+1)
// (interleaved) or (i, i + 32) (halves).  inverse: the angles negated, which is
// the transposed map and so the gradient.
//
// Bound: 256 bytes a vector read and written against 6 operations a pair, so HBM
// bounds long calls of many heads (8192 rows of 128 heads 42 us, 6,400 GB/s).  A row's
// 32 cosines and sines (about 70 operations each) are computed once by a CTA for all the
// heads it takes, while its loads are in flight; with one head a row they bound the call
// (262,144 keys 67 us, 1,010 GB/s; 16,384 7.1).  A thread takes two 16-byte pieces of a vector, 64 bytes apart: with
// both layouts the pieces hold whole pairs, so a vector may be rotated in place.
// A CTA takes 64 vectors a step (64 heads of a row, or fewer heads of more rows)
// and kSteps steps, whose loads are all issued before the first result is needed.
#include "rope.cuh"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / 4;   // vectors a step

// Two bf16 values as floats, and rounded back.
__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// `by` heads of a row a step (a power of two, at most kUnits).
template <bool kInterleaved, int kSteps>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p, int by) {
  __shared__ float4 s_table[64];
  __shared__ float2 s_turn[kUnits][kRopePairs];   // rows of this CTA: (cos, sin) times the scale
  const int t = threadIdx.x, unit = t >> 2, q = t & 3;
  const int rows_step = kUnits / by, rows_cta = rows_step * kSteps;   // at most kUnits rows (see launch)
  const int row0 = blockIdx.x * rows_cta, head = blockIdx.y * by + unit % by;
  uint4 v[kSteps][2];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int row = row0 + k * rows_step + unit / by;
    v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
    if (row < p.rows && head < p.heads) {
      const __nv_bfloat16* src = p.x + row * p.x_t + head * p.x_h + 8 * q;
      v[k][0] = *reinterpret_cast<const uint4*>(src);
      v[k][1] = *reinterpret_cast<const uint4*>(src + 32);
    }
  }
  if (t < 64) s_table[t] = turn_entry(t);
  __syncthreads();
  for (int i = t; i < rows_cta * kRopePairs; i += kThreads) {
    const int r = i / kRopePairs, pair = i % kRopePairs;
    if (row0 + r >= p.rows) break;
    const int64_t at = __ldg(p.positions + row0 + r);
    Two c, s;
    turn_cos_sin(static_cast<uint64_t>(at) * p.rope.turns[pair], s_table, c, s);
    s_turn[r][pair] = make_float2(c.hi * p.rope.scale, (p.inverse ? -s.hi : s.hi) * p.rope.scale);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int r = k * rows_step + unit / by, row = row0 + r;
    if (row >= p.rows || head >= p.heads) continue;
    const uint32_t a[4] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w};
    const uint32_t b[4] = {v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
    uint32_t ya[4], yb[4];
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 ta = s_turn[r][4 * q + i], tb = s_turn[r][16 + 4 * q + i];
        const float2 xa = unpack(a[i]), xb = unpack(b[i]);
        ya[i] = pack(xa.x * ta.x - xa.y * ta.y, xa.x * ta.y + xa.y * ta.x);
        yb[i] = pack(xb.x * tb.x - xb.y * tb.y, xb.x * tb.y + xb.y * tb.x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t0 = s_turn[r][8 * q + 2 * i], t1 = s_turn[r][8 * q + 2 * i + 1];
        const float2 xa = unpack(a[i]), xb = unpack(b[i]);
        ya[i] = pack(xa.x * t0.x - xb.x * t0.y, xa.y * t1.x - xb.y * t1.y);
        yb[i] = pack(xa.x * t0.y + xb.x * t0.x, xa.y * t1.y + xb.y * t1.x);
      }
    }
    __nv_bfloat16* dst = p.out + row * p.out_t + head * p.out_h + 8 * q;
    *reinterpret_cast<uint4*>(dst) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
    *reinterpret_cast<uint4*>(dst + 32) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
  }
}

template <int kSteps>
cudaError_t launch(const RopeParams& p, int by, cudaStream_t stream) {
  const int rows = kUnits / by * kSteps;
  const dim3 grid((p.rows + rows - 1) / rows, (p.heads + by - 1) / by);
  return p.rope.interleaved ? launch_kernel(rope_kernel<true, kSteps>, grid, dim3(kThreads), 0, stream, p, by)
                            : launch_kernel(rope_kernel<false, kSteps>, grid, dim3(kThreads), 0, stream, p, by);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  if (p.rows <= 0 || p.heads <= 0) return cudaSuccess;
  int by = 1;
  while (by < kUnits && by < p.heads) by *= 2;
  // four steps where they still make two CTAs an SM, and the rows fit the table
  const bool many = 4 * (kUnits / by) <= kUnits && static_cast<long long>(p.rows) * p.heads >= 4ll * kUnits * 2 * 152;
  return many ? launch<4>(p, by, stream) : launch<1>(p, by, stream);
}

}  // namespace mla
