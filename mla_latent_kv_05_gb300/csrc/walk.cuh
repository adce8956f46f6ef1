// The planner's page ranges as row segments, and the visibility of drafted
// tokens: shared by the attention kernels that run the split-KV plan.
#pragma once
#include "common.cuh"

namespace mla {
namespace dk {

struct Segment {
  int b;          // batch row
  int t0, t1;     // row-local page range [t0, t1)
};

// Walks the segments of one pair: the pair's page range [lo, hi) cut at row
// boundaries.  Every role of both ranks walks the same sequence; inside a
// segment the half pages [2*t0, 2*t1) are taken kTileHalves at a time.
struct SegWalker {
  const int* tile_start;
  int batch, b, lo, hi;
  // b0: the row holding page lo (the planner's pair_b0)
  __device__ void init(const int* ts, int nb, int lo_, int hi_, int b0) {
    tile_start = ts; batch = nb; lo = lo_; hi = hi_;
    b = lo >= hi ? nb : b0;
  }
  __device__ bool next(Segment& s) {
    while (b < batch) {
      const int a = __ldg(tile_start + b), e = __ldg(tile_start + b + 1);
      if (a >= hi) { b = batch; return false; }
      const int cb = b++;
      if (e >= hi) b = batch;   // this segment reaches the end of the range: no read for the next call
      if (e > a) {
        s.b = cb;
        s.t0 = max(lo, a) - a;
        s.t1 = min(hi, e) - a;
        if (s.t1 > s.t0) return true;
      }
    }
    return false;
  }
};

// Tree decode: bits of the columns starting at some token that a node sees,
// `ctx` of them context (may be negative or large), `valid` of them at most;
// draft token a is column ctx + a and seen when bit a of `seen` is set.
__device__ __forceinline__ uint64_t tree_bits(uint64_t seen, int ctx, int valid) {
  uint64_t m;
  if (ctx >= 64) m = ~uint64_t{0};
  else if (ctx > 0) m = (seen << ctx) | ((uint64_t{1} << ctx) - 1);
  else m = ctx > -64 ? seen >> -ctx : 0;
  if (valid <= 0) return 0;
  return valid >= 64 ? m : m & ((uint64_t{1} << valid) - 1);
}

}  // namespace dk
}  // namespace mla
