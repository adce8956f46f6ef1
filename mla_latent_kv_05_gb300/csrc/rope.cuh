// Rotary positions: the angle arithmetic that the rotation kernel and the
// rotating cache append share, and the rotation's launcher.
//
// Pair i of a 64-value vector at position p is turned by the angle p f_i.  The
// table holds f_i / (2 pi) as a 64-bit fraction of a turn, so p times it,
// modulo 2^64, is the angle's fraction of a turn with no rounding at all: far
// positions lose nothing (in fp32 an angle of 10^5 radians is known to 2^-8).
// The error is the table's own, |p| 2^-65 turns (|p| 2^-62.3 rad).
//
// Sine and cosine come from the addition theorems: the fraction is split into
// the nearest 64th of a turn, whose values a table holds, and a rest d of at
// most a 128th (0.049 rad), whose sine and cosine are the first terms of their
// Taylor series.  Everything that matters is kept as an unevaluated sum of two
// floats (products and sums by the error-free transformations of Dekker and
// Knuth, with fma), so that a rotated value is known to 2^-37 of its pair (the cube of
// d, up to 2e-5, is a product of fp32 roundings) besides the angle's error, and can be rounded to a cache's codes as the exact value would be; one in fp32
// lands on the other side of a border for about one value in 2^19.  The rotation on
// its own (rope.cu) takes the high parts and multiplies in fp32.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace mla {

constexpr int kRopePairs = kDr / 2;

// An unevaluated sum of two floats.
struct Two {
  float hi, lo;
};

// cos(2 pi j / 64), j = 0..16.
__device__ const float2 kCosine64[17] = {
    {1.f, 0.f},
    {0.99518472f, 7.10966619e-09f},
    {0.980785251f, 2.97394731e-08f},
    {0.956940353f, -1.7184508e-08f},
    {0.923879504f, 2.83074897e-08f},
    {0.881921291f, -2.70029634e-08f},
    {0.831469595f, 1.68702634e-08f},
    {0.773010433f, 2.06425526e-08f},
    {0.707106769f, 1.21016175e-08f},
    {0.634393275f, 9.37955758e-09f},
    {0.555570245f, -1.17695214e-08f},
    {0.471396744f, -7.42525375e-09f},
    {0.382683426f, 6.22335072e-09f},
    {0.290284663f, 1.38156651e-08f},
    {0.195090324f, -1.67047143e-09f},
    {0.0980171412f, -8.93393193e-10f},
    {0.f, 0.f}};

// Entry j of the table of 64 (cos hi, cos lo, sin hi, sin lo), from the first quadrant.
__device__ __forceinline__ float4 turn_entry(int j) {
  const float2 a = kCosine64[j & 15], b = kCosine64[16 - (j & 15)];
  switch (j >> 4) {
    case 0: return make_float4(a.x, a.y, b.x, b.y);
    case 1: return make_float4(-b.x, -b.y, a.x, a.y);
    case 2: return make_float4(-a.x, -a.y, -b.x, -b.y);
    default: return make_float4(b.x, b.y, -a.x, -a.y);
  }
}

// x + y with |x| >= |y| or x = 0, and any two floats.
__device__ __forceinline__ Two quick_sum(float x, float y) {
  const float s = __fadd_rn(x, y);
  return {s, __fsub_rn(y, __fsub_rn(s, x))};
}
__device__ __forceinline__ Two any_sum(float x, float y) {
  const float s = __fadd_rn(x, y), b = __fsub_rn(s, x);
  return {s, __fadd_rn(__fsub_rn(x, __fsub_rn(s, b)), __fsub_rn(y, b))};
}
__device__ __forceinline__ Two product(float x, float y) {
  const float p = __fmul_rn(x, y);
  return {p, __fmaf_rn(x, y, -p)};
}
__device__ __forceinline__ Two product(Two x, Two y) {
  const Two p = product(x.hi, y.hi);
  return {p.hi, __fmaf_rn(x.hi, y.lo, __fmaf_rn(x.lo, y.hi, p.lo))};
}

// Cosine and sine of the angle t / 2^64 turns; `table` has the 64 entries.
__device__ __forceinline__ void turn_cos_sin(uint64_t t, const float4* table, Two& c, Two& s) {
  const uint32_t j = static_cast<uint32_t>((t + (uint64_t{1} << 57)) >> 58);   // 64 stands for 0
  const int64_t d = static_cast<int64_t>(t - (static_cast<uint64_t>(j) << 58));
  // d 2 pi / 2^64 in two exact parts of 24 bits
  const float d1 = static_cast<float>(static_cast<int>(d >> 34));
  const float d2 = static_cast<float>(static_cast<int>(d >> 10) & 0xFFFFFF);
  constexpr float kHi = 6.28318548f, kLo = -1.74845553e-07f;   // 2 pi
  const Two a = product(d1, kHi * 0x1p-30f);
  const Two x = quick_sum(a.hi, __fmaf_rn(d2, kHi * 0x1p-54f, __fmaf_rn(d1, kLo * 0x1p-30f, a.lo)));
  const Two q = product(x, x);
  // sin x - x and cos x - 1
  const float cube = __fmul_rn(__fmul_rn(x.hi, q.hi),
                               __fmaf_rn(q.hi, __fmaf_rn(q.hi, -1.f / 5040.f, 1.f / 120.f), -1.f / 6.f));
  const Two sine = quick_sum(x.hi, __fadd_rn(x.lo, cube));
  const Two less = {-0.5f * q.hi, __fmaf_rn(__fmul_rn(q.hi, q.hi), __fmaf_rn(q.hi, -1.f / 720.f, 1.f / 24.f), -0.5f * q.lo)};
  const float4 e = table[j & 63u];
  const Two C = {e.x, e.y}, S = {e.z, e.w};
  // cos = C + (C less - S sine), sin = S + (S less + C sine)
  const Two c1 = product(C, less), c2 = product(S, sine), s1 = product(S, less), s2 = product(C, sine);
  const Two ca = any_sum(c1.hi, -c2.hi), sa = any_sum(s1.hi, s2.hi);
  const Two cb = any_sum(C.hi, ca.hi), sb = any_sum(S.hi, sa.hi);
  c = quick_sum(cb.hi, __fadd_rn(cb.lo, __fadd_rn(__fadd_rn(ca.lo, C.lo), __fsub_rn(c1.lo, c2.lo))));
  s = quick_sum(sb.hi, __fadd_rn(sb.lo, __fadd_rn(__fadd_rn(sa.lo, S.lo), __fadd_rn(s1.lo, s2.lo))));
}

// x a + y b as a float that rounds to every shorter format as the exact sum does
// ("round to odd": where digits are lost, the last bit kept is 1).  x and y are
// bf16 values.
__device__ __forceinline__ float odd_sum(float x, Two a, float y, Two b) {
  const Two p = product(x, a.hi), q = product(y, b.hi);
  const Two h = any_sum(p.hi, q.hi);
  const float rest = __fadd_rn(h.lo, __fadd_rn(__fmaf_rn(x, a.lo, p.lo), __fmaf_rn(y, b.lo, q.lo)));
  const Two r = any_sum(h.hi, rest);
  const uint32_t bits = __float_as_uint(r.hi);
  // (a NaN rest, of an infinite x or y, compares false)
  if (!(fabsf(r.lo) > 0.f) || (bits & 1u)) return isfinite(rest) ? r.hi : h.hi;
  return __uint_as_float((r.lo > 0.f) == (r.hi > 0.f) ? bits + 1u : bits - 1u);
}

struct RopeParams {
  const __nv_bfloat16* x;     // [rows, heads, 64], strides in values
  long long x_t, x_h, out_t, out_h;
  const int32_t* positions;   // [rows]
  int rows, heads, inverse;
  __nv_bfloat16* out;
  mla_rope rope;
};

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream);

}  // namespace mla
