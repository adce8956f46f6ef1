// Cache rows: write new tokens' latent rows into a paged cache (append) and
// read a sequence's rows back as bf16 (gather), in the five cache formats the
// decode reads.
//
// Packed rows: sequence b owns rows [cu[b], cu[b+1]) of the packed tensors,
// which are the LAST n_b = cu[b+1] - cu[b] of its seq_lens[b] tokens: packed
// row i is token seq_lens[b] - cu[b+1] + i.
//
// Quantisation (the inverse of the decode's dequantisation): a group of G
// values (G = 32 e4m3, 16 e2m1) with largest magnitude a takes the smallest
// k with a <= M 2^k (M = 448, 6; k = 0 for an all-zero group), stored as the
// e8m0 byte k + 127, and the codes round(v 2^-k) to nearest, ties to even.
// With a = m 2^E, m in [1/2, 1): 448 = 0.875 2^9, 6 = 0.75 2^3, so k is E - 9
// or E - 8 (E - 3 or E - 2), read from a's exponent and mantissa bits with no
// rounding.  k is kept in [-127, 119] ([-127, 125]): at the top the codes
// saturate instead of standing for values beyond bf16.  A group that holds
// an infinity or a NaN takes scale byte 255 (the NaN scale) and zero codes.
//
// Both directions only move bytes, so they are bound by HBM when long and by
// the launch and two dependent reads (the row's sequence, then its page) when
// short.  One thread takes eight consecutive values (16 bytes of bf16), so
// the bf16 side is one coalesced 16-byte access a thread and a group's
// maximum needs one or two shuffles.  A CTA takes kGroups groups of four rows:
// one group for short calls (more CTAs, and the values are on their way while
// a warp looks the slots up), four for long ones, whose loads are all in
// flight at once.
//
// Measured (bytes read and written a second; a copy reaches 6670 GB/s), 262,144
// rows: bf16 append 89 us (6810 GB/s) and gather 90, fp8 81 (5640) and 84, fp4
// 72 (5380) and 63 (6180), V4.1 rows 66, 64 (6150, 5410: they read 1024 of a row's
// 1152 bytes) and 68, 61 (6470, 6190); the 594- and 324-byte rows are off 16-byte
// boundaries, so their accesses are smaller.
// 16,384 rows: 5.2 to 7.2 us; 64 rows: 2.3 us.
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rows.cuh"

namespace mla {

namespace {

constexpr int kGroupRows = 4;
constexpr int kPiece = 8;   // values per thread

template <RowFormat F> struct Fmt;
template <> struct Fmt<RowFormat::kBf16> {
  static constexpr int kValues = kRow, kBytes = kRow * 2;
};
template <> struct Fmt<RowFormat::kFp8> {
  static constexpr int kValues = kRow, kBytes = kFp8Row, kGroup = 32, kScales = kRow, kTopK = 119;
};
template <> struct Fmt<RowFormat::kFp4> {
  static constexpr int kValues = kRow, kBytes = kFp4Row, kGroup = 16, kScales = kFp4Codes, kTopK = 125;
};
template <> struct Fmt<RowFormat::kFp8V41> {
  static constexpr int kValues = kV41Values, kBytes = kV41Row, kGroup = 32, kScales = kV41Values, kTopK = 119;
};
template <> struct Fmt<RowFormat::kFp4V41> {
  static constexpr int kValues = kV41Values, kBytes = kV41Fp4Row, kGroup = 16, kScales = kV41Values / 2, kTopK = 125;
};
template <RowFormat F> constexpr bool kIsFp4 = F == RowFormat::kFp4 || F == RowFormat::kFp4V41;
template <RowFormat F> constexpr bool kIsV41 = F == RowFormat::kFp8V41 || F == RowFormat::kFp4V41;

// Cache slots (page * 64 + offset) of this CTA's rows, by its first warp, a lane
// a row: -1 for a row past the last sequence (left alone), -2 for one whose
// token or page lies outside the cache (recorded in the status word; never read
// or written).  One search for all rows: a warp's search for each took more
// instructions than the rows' values (131,072 rows: fp8 append 56 us).
template <int kRows>
__device__ __forceinline__ void look_up(const RowsParams& p, int row0, int* s_slot) {
  static_assert(kRows <= 32, "a lane a row");
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    // a sequence b with cu[b] <= row0 and cu[b + 32] > row0 or b + 32 > batch, 32 probes a round
    int lo = 0, hi = p.batch;            // cu[lo] <= row0 is assumed, cu[hi + 1] is not probed
    while (hi - lo > 31) {
      const int step = (hi - lo + 31) / 32;
      const int probe = lo + (lane + 1) * step;
      const bool le = probe <= hi && __ldg(p.cu_rows + probe) <= row0;
      const int n = __popc(__ballot_sync(0xffffffffu, le));   // cu is non-decreasing: the probes that hold come first
      const int nlo = lo + n * step;
      hi = min(hi, nlo + step - 1);
      lo = min(nlo, hi);
    }
    // each row's sequence: the largest b with cu[b] <= row
    const int next = lo + 1 + lane <= p.batch ? __ldg(p.cu_rows + lo + 1 + lane) : INT_MAX;
    int b = lo;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int n = __popc(__ballot_sync(0xffffffffu, next <= row0 + r));
      if (lane == r) b = lo + n;
    }
    const int i = row0 + lane;
    if (lane < kRows) {
      // (32 sequences begin in these rows, most of them empty: look further)
      if (b == lo + 32)
        while (b < p.batch && __ldg(p.cu_rows + b + 1) <= i) ++b;
      int slot = -1;
      if (i < p.rows && b < p.batch) {   // (cu[batch] <= i: behind the last sequence)
        const int c0 = __ldg(p.cu_rows + b), c1 = __ldg(p.cu_rows + b + 1);
        int code = MLA_STATUS_BAD_SEQ_LEN;
        slot = -2;
        if (i >= c0 && i < c1) {
          const long long pos = static_cast<long long>(__ldg(p.seq_lens + b)) - c1 + i;
          if (pos >= 0 && pos < static_cast<long long>(p.max_pages) * kPage) {
            const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + (pos >> 6));
            if (page >= 0 && page < p.num_pages) slot = page * kPage + static_cast<int>(pos & 63);
            else code = MLA_STATUS_BAD_PAGE;
          }
        }
        if (slot < 0) set_status(p.status, code);
      }
      s_slot[lane] = slot;
    }
  }
  __syncthreads();
}

// Scale exponent of a group whose largest magnitude has the bf16 bits `a`
// (finite, sign cleared): see the top of the file.
template <RowFormat F>
__device__ __forceinline__ int scale_exponent(uint32_t a) {
  if (a == 0) return 0;
  const int e = static_cast<int>(a >> 7) - 126;     // a = m 2^e, m in [1/2, 1) (a subnormal lands below the clamp)
  const uint32_t man = a & 0x7Fu;
  const int k = kIsFp4<F> ? e - 3 + (man > 0x40u) : e - 9 + (man > 0x60u);
  return min(max(k, -127), Fmt<F>::kTopK);
}

// One piece of a quantised or bf16 row into its cache row.
template <RowFormat F>
__device__ __forceinline__ void append_piece(const RowsParams& p, uint4 v, int slot, int j) {
  using T = Fmt<F>;
  uint8_t* dst = p.cache + static_cast<size_t>(slot < 0 ? 0 : slot) * T::kBytes;
  if constexpr (F == RowFormat::kBf16) {
    if (slot >= 0) *reinterpret_cast<uint4*>(dst + j * 16) = v;
  } else {
    // largest magnitude of the group as bf16 bits (their order as integers
    // is the order of the magnitudes, infinities and NaNs at the top)
    const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
    for (int o = 1; o < T::kGroup / kPiece; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool finite = m < 0x7F80u;
    const int k = finite ? scale_exponent<F>(m) : 0;
    const float mul = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);   // 2^-k, normal: k <= 125
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // exact: a product that is not (below 2^-126) is far under the smallest code
      const float lo = finite ? __uint_as_float(w[i] << 16) * mul : 0.f;
      const float hi = finite ? __uint_as_float(w[i] & 0xFFFF0000u) * mul : 0.f;
      if constexpr (kIsFp4<F>) {
        asm("{\n .reg .b8 c;\n cvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n cvt.u32.u8 %0, c;\n}"
            : "=r"(code[i]) : "f"(lo), "f"(hi));
      } else {
        unsigned short c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(lo), "f"(hi));
        code[i] = c;
      }
    }
    if (slot < 0) return;
    if constexpr (kIsFp4<F>) {
      // rows start on 4-byte boundaries
      *reinterpret_cast<uint32_t*>(dst + j * 4) = code[0] | (code[1] << 8) | (code[2] << 16) | (code[3] << 24);
    } else if constexpr (F == RowFormat::kFp8V41) {
      *reinterpret_cast<uint2*>(dst + j * 8) = make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
    } else if (slot & 1) {
      // 594-byte rows: an odd slot starts between two words
      *reinterpret_cast<uint16_t*>(dst + j * 8) = static_cast<uint16_t>(code[0]);
      *reinterpret_cast<uint32_t*>(dst + j * 8 + 2) = code[1] | (code[2] << 16);
      *reinterpret_cast<uint16_t*>(dst + j * 8 + 6) = static_cast<uint16_t>(code[3]);
    } else {
      *reinterpret_cast<uint32_t*>(dst + j * 8) = code[0] | (code[1] << 16);
      *reinterpret_cast<uint32_t*>(dst + j * 8 + 4) = code[2] | (code[3] << 16);
    }
    if (j % (T::kGroup / kPiece) == 0)
      dst[T::kScales + j / (T::kGroup / kPiece)] = static_cast<uint8_t>(finite ? k + 127 : 255);
  }
}

template <RowFormat F, int kGroups>
__global__ void __launch_bounds__(kGroupRows * Fmt<F>::kValues / kPiece) append_kernel(const RowsParams p) {
  constexpr int kPieces = Fmt<F>::kValues / kPiece;
  __shared__ int s_slot[kGroups * kGroupRows];
  const int r = threadIdx.x / kPieces, j = threadIdx.x - r * kPieces;
  const int row0 = blockIdx.x * kGroups * kGroupRows;
  // V4.1 rows: values 0..447 are the latent's first 448, then the RoPE values
  constexpr int kLatentPieces = (kIsV41<F> ? kV41Latent : kDc) / kPiece;
  uint4 v[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int row = row0 + g * kGroupRows + r;
    v[g] = make_uint4(0, 0, 0, 0);
    if (row < p.rows)
      v[g] = __ldg(reinterpret_cast<const uint4*>(
          j < kLatentPieces ? p.c_kv + static_cast<size_t>(row) * p.c_stride + j * kPiece
                            : p.k_rope + static_cast<size_t>(row) * p.r_stride + (j - kLatentPieces) * kPiece));
  }
  look_up<kGroups * kGroupRows>(p, row0, s_slot);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) append_piece<F>(p, v[g], s_slot[g * kGroupRows + r], j);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A stored piece (codes and their scale) as read, and as eight bf16 values.
struct Piece {
  uint4 raw;
  uint32_t scale;
};

template <RowFormat F>
__device__ __forceinline__ Piece read_piece(const RowsParams& p, int slot, int j) {
  using T = Fmt<F>;
  Piece x;
  x.raw = make_uint4(0, 0, 0, 0);            // a row outside the cache reads as zeros
  x.scale = 127;
  // V4.1 rows: latent dims 448..511 are zero, the RoPE values are the row's last 64
  constexpr int kPad0 = kIsV41<F> ? kV41Latent / kPiece : kRow / kPiece, kPad1 = kDc / kPiece;
  if (slot < 0 || (j >= kPad0 && j < kPad1)) return x;
  const int q = kIsV41<F> && j >= kPad1 ? j - (kPad1 - kPad0) : j;         // piece of the stored row
  const uint8_t* src = p.cache + static_cast<size_t>(slot) * T::kBytes;
  if constexpr (F == RowFormat::kBf16) {
    x.raw = __ldg(reinterpret_cast<const uint4*>(src + q * 16));
  } else {
    x.scale = __ldg(src + T::kScales + q / (T::kGroup / kPiece));
    if constexpr (kIsFp4<F>) {
      x.raw.x = __ldg(reinterpret_cast<const uint32_t*>(src + q * 4));
    } else if constexpr (F == RowFormat::kFp8V41) {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(src + q * 8));
      x.raw.x = c.x;
      x.raw.y = c.y;
    } else if (slot & 1) {
      // 594-byte rows: an odd slot starts between two words
      const uint32_t a = __ldg(reinterpret_cast<const uint16_t*>(src + q * 8));
      const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(src + q * 8 + 2));
      const uint32_t c = __ldg(reinterpret_cast<const uint16_t*>(src + q * 8 + 6));
      x.raw.x = a | (b << 16);
      x.raw.y = (b >> 16) | (c << 16);
    } else {
      x.raw.x = __ldg(reinterpret_cast<const uint32_t*>(src + q * 8));
      x.raw.y = __ldg(reinterpret_cast<const uint32_t*>(src + q * 8 + 4));
    }
  }
  return x;
}

template <RowFormat F>
__device__ __forceinline__ uint4 values_of(const Piece& x) {
  if constexpr (F == RowFormat::kBf16) {
    return x.raw;
  } else {
    const uint32_t e = x.scale;
    const float sc = __uint_as_float(e == 0 ? 0x00400000u : (e == 255 ? 0x7FC00000u : e << 23));
    uint32_t h[4], w[4];
    if constexpr (kIsFp4<F>) {
      asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
          " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
          " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
          : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(x.raw.x));
    } else {
      const uint32_t c[2] = {x.raw.x, x.raw.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"(static_cast<unsigned short>(c[i >> 1] >> (16 * (i & 1)))));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      w[i] = bf16_pair(f.x * sc, f.y * sc);   // exact in fp32, rounded once
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <RowFormat F, int kGroups>
__global__ void __launch_bounds__(kGroupRows * kRow / kPiece) gather_kernel(const RowsParams p) {
  constexpr int kPieces = kRow / kPiece;     // the output row has 576 values in every format
  __shared__ int s_slot[kGroups * kGroupRows];
  const int r = threadIdx.x / kPieces, j = threadIdx.x - r * kPieces;
  const int row0 = blockIdx.x * kGroups * kGroupRows;
  look_up<kGroups * kGroupRows>(p, row0, s_slot);
  Piece x[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) x[g] = read_piece<F>(p, s_slot[g * kGroupRows + r], j);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (s_slot[g * kGroupRows + r] == -1) continue;   // behind the last sequence: left as it was
    const size_t row = static_cast<size_t>(row0) + g * kGroupRows + r;
    *reinterpret_cast<uint4*>(p.out + row * kRow + j * kPiece) = values_of<F>(x[g]);
  }
}

// The pages of a batch of sequences as bf16 rows: token t of sequence b becomes
// row b max_pages 64 + t.  blockIdx.y is the sequence, whose tokens the CTAs of
// a column take 16 at a time (the last 16 are filled up with zero rows).
template <RowFormat F>
__global__ void __launch_bounds__(kGroupRows * kRow / kPiece) widen_kernel(const RowsParams p) {
  constexpr int kPieces = kRow / kPiece, kRows = 4 * kGroupRows;
  const int r = threadIdx.x / kPieces, j = threadIdx.x - r * kPieces;
  const int b = blockIdx.y, len = min(__ldg(p.seq_lens + b), p.max_pages * kPage);
  for (int t = blockIdx.x * kRows + r; t - r < len; t += gridDim.x * kRows) {
    const size_t at = static_cast<size_t>(b) * p.max_pages;
    const int page = __ldg(p.block_table + at + (t - r) / kPage);
    const bool bad = page < 0 || page >= p.num_pages;
    if (bad && threadIdx.x == 0) set_status(p.status, MLA_STATUS_BAD_PAGE);
    Piece x[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int row = t + g * kGroupRows;
      x[g] = read_piece<F>(p, bad || row >= len ? -1 : page * kPage + row % kPage, j);
    }
    __nv_bfloat16* dst = p.out + (at * kPage + t) * kRow + j * kPiece;
#pragma unroll
    for (int g = 0; g < 4; ++g) *reinterpret_cast<uint4*>(dst + g * kGroupRows * kRow) = values_of<F>(x[g]);
  }
}

// Rows of a call from which a CTA takes four groups instead of one.
constexpr int kLongCall = 8192;

template <RowFormat F, int kGroups>
cudaError_t launch(const RowsParams& p, bool append, cudaStream_t stream) {
  const dim3 grid((p.rows + kGroups * kGroupRows - 1) / (kGroups * kGroupRows));
  if (append)
    return launch_kernel(append_kernel<F, kGroups>, grid, dim3(kGroupRows * Fmt<F>::kValues / kPiece), 0, stream, p);
  return launch_kernel(gather_kernel<F, kGroups>, grid, dim3(kGroupRows * kRow / kPiece), 0, stream, p);
}

template <RowFormat F>
cudaError_t launch(const RowsParams& p, bool append, cudaStream_t stream) {
  return p.rows >= kLongCall ? launch<F, 4>(p, append, stream) : launch<F, 1>(p, append, stream);
}

}  // namespace

cudaError_t launch_widen(RowFormat fmt, const RowsParams& p, cudaStream_t stream) {
  if (p.batch <= 0) return cudaSuccess;
  // about 1000 CTAs are resident; at least 32 columns for a batch of uneven lengths
  const int share = (2048 + p.batch - 1) / p.batch;
  const int columns = share < 32 ? 32 : share, most = p.max_pages * (kPage / (4 * kGroupRows));
  const dim3 grid(columns < most ? columns : most, p.batch), block(kGroupRows * kRow / kPiece);
  switch (fmt) {
    case RowFormat::kBf16: break;
    case RowFormat::kFp8: return launch_kernel(widen_kernel<RowFormat::kFp8>, grid, block, 0, stream, p);
    case RowFormat::kFp4: return launch_kernel(widen_kernel<RowFormat::kFp4>, grid, block, 0, stream, p);
    case RowFormat::kFp8V41: return launch_kernel(widen_kernel<RowFormat::kFp8V41>, grid, block, 0, stream, p);
    case RowFormat::kFp4V41: return launch_kernel(widen_kernel<RowFormat::kFp4V41>, grid, block, 0, stream, p);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rows(RowFormat fmt, const RowsParams& p, bool append, cudaStream_t stream) {
  if (p.rows <= 0) return cudaSuccess;
  switch (fmt) {
    case RowFormat::kBf16: return launch<RowFormat::kBf16>(p, append, stream);
    case RowFormat::kFp8: return launch<RowFormat::kFp8>(p, append, stream);
    case RowFormat::kFp4: return launch<RowFormat::kFp4>(p, append, stream);
    case RowFormat::kFp8V41: return launch<RowFormat::kFp8V41>(p, append, stream);
    case RowFormat::kFp4V41: return launch<RowFormat::kFp4V41>(p, append, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace mla
