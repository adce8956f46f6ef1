// Cache rows: parameters and launcher of the append and gather kernels.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace mla {

enum class RowFormat { kBf16, kFp8, kFp4, kFp8V41, kFp4V41 };

struct RowsParams {
  const __nv_bfloat16* c_kv;     // append: [rows, >= 512], row stride c_stride values
  const __nv_bfloat16* k_rope;   // append: [rows, >= 64], row stride r_stride values
  long long c_stride, r_stride;
  uint8_t* cache;                // [num_pages, 64, row bytes]
  const int32_t* block_table;    // [batch, max_pages]
  const int32_t* seq_lens;       // [batch]
  const int32_t* cu_rows;        // [batch + 1]
  int batch, rows, num_pages, max_pages;
  __nv_bfloat16* out;            // gather and widen: rows of 576
  int* status;
};

// The rotation of an append's RoPE values: the rows' positions (null: their
// token indexes) and the table.
struct RowsRope {
  const int32_t* positions;      // [rows]
  mla_rope table;
};

// The sequences' pages in a quantised format as bf16 rows [batch, max_pages 64,
// 576] in p.out (p.cache, block_table, seq_lens, batch, num_pages, max_pages
// set; batch <= 65535).
cudaError_t launch_widen(RowFormat fmt, const RowsParams& p, cudaStream_t stream);
cudaError_t launch_rows(RowFormat fmt, const RowsParams& p, bool append, cudaStream_t stream);
cudaError_t launch_append_rope(RowFormat fmt, const RowsParams& p, const RowsRope& rope, cudaStream_t stream);

}  // namespace mla
