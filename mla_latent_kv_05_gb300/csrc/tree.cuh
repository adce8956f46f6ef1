// Tree decode over bf16 rows: tensor maps and launcher (see tree.cu).
#pragma once
#include "decode.cuh"

namespace mla {

// 64 values x 64 rows x chunks: absorbed queries (eight chunks of 64 heads),
// their RoPE part, and a page's K groups and V halves.
struct TreeMaps {
  CUtensorMap q, qr, k, v;
};

// p.kv_bf16, p.tree_nodes and p.tree_seqs set; rows planned with one query each,
// node by node.  p.block_table
// may be null: page t of sequence b is page b p.max_pages + t.
cudaError_t launch_tree(PFN_cuTensorMapEncodeTiled_v12000 encode, const DecodeParams& p, int n_pairs, bool pdl,
                        cudaStream_t stream);

// A part of a row in launch_tree's partials: fp32 pieces of 32 heads x 8 columns
// (a head's eight in a row), as a warp holds them.  Offset of the piece of heads
// [32 group, +32) and columns [128 quarter + 8 chunk, +8).
__host__ __device__ inline int part_piece(int group, int quarter, int chunk) {
  return ((group * 4 + quarter) * 16 + chunk) * 256;
}

// The merge of split rows, and of rows with no token: `rows` planned rows, node
// by node over `seqs` sequences.
cudaError_t launch_combine_tree(const void* ws, const WsLayout& Lw, int rows, int seqs, __nv_bfloat16* out, float* lse,
                                bool pdl, cudaStream_t stream);

}  // namespace mla
