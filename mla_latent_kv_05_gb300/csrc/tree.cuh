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

}  // namespace mla
