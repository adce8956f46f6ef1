// Expansion of latent rows into keys and values: launcher (see expand.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"

namespace mla {

// latent: [rows, 512] bf16, row stride in values; w_uk, w_uv: [128, 128, 512]
// bf16; k_nope, v: [rows, 128, 128] bf16; sms: CTAs to launch at most.
cudaError_t launch_expand(PFN_cuTensorMapEncodeTiled_v12000 encode, const void* latent, long long row_stride,
                          const void* w_uk, const void* w_uv, int rows, void* k_nope, void* v, void* hdr, int sms,
                          cudaStream_t stream);

}  // namespace mla
