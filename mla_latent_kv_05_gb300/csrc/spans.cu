#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "spans.cuh"

namespace mla {

namespace {
constexpr uint64_t kFast = 128u << 10;   // see spans.cuh
}

uint64_t tma_far(const void* base, uint64_t bytes) {
  if (bytes >= kFast) return 0;
  static const PFN_cuMemGetAddressRange_v3020 range = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &ptr, 3020, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuMemGetAddressRange_v3020>(ptr);
  }();
  CUdeviceptr start = 0;
  size_t size = 0;
  const CUdeviceptr at = reinterpret_cast<CUdeviceptr>(base);
  if (!range || range(&start, &size, at) != CUDA_SUCCESS) return 0;
  return at >= start && at + kFast + bytes <= start + size ? kFast : 0;
}

}  // namespace mla
