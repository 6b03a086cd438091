// Tensor maps for TMA copies of the caller's tensors, encoded per call.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8moe {

// A map of a tensor of `rank` dimensions, the innermost (contiguous) first:
// sizes in elements, strides in bytes of the outer dimensions (multiples of 16),
// the box that a copy takes, 128-byte swizzle (the box's rows are 128 bytes).
// Elements outside the tensor read as zeros.
inline bool encode_tile_map(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *ptr, const uint64_t *sizes,
                            const uint64_t *strides, const uint32_t *box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (encode == nullptr) return false;
  cuuint64_t n[5], st[5];
  cuuint32_t b[5], one[5];
  for (int i = 0; i < rank; ++i) {
    n[i] = sizes[i];
    b[i] = box[i];
    one[i] = 1;
    if (i + 1 < rank) st[i] = strides[i];
  }
  return encode(m, type, (cuuint32_t)rank, const_cast<void *>(ptr), n, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fp8moe
