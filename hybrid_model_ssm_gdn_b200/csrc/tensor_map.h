// tensor_map.h -- tensor maps of the kernels that load tiles by TMA.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace rssm {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled from the driver that is loaded (the library links the runtime alone)
inline cudaError_t map_encoder(EncodeTiled *fn) {
  void *p = nullptr;
  cudaDriverEntryPointQueryResult found;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
  *fn = reinterpret_cast<EncodeTiled>(p);
  return cudaSuccess;
}

// tiles, unless told otherwise of rows of 128 bytes with the 128-byte swizzle; what lies outside the tensor reads as zero and
// is not written
inline cudaError_t make_map(EncodeTiled fn, CUtensorMap *map, CUtensorMapDataType type, const void *p, int dims,
                            const cuuint64_t *size, const cuuint64_t *stride, const cuuint32_t *box,
                            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = fn(map, type, dims, const_cast<void *>(p), size, stride, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace rssm
