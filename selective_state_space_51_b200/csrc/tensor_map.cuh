// TMA descriptors of token rows.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t,
                                 void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

// The driver's encoder, by name (the library links no driver).
inline EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// [batch][token][head][size] bfloat16 rows, `stride` elements from a token to
// the next, read in boxes of `tokens` rows of 64 elements (128 bytes, in the
// 128-byte swizzle); what lies outside the tensor reads as zero. The base and
// the strides are multiples of 16 bytes (the caller has checked), and every
// box starts at a multiple of 64 elements.
inline bool row_map(CUtensorMap *map, const void *base, int64_t batch,
                    int64_t seqlen, int heads, int size, int64_t stride,
                    int tokens) {
  const EncodeTiled encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[4] = {cuuint64_t(size), cuuint64_t(heads),
                              cuuint64_t(seqlen), cuuint64_t(batch)};
  const cuuint64_t steps[3] = {cuuint64_t(size) * 2, cuuint64_t(stride) * 2,
                               cuuint64_t(stride) * cuuint64_t(seqlen) * 2};
  const cuuint32_t box[4] = {64, 1, cuuint32_t(tokens), 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void *>(base), dims, steps, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ssm
