// What the two kernels behind flux_linear_fp8 share: tensor maps over 8-bit rows.
#pragma once

#include "linear_common.cuh"

namespace flux {

// Channels of a group (a scale's, and a pipeline stage's: 128 bytes, one
// swizzle row).
constexpr int kGroupK = 128;

// A 3-D tensor map over 8-bit rows [B, S, cols] with the given strides; one box
// = 128 columns x box_rows tokens, swizzled over its 128 bytes. Elements
// outside the tensor read as zero.
inline bool make_byte_map(CUtensorMap *map, const void *base, int64_t cols, int64_t S, int64_t B,
                          int64_t row_stride, int64_t batch_stride, uint32_t box_rows) {
  auto fn = reinterpret_cast<CUresult (*)(
      CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
      const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)>(
      tensor_map_encode_entry());
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(S),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_stride),
                                 static_cast<cuuint64_t>(batch_stride)};
  const cuuint32_t box[3] = {kGroupK, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

}  // namespace flux
