// Host-side TMA tensor-map construction through the driver entry point
// (no link-time dependency on libcuda).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <cstdint>

namespace fa {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// 3-D map over 16-bit rows of `cols` contiguous elements, row_stride elements apart, in `heads`
// matrices head_stride elements apart (strides multiples of 16 bytes); boxes and fill as below.
inline bool make_tmap_16bit_strided(CUtensorMap* map, const void* base, bool bf16, uint64_t cols, uint64_t rows,
                                    uint64_t heads, uint64_t row_stride, uint64_t head_stride, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, heads};
  cuuint64_t strides[2] = {row_stride * 2, head_stride * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D map over a [heads][rows][cols] row-major array of 16-bit elements (cols
// contiguous), read in boxes of 64 columns (128 bytes) x box_rows rows with the
// 128-byte swizzle; rows beyond `rows` read as zero.
inline bool make_tmap_16bit_3d(CUtensorMap* map, const void* base, bool bf16, uint64_t cols, uint64_t rows,
                               uint64_t heads, uint32_t box_rows) {
  return make_tmap_16bit_strided(map, base, bf16, cols, rows, heads, cols, cols * rows, box_rows);
}

// 3-D map over a [heads][rows][cols] row-major array of bytes (FP8 codes), boxes of 128 columns
// (128 bytes) x box_rows rows with the 128-byte swizzle, or, for 64-byte rows (swizzle_bytes 64),
// boxes of 64 columns with the 64-byte swizzle; rows beyond `rows` read as zero.
inline bool make_tmap_8bit_3d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t heads,
                              uint32_t box_rows, uint32_t swizzle_bytes = 128) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, heads};
  cuuint64_t strides[2] = {cols, cols * rows};
  cuuint32_t box[3] = {swizzle_bytes, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D map over a [heads][rows][cols] row-major fp32 array, boxes of box_cols x box_rows,
// optionally with the 128-byte swizzle (then box_cols * 4 must be 128).
inline bool make_tmap_f32_3d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t heads,
                             uint32_t box_cols, uint32_t box_rows, bool swizzle128) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, heads};
  cuuint64_t strides[2] = {cols * 4, cols * rows * 4};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace fa
