// Pieces shared by the grouped products (grouped_gemm.cu, ffn.cu): an expert's
// segment and the tensor maps of row operands.
#pragma once

#include "lrm_internal.cuh"

namespace lrm {

constexpr int MAX_E = 1024;

// Start row and length of expert e's segment, clamped to the buffers.
__device__ __forceinline__ void segment(const int32_t* __restrict__ sel_offsets, int e, int max_rows, int& start,
                                        int& len) {
  int st = __ldg(sel_offsets + e), en = __ldg(sel_offsets + e + 1);
  st = min(max(st, 0), max_rows);
  en = min(max(en, st), max_rows);
  start = st;
  len = en - st;
}

// Row-major 2-D bf16 tensor [rows][cols] with [box_rows][64] boxes.
inline lrm_status encode_2d(lrm_ctx* ctx, CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                            uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = ctx->encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                                 box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LRM_OK : LRM_ERR_CUDA;
}

}  // namespace lrm
