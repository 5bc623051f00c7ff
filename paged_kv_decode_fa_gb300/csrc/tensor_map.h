// TMA descriptors of query rows and cache pages for the tcgen05 kernels: boxes of 64
// 16-bit elements (128 bytes, swizzled), the rows of a K-major operand, or of codes.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "fa_decode.h"
#include "kernels.h"

namespace fadecode {

inline bool encode_map(CUtensorMap* map, fa_dtype dt, int rank, const void* base,
                       const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                       bool swizzle64 = false) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (!fn) return false;
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return fn(map,
            dt == FA_DTYPE_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
            : dt == FA_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
            (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether q's rows can be described to the tensor copies: strides that are taken are
// positive, whole 16 bytes and below 2^40 bytes.
inline bool q_rows_fit(const fa_rows& q, int64_t rows, int heads) {
  const auto fits = [](int64_t stride) { return stride > 0 && stride < (int64_t)1 << 39; };
  return reinterpret_cast<uintptr_t>(q.data) % 16 == 0 && q.token_stride % 8 == 0 &&
         q.head_stride % 8 == 0 && (rows <= 1 || fits(q.token_stride)) &&
         (heads <= 1 || fits(q.head_stride));
}

// q [rows, heads, D]: a box is the `group` heads of 128 / group rows, 64 dims.
inline bool encode_q_rows(CUtensorMap* map, fa_dtype dt, const fa_rows& q, int64_t rows,
                          int heads, int D, int group) {
  // a stride that is never taken may be anything: one that the encoder accepts
  const cuuint64_t row = (cuuint64_t)D * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {heads > 1 ? (cuuint64_t)q.head_stride * 2 : row,
                                 rows > 1 ? (cuuint64_t)q.token_stride * 2 : row};
  const cuuint32_t box[3] = {64u, (cuuint32_t)group, (cuuint32_t)(128 / group)};
  return encode_map(map, dt, 3, q.data, dims, strides, box);
}

// The pages of a cache, [2 * pages][16][heads][D]: a box is one head's rows of one
// page's K or V, 64 dims.
inline bool encode_pages(CUtensorMap* map, fa_dtype dt, const void* kv, int64_t pages, int heads,
                         int D) {
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)kPageSize,
                              (cuuint64_t)(2 * pages)};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2,
                                 (cuuint64_t)kPageSize * heads * D * 2};
  const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)kPageSize, 1u};
  return encode_map(map, dt, 4, kv, dims, strides, box);
}

// The pages of an E4M3 cache: a box is one head's rows of one page's K or V, D codes
// (64 or 128 bytes, swizzled in spans of as many).
inline bool encode_codes(CUtensorMap* map, const void* kv, int64_t pages, int heads, int D) {
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)kPageSize,
                              (cuuint64_t)(2 * pages)};
  const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)heads * D,
                                 (cuuint64_t)kPageSize * heads * D};
  const cuuint32_t box[4] = {(cuuint32_t)D, 1u, (cuuint32_t)kPageSize, 1u};
  return encode_map(map, FA_DTYPE_E4M3, 4, kv, dims, strides, box, D == 64);
}

}  // namespace fadecode
