// cuTensorMapEncodeTiled through the runtime, so that the library does not link the driver.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "paged.cuh"

namespace binattn {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Tokens that one copy brings of a block of `block` keys: the largest of block, block / 2, .. 16 that
// divides a page.
inline int v_unit(const CacheView& cv, int block) {
  int unit = block;
  while (cv.page_size % unit != 0) unit /= 2;
  return unit;
}

// The V rows of all blocks of a cache as (byte, token, block): a copy brings `unit` rows of a page,
// padded with zeros to `row` (64 or 128) bytes and swizzled over that width.
inline bool v_rows_map(const CacheView& cv, int row, int unit, CUtensorMap* map) {
  *map = CUtensorMap{};
  if (cv.num_pages == 0) return true;  // never used
  EncodeTiledFn enc = encode_fn();
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cv.dp), static_cast<cuuint64_t>(cv.page_size),
                              static_cast<cuuint64_t>(cv.num_pages) * cv.heads};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cv.dp), static_cast<cuuint64_t>(cv.block_bytes)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(row), static_cast<cuuint32_t>(unit), 1}, step[3] = {1, 1, 1};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, cv.data, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace binattn
