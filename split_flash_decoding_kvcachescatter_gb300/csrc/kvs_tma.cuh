// kvs_tma.cuh -- tensor maps: multi-dimensional bulk copies (TMA) of cache
// rows into shared memory with the 128-byte swizzle.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kvs_device.cuh"
#include "kvsdecode.h"

namespace kvs {

using TensorMapEncode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                     const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                     const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder (nullptr if it cannot be found).
static inline TensorMapEncode tensor_map_encoder() {
  static TensorMapEncode fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return (TensorMapEncode) nullptr;
    }
    return reinterpret_cast<TensorMapEncode>(p);
  }();
  return fn;
}

// Calls the encoder.  It needs the device's context current in the calling
// thread, which a thread has only once it has made a runtime call that binds
// it; the encoder itself does not.
template <typename... Args>
static inline int encode_map(Args... args) {
  const TensorMapEncode enc = tensor_map_encoder();
  if (!enc) return KVS_ERR_LAUNCH;
  CUresult r = enc(args...);
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) {
      cudaGetLastError();
      return KVS_ERR_LAUNCH;
    }
    r = enc(args...);
  }
  return r == CUDA_SUCCESS ? KVS_OK : KVS_ERR_LAUNCH;
}

// Map over `rows` rows of D elements (contiguous), cut into column blocks of
// 128 bytes: a copy of box_rows rows and `blocks` column blocks fills
// [blocks][box_rows][128 bytes] of shared memory, 16-byte pieces swizzled by
// the row (piece c of row r at c ^ (r % 8)).  Coordinates (0, row, block).
static inline int make_row_map(CUtensorMap *map, const void *base, uint64_t rows, int D, int dtype,
                               int box_rows, int blocks) {
  const int size = dtype == KVS_F32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)(128 / size), rows, (cuuint64_t)(D * size / 128)};
  const cuuint64_t strides[2] = {(cuuint64_t)D * size, 128};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, (cuuint32_t)blocks};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUtensorMapDataType type = dtype == KVS_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == KVS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode_map(map, type, 3, const_cast<void *>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Map over `lines` lines of 128 bytes: a copy of box_lines of them, 16-byte pieces
// swizzled likewise.  Coordinates (0, line, 0).
static inline int make_line_map(CUtensorMap *map, const void *base, uint64_t lines, int box_lines) {
  const cuuint64_t dims[3] = {128, lines, 1};
  const cuuint64_t strides[2] = {128, 128};
  const cuuint32_t box[3] = {128, (cuuint32_t)box_lines, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides,
                    box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Map over rows of [heads][D] 16-bit elements, row_stride elements apart: a
// copy takes box_heads heads of box_rows rows, one column block of 64
// elements, as [box_rows][box_heads][128 bytes], swizzled likewise.
// Coordinates (0, head, row, block).
static inline int make_q_map(CUtensorMap *map, const void *base, uint64_t rows, int64_t row_stride,
                             int heads, int D, int dtype, int box_rows, int box_heads) {
  const cuuint64_t dims[4] = {64, (cuuint64_t)heads, rows, (cuuint64_t)(D / 64)};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)row_stride * 2, 128};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type =
      dtype == KVS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode_map(map, type, 4, const_cast<void *>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The box at row `row` into dst (1024-byte aligned), counted on `bar`.
__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *map, int row, uint64_t *bar,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(0), "r"(row), "r"(0), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// Four bytes global -> shared, asynchronously ...
__device__ __forceinline__ void copy_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// ... and an arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void arrive_when_copied(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace kvs
