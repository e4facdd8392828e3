// kvs_paged.cuh -- the device view of a ragged batch over a paged cache, and
// the element types of the paged-cache and logit kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvs_device.cuh"
#include "kvs_launch.h"
#include "kvsdecode.h"

namespace kvs {

// One sequence of the batch: first position, new tokens and first row of q
// and out; n = 0 when there is nothing to do, err when the sequence is bad
// (n and row0 are then the rows to mark, 0 rows if the offsets are bad).
struct PagedSeq {
  int p, n, row0, err;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs &b, int i) {
  const int a = __ldca(b.row_offsets + i), e = __ldca(b.row_offsets + i + 1);
  const int p = __ldca(b.positions + i);
  PagedSeq s{p, 0, a, KVS_OK};
  if (a < 0 || e < a || e > b.num_rows || e - a > b.max_new) {
    s.err = KVS_ERR_ROWS;
    return s;
  }
  s.n = e - a;
  if (s.n > 0 && (p < 0 || (long long)p + s.n > (long long)b.max_pages << b.page_shift))
    s.err = KVS_ERR_POSITION;
  return s;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N elements of T moved by one load or store (N * sizeof(T) = 2, 4, 8 or 16
// bytes, aligned to that).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T e[N];
};

// Coherent at L2: with programmatic dependent launch the data may have been
// written by the preceding kernel.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> vec_load(const T *p) {
  Vec<T, N> v;
  if constexpr (sizeof(v) == 16) {
    *reinterpret_cast<uint4 *>(&v) = __ldcg(reinterpret_cast<const uint4 *>(p));
  } else if constexpr (sizeof(v) == 8) {
    *reinterpret_cast<uint2 *>(&v) = __ldcg(reinterpret_cast<const uint2 *>(p));
  } else if constexpr (sizeof(v) == 4) {
    *reinterpret_cast<unsigned *>(&v) = __ldcg(reinterpret_cast<const unsigned *>(p));
  } else {
    *reinterpret_cast<unsigned short *>(&v) = __ldcg(reinterpret_cast<const unsigned short *>(p));
  }
  return v;
}

template <typename T, int N>
__device__ __forceinline__ void vec_store(T *p, const Vec<T, N> &v) {
  if constexpr (sizeof(v) == 16) {
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&v);
  } else if constexpr (sizeof(v) == 8) {
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(&v);
  } else if constexpr (sizeof(v) == 4) {
    *reinterpret_cast<unsigned *>(p) = *reinterpret_cast<const unsigned *>(&v);
  } else {
    *reinterpret_cast<unsigned short *>(p) = *reinterpret_cast<const unsigned short *>(&v);
  }
}

}  // namespace kvs
