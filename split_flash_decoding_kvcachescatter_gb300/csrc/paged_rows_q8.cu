// paged_rows_q8.cu -- attention of chunks of new tokens in float32 over a paged KV
// cache in 8 bits (the kernel: kvs_rows.cuh, the products: kvs_rows_q8.cuh).
//
// Bound: mma.sync and the conversion of each number to float16, once for 16 rows; two
// products a weight or score, where plain float32 pages take three of half the rate.
// Measured: 1001 new tokens of three sequences over up to 2048, H 14 / 2, D 64 42 us
// (plain pages 80 to 93), H 40 / 8, D 128 201 us; by units of 16 rows 75 and 427.

#include "kvs_rows.cuh"
#include "kvs_rows_q8.cuh"

namespace kvs {

namespace {

// Pages in 8 bits under q and out in float32.
template <int D_>
struct RowPagesQ8 : LinesQ8<D_, RowsQ8<float, D_, false>::KT> {
  static constexpr int D = D_, kElem = 1;
  using Rows = RowsQ8<float, D, false>;
  static constexpr bool kScaled = true;
  // 600 new tokens of nine sequences, six of them decoding, over up to 3000 keys, H 40 / 8, D 128: 227
  // us at 32 cost rows, 218 at 64, 210 at 128, 215 at 256, 227 at 512
  static constexpr int kFix = 128;
  using Extra = ScalesQ8;
};

template <int D>
int launch_q8(const void *q, long long q_stride, const kvs_paged_cache_q8 &cache,
              const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
              int *d_status, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)cache.num_pages * cache.num_kv_heads * cache.page_size;
  int rc = make_line_map(&kmap, cache.k_pages, rows * D / 128, 16 * D / 128);
  if (rc == KVS_OK) rc = make_line_map(&vmap, cache.v_pages, rows * D / 128, 16 * D / 128);
  if (rc != KVS_OK) return rc;
  return launch_rows<RowPagesQ8<D>>(q, q_stride, kmap, vmap, {cache.k_scales, cache.v_scales},
                                    cache.num_kv_heads, pa, out, out_stride, H, workspace, d_status,
                                    stream);
}

}  // namespace

int set_wait_limit_rows_q8(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

size_t paged_rows_workspace_bytes(int D) { return rows_workspace_bytes(D); }

int launch_paged_rows_q8(const void *q, long long q_stride, const kvs_paged_cache_q8 &cache,
                         const PagedArgs &pa, void *out, long long out_stride, int H,
                         void *workspace, int *d_status, cudaStream_t stream) {
  return cache.head_dim == 64 ? launch_q8<64>(q, q_stride, cache, pa, out, out_stride, H, workspace,
                                              d_status, stream)
                              : launch_q8<128>(q, q_stride, cache, pa, out, out_stride, H, workspace,
                                               d_status, stream);
}

}  // namespace kvs
