// paged_attention.cu -- attention of a ragged batch's new tokens over a paged
// KV cache: the choice of kernel, and chunks in float32 (the kernel: kvs_rows.cuh).
//
// Mathematics: flash attention over a split key axis.  For a row (token,
// query head) and a set of keys, (m, l, acc) = (max s_j, sum 2^(s_j - m),
// sum 2^(s_j - m) v_j), s_j = log2(e) q.k_j / sqrt(D); sets merge by
// rescaling to the larger m, and the row's output is acc / l.
//
// Work unit of all kernels: (sequence, row tile, kv head).  A row tile
// is TT = RT / G whole tokens with the G query heads of the group: RT rows
// share every K and V row.  Units follow each other on one line of "cost
// rows" (a fixed price, then one per key a unit attends); the line is cut
// into ranges, whatever the lengths are: a block runs the key tiles that
// start in its range.  A unit inside one range is written directly; the
// pieces of a unit that spans ranges go to the workspace, and the block that
// completes the unit merges them in order (the tagged counters of
// kvs_tags.cuh; no block waits for another).  Everything is derived on the
// device from the positions and offsets, so a captured graph follows them.
//
// Kernels: rows that a unit's 16 can hold (max_new G <= 16: a decode step)
// paged_decode.cu; more rows in 16 bits paged_chunk.cu (tcgen05); more rows
// in float32 kvs_rows.cuh's, on mma.sync: float32 as three TF32 products of a
// high and a low part (hi hi + hi lo + lo hi), off by 2^-21 of it at most (lo lo 2^-22,
// a lost bit of each lo 2^-23).
//
// Measured (chunks in float32): 1001 new tokens of three sequences over up to 2048, H 14 / 2, D 64:
// 57 to 74 us by the positions (65 us at 3.7 GFLOP, whose three TF32 products
// would take 36 us at the 303 TFLOP/s that mma.sync reaches here; splitting the
// operands and the softmax take the rest).  At positions where it took 82 us:
// 101 with the pieces of split units joined from memory by one group of threads;
// dearer units in the split 84 us (128 cost rows) and 92 (256); 11 warps of fewer
// registers 84.  1001 tokens over up to 1900, H 40 / 8, D 128: 483 us
// (22.6 GFLOP; 223 us).


#include "kvs_rows.cuh"

namespace kvs {

namespace {

// Plain pages in float32 (kvs_rows.cuh).
template <int D_>
struct PlainRows {
  static constexpr int D = D_, kElem = 4;
  using Rows = WarpRows<float, D>;
  static constexpr bool kScaled = false;
  static constexpr int kFix = 64;
  struct Extra {};
  static __device__ __forceinline__ int map_row(int row) { return row; }
  // Rows `left` and up of a tile become zero (by one warp).
  static __device__ __forceinline__ void clear_rows(unsigned char *tile, int left) {
    constexpr int KT = Rows::KT, GB = 16 * D * 4, BLK = 2048;  // BLK: a column block of a 16-row copy
    const int lane = threadIdx.x & 31;
    for (int e = lane; e < (KT - left) * (D / 4); e += 32) {
      const int row = left + e % (KT - left), pc = e / (KT - left);
      *reinterpret_cast<uint4 *>(tile + (row >> 4) * GB + (pc >> 3) * BLK +
                                 (row & 15) * 128 + (pc & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
};

template <int D>
int launch_plain(const void *q, long long q_stride, const kvs_paged_cache &cache,
                 const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                 int *d_status, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)cache.num_pages * cache.num_kv_heads * cache.page_size;
  int rc = make_row_map(&kmap, cache.k_pages, rows, D, cache.dtype, 16, D / 32);
  if (rc == KVS_OK) rc = make_row_map(&vmap, cache.v_pages, rows, D, cache.dtype, 16, D / 32);
  if (rc != KVS_OK) return rc;
  return launch_rows<PlainRows<D>>(q, q_stride, kmap, vmap, {}, cache.num_kv_heads, pa, out,
                                   out_stride, H, workspace, d_status, stream);
}

// A decode step: every sequence's rows with the G heads of a group fit the 16
// rows of a paged_decode unit.
bool is_decode(long long max_new, int G) { return max_new * G <= 16; }

}  // namespace

int set_wait_limit_paged(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

size_t paged_attention_workspace_bytes(int H, int Hkv, int D, int max_new) {
  if (is_decode(max_new, H / Hkv)) return paged_decode_workspace_bytes(D);
  return std::max(rows_workspace_bytes(D), paged_chunk_workspace_bytes(D));
}

int launch_paged_attention(const void *q, long long q_stride, const kvs_paged_cache &cache,
                           const PagedArgs &pa, void *out, long long out_stride, int H,
                           void *workspace, int *d_status, cudaStream_t stream) {
  if (is_decode(pa.max_new, H / cache.num_kv_heads))
    return launch_paged_decode(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status,
                               stream);
  if (cache.dtype != KVS_F32)
    return launch_paged_chunk(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status,
                              stream);
  if (cache.head_dim == 64)
    return launch_plain<64>(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status, stream);
  return launch_plain<128>(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status, stream);
}

}  // namespace kvs
