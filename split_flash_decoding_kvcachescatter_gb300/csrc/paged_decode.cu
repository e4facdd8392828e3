// paged_decode.cu -- attention of single tokens over a paged KV cache of
// float32, float16 or bfloat16 (the kernels: kvs_decode.cuh).
//
// Products run on mma.sync (16 rows: an M = 128 tcgen05 tile would be seven
// eighths padding): m16n8k16 for the 16-bit types, float32 as three TF32
// products.  A 32-key tile of a decode step costs a warp about 900 cycles for
// 16 KB where HBM delivers 23 bytes a cycle an SM, so four warps keep ahead.
//
// Measured (GB300, copy peak 6.79 TB/s): 8 x 32768 keys, H 32 / 8, D 128,
// float16 (1.07 GB) 162 us, 97 % of the peak; 32 sequences of up to 8192 keys
// in bfloat16 (586 MB) 93 us, 93 %; 8 x 32768 in float32 (2.15 GB; 16-key tiles,
// q split again for each) 403 us, 79 %.  (float32, D 64: 76 bytes a thread
// spill.)  Tried: one producer warp for all four rings 190 us (it needs about
// 1000 cycles a tile), two producers of two rings 234 us (rings wait for each
// other); a warp of its own for the joining 171 and 107 us; with it the last
// fifth of the line in short ranges handed out by a counter, 180 and 114 us
// (blocks then finish within 10 % of each other, not 26 %, but a long unit's 24
// pieces are slow to join).

#include "kvs_decode.cuh"

namespace kvs {

namespace {

// Pages of T (kvs_decode.cuh).
template <typename Type, int D_>
struct PlainPages {
  using T = Type;
  using Rows = WarpRows<T, D_>;
  static constexpr int D = D_, kElem = sizeof(T);
  static constexpr int kRings = 4;
  static constexpr bool kScaled = false, kOnlyFew = false;
  static constexpr bool kFewForm = !std::is_same<T, float>::value;  // units of 8 rows have a form
  struct Extra {};
  // A unit's fixed price (its start, the joining of its four states, its output)
  // in bytes of K and V: 32 sequences of up to 8192 keys, H 32 / 8, D 128,
  // bfloat16, took 104 us at 32 KB, 98 at 96, 94 at 128, 92.7 at 192, 93.0 at
  // 256; 32 of up to 4500 62, 55, 48.6, 45.6 and 44.7 us (float32: 134, 123,
  // 121, 123, 125).
  static constexpr int kFixBytes = 192 << 10;
  // Rules for clusters: the K and V bytes of a block, and those of a unit that
  // halves the block, all counted as if every page of a table were in use.
  static constexpr long long kBlockBytes = 1 << 20;
  static constexpr long long kShortBytes = kElem == 4 ? 128 << 10 : 512 << 10;
  static __device__ __forceinline__ int map_row(int row) { return row; }
  // Rows `left` and up of a tile become zero (by one warp).
  static __device__ __forceinline__ void clear_rows(unsigned char *tile, int left) {
    constexpr int KT = Rows::KT;
    for (int e = threadIdx.x & 31; e < (KT - left) * (D * kElem / 16); e += 32) {
      const int row = left + e % (KT - left), pc = e / (KT - left);
      *reinterpret_cast<uint4 *>(tile + (row >> 4) * (16 * D * kElem) + (pc >> 3) * 2048 +
                                 (row & 15) * 128 + (pc & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
};

template <typename T, int D>
int launch_plain(const void *q, long long q_stride, const kvs_paged_cache &cache,
                 const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                 int *d_status, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)cache.num_pages * cache.num_kv_heads * cache.page_size;
  int rc = make_row_map(&kmap, cache.k_pages, rows, D, cache.dtype, 16,
                        D * (int)sizeof(T) / 128);
  if (rc == KVS_OK) rc = make_row_map(&vmap, cache.v_pages, rows, D, cache.dtype, 16,
                        D * (int)sizeof(T) / 128);
  if (rc != KVS_OK) return rc;
  return launch_decode<PlainPages<T, D>>(q, q_stride, kmap, vmap, {}, cache.num_kv_heads, pa, out,
                                         out_stride, H, workspace, d_status, stream);
}

}  // namespace

int set_wait_limit_decode(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

// Workspace: 256 bytes (epoch), a counter per block, then per block two
// partial slots (0: a unit begun in an earlier range, 1: one begun here and
// not finished).
size_t paged_decode_workspace_bytes(int D) {
  return 256 + (size_t)kPagedMaxBlocks * 8 +
         2 * (size_t)kPagedMaxBlocks * paged_slot_floats(kDRows, D) * 4;
}

int launch_paged_decode(const void *q, long long q_stride, const kvs_paged_cache &cache,
                        const PagedArgs &pa, void *out, long long out_stride, int H,
                        void *workspace, int *d_status, cudaStream_t stream) {
#define KVS_DECODE(T)                                                                           \
  return cache.head_dim == 64                                                                   \
             ? launch_plain<T, 64>(q, q_stride, cache, pa, out, out_stride, H, workspace,      \
                                    d_status, stream)                                           \
             : launch_plain<T, 128>(q, q_stride, cache, pa, out, out_stride, H, workspace,     \
                                     d_status, stream)
  if (cache.dtype == KVS_F32) KVS_DECODE(float);
  if (cache.dtype == KVS_F16) KVS_DECODE(__half);
  KVS_DECODE(__nv_bfloat16);
#undef KVS_DECODE
}

}  // namespace kvs
