// paged_decode_q8.cu -- attention over a paged KV cache in 8 bits: the choice of
// kernel, and single tokens (the kernels: kvs_decode.cuh, the products:
// kvs_rows_q8.cuh).  Chunks in 16 bits: paged_chunk_q8.cu, long ones in float32:
// paged_rows_q8.cu.
//
// Bound: HBM, half the bytes of 16-bit pages; then the conversions and products of what
// comes twice as fast.  Measured (H 32 / 8, D 128): 8 x 32768 keys in float16 90 us, 88% of
// the copy rate (4 consumer warps 108, 6 with spilled registers 125); 32 of up to 8192 in
// bfloat16 58 us (66 by 4 warps).

#include "kvs_decode.cuh"
#include "kvs_rows_q8.cuh"

namespace kvs {

namespace {

// Pages in 8 bits under q and out of Type (kvs_decode.cuh); kFew: units of 8 rows at most,
// for which 16-bit rows leave registers for eight consumer warps a block.
template <typename Type, int D_, bool kFew>
struct PagesQ8 : LinesQ8<D_, RowsQ8<Type, D_>::KT> {
  using T = Type;
  using Rows = RowsQ8<T, D_>;
  static constexpr int D = D_, kElem = 1;
  static constexpr int kRings = kFew && sizeof(T) == 2 ? 8 : 4;
  static constexpr bool kScaled = true, kOnlyFew = kFew;
  static constexpr bool kFewForm = true;
  using Extra = ScalesQ8;
  // as PlainPages'; 32 sequences of up to 8192 keys in bfloat16 took 66.3 us at 96 KB, 58.3 at 192,
  // 60.6 at 384, 65.6 at 768
  static constexpr int kFixBytes = 192 << 10;
  // us by clusters and by equal ranges, bfloat16, all of full length, H 32 / 8, D 128:
  //   sequences x keys       1x16384   4x8192  16x2048  32x1024  64x1024  32x2048  64x2048  16x4096
  //   KB a block                 256      512      512      256      256      512      512     1024
  //   clusters                  19.1     19.9     19.6     24.1     46.2     37.6     73.3     33.0
  //   equal ranges              19.7     22.4     24.8     27.0     42.1     36.4     60.8     33.6
  //   1/8 to all, clusters      14.4     19.3     18.7     20.5     37.1     30.9     53.6     32.5
  //   the same, ranges          17.5     19.1     20.7     23.2     35.3     29.4     46.0     26.8
  // (H 14 / 2, D 64, 16 x 16384, 512 KB: 20.8 and 22.5, 20.1 and 18.0.)  Twice as much a block
  // loses up to a fifth where lengths differ, half as much 5 us for one to 16 sequences.
  static constexpr long long kBlockBytes = 512 << 10;
  // us with half a block an SM and with a whole one, 64 x 256, 512, 1024, 2048 keys: 20.5, 29.2,
  // 45.5, 77.9 and 24.7, 32.1, 46.2, 73.3; of 1/8 to all 19.2, 25.7, 39.1, 63.5 and 23.6, 27.9,
  // 37.1, 53.6 (64, 128, 256, 512 KB a unit)
  static constexpr long long kShortBytes = 128 << 10;
};

template <typename T, int D>
int launch_q8(const void *q, long long q_stride, const kvs_paged_cache_q8 &cache,
              const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
              int *d_status, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)cache.num_pages * cache.num_kv_heads * cache.page_size;
  int rc = make_line_map(&kmap, cache.k_pages, rows * D / 128, 16 * D / 128);
  if (rc == KVS_OK) rc = make_line_map(&vmap, cache.v_pages, rows * D / 128, 16 * D / 128);
  if (rc != KVS_OK) return rc;
  if ((long long)pa.max_new * (H / cache.num_kv_heads) <= 8)
    return launch_decode<PagesQ8<T, D, true>>(q, q_stride, kmap, vmap, {cache.k_scales, cache.v_scales},
                                              cache.num_kv_heads, pa, out, out_stride, H, workspace,
                                              d_status, stream);
  return launch_decode<PagesQ8<T, D, false>>(q, q_stride, kmap, vmap, {cache.k_scales, cache.v_scales},
                                             cache.num_kv_heads, pa, out, out_stride, H, workspace,
                                             d_status, stream);
}

}  // namespace

int set_wait_limit_decode_q8(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

size_t paged_attention_q8_workspace_bytes(int H, int Hkv, int D, int max_new) {
  const size_t few = paged_decode_workspace_bytes(D);
  return (long long)max_new * (H / Hkv) <= kDRows
             ? few
             : std::max({few, paged_chunk_workspace_bytes(D), paged_rows_workspace_bytes(D)});
}

int launch_paged_attention_q8(const void *q, long long q_stride, const kvs_paged_cache_q8 &cache,
                              int dtype, const PagedArgs &pa, void *out, long long out_stride, int H,
                              void *workspace, int *d_status, cudaStream_t stream) {
  const int G = H / cache.num_kv_heads;
  if ((long long)pa.max_new * G > kDRows) {
    if (dtype != KVS_F32)
      return launch_paged_chunk_q8(q, q_stride, cache, dtype, pa, out, out_stride, H, workspace,
                                   d_status, stream);
    // Units of 112 rows share their keys where there are rows for them; below that more of the
    // SM's warps have work in units of 16.  us by units of 112 and of 16, H 14 / 2, D 64 and
    // H 40 / 8, D 128: 4 sequences of up to 3000 keys with 40, 100, 250, 700 new tokens 23.5, 25.8,
    // 30.7, 46.3 (15.4, 22.3, 39.2, 73.6) and 35, 48, 92, 243 (36, 66, 161, 439); 16 of up to
    // 2500 with 100, 250 23.4, 27.3 (21.2, 32.6) and 86, 89 (77, 120); one of 12,000 with 40
    // 29.8 (19.5) and 65 (94).
    if ((long long)pa.num_rows * H >= 1500 && (long long)pa.num_rows * G >= 32ll * pa.M)
      return launch_paged_rows_q8(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status,
                                  stream);
  }
#define KVS_DECODE(T)                                                                           \
  return cache.head_dim == 64                                                                   \
             ? launch_q8<T, 64>(q, q_stride, cache, pa, out, out_stride, H, workspace,          \
                                d_status, stream)                                               \
             : launch_q8<T, 128>(q, q_stride, cache, pa, out, out_stride, H, workspace,         \
                                 d_status, stream)
  if (dtype == KVS_F32) KVS_DECODE(float);
  if (dtype == KVS_F16) KVS_DECODE(__half);
  KVS_DECODE(__nv_bfloat16);
#undef KVS_DECODE
}

}  // namespace kvs
