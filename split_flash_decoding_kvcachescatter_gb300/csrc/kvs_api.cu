// kvs_api.cu -- the C ABI (include/kvsdecode.h): argument validation on the
// host, the chunk-size rule, workspace sizing, and dispatch to the kernel
// launchers.  Nothing here allocates, frees or synchronises.

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "kvs_launch.h"
#include "kvsdecode.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool head_dim_supported(int D) { return D == 64 || D == 128; }

// Shape checks shared by the attention entry points (no pointers).
int check_attention_shape(int M, int H, int Hkv, int D, int max_len, int chunk) {
  if (M < 0 || H < 1 || Hkv < 1 || max_len < 1 || chunk < 0) return KVS_ERR_DIMS;
  if (H % Hkv != 0) return KVS_ERR_DIMS;
  if (!head_dim_supported(D)) return KVS_ERR_UNSUPPORTED;
  if (H / Hkv > 8) return KVS_ERR_UNSUPPORTED;
  if ((int64_t)M * H > 0x7fffffffll) return KVS_ERR_DIMS;
  return KVS_OK;
}

// Kernel schedule (kvs_set_schedule); process-wide.
std::atomic<int> g_schedule{KVS_SCHEDULE_AUTO};

// Wait bound of each device (kvs_set_wait_limit_ns), as last set.
constexpr int kMaxLimitDevices = 64;
std::mutex g_limit_mu;
std::atomic<uint64_t> g_limit[kMaxLimitDevices] = {};
struct LimitInit {
  LimitInit() {
    for (auto &x : g_limit) x.store(KVS_WAIT_LIMIT_DEFAULT_NS);
  }
} g_limit_init;

// Upper bound of the K/V bytes of one step above which the automatic
// schedule never considers the cluster kernel (checked before any device
// query).
constexpr long long kClusterAutoBytes = 64ll << 20;

bool use_cluster(int M, int H, int Hkv, int D, int max_len) {
  const long long pairs = (long long)M * Hkv;
  if (pairs > kvs::kMaxClusterPairs) return false;
  switch (g_schedule.load(std::memory_order_relaxed)) {
    case KVS_SCHEDULE_PERSISTENT: return false;
    case KVS_SCHEDULE_CLUSTER: return true;
    default:
      if (pairs * max_len * D * 8 > kClusterAutoBytes) return false;
      return kvs::cluster_auto_ok(M, H, Hkv, D, max_len) != 0;
  }
}

// The attention launch of kvs_flash_decode (k_rows == nullptr) and
// kvs_decode_step, on the schedule in force.
int launch_attention(const float *q, float *k_cache, float *v_cache, const kvs::SeqArgs &seqs,
                     const float *k_rows, const float *v_rows, float *out, int M, int H, int Hkv,
                     int D, int chunk, void *workspace, int *d_status, cudaStream_t stream) {
  if (use_cluster(M, H, Hkv, D, seqs.max_len))
    return kvs::launch_fd_cluster(q, k_cache, v_cache, seqs, k_rows, v_rows, out, M, H, Hkv, D,
                                  d_status, stream);
  return kvs::launch_fd_step(q, k_cache, v_cache, seqs, k_rows, v_rows, out, M, H, Hkv, D, chunk,
                             workspace, d_status, stream);
}

// chunk_size == 0 -> the library rule on the current device.
int resolve_chunk(int M, int Hkv, int D, int max_len, int chunk) {
  if (chunk > 0) return chunk;
  return kvs_choose_chunk_size(M, Hkv, D, max_len, 0);
}

}  // namespace

bool kvs::poll_waits() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxLimitDevices) {
    cudaGetLastError();
    return false;
  }
  return g_limit[dev].load(std::memory_order_relaxed) < KVS_WAIT_LIMIT_DEFAULT_NS;
}

extern "C" {

const char *kvs_strerror(int status) {
  switch (status) {
    case KVS_OK: return "ok";
    case KVS_ERR_NULL: return "a required pointer is NULL";
    case KVS_ERR_DIMS: return "invalid dimensions";
    case KVS_ERR_UNSUPPORTED: return "unsupported head_dim or query-head group";
    case KVS_ERR_ALIGN: return "pointer not aligned (16 bytes for tensors, 256 for workspace)";
    case KVS_ERR_WORKSPACE: return "workspace missing or too small";
    case KVS_ERR_LAUNCH: return "CUDA launch or device query failed";
    case KVS_ERR_POSITION: return "a position is outside [0, max_len)";
    case KVS_ERR_TIMEOUT: return "a bounded device pipeline wait expired";
    case KVS_ERR_SLOT: return "a cache slot is outside [0, num_slots)";
    case KVS_ERR_MEMORY: return "the device could not provide the library's own buffer";
    case KVS_ERR_PAGE: return "a page or mask number is out of range";
    case KVS_ERR_ROWS: return "row offsets decrease or leave their list";
    case KVS_ERR_OVERLAP: return "an output overlaps an input";
    default: return "unknown kvs status";
  }
}

int kvs_kv_scatter(const float *k_rows, const float *v_rows, const int32_t *positions,
                   float *k_cache, float *v_cache, int M, int num_kv_heads, int head_dim,
                   int max_len, int *d_status, kvs_stream_t stream) {
  if (M < 0 || num_kv_heads < 1 || max_len < 1) return KVS_ERR_DIMS;
  if (!head_dim_supported(head_dim)) return KVS_ERR_UNSUPPORTED;
  if (M == 0) return KVS_OK;
  if (!k_rows || !v_rows || !positions || !k_cache || !v_cache) return KVS_ERR_NULL;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(positions, 4))
    return KVS_ERR_ALIGN;
  return kvs::launch_kv_scatter(k_rows, v_rows, positions, k_cache, v_cache, M, num_kv_heads,
                                head_dim, max_len, d_status,
                                reinterpret_cast<cudaStream_t>(stream));
}

int kvs_choose_chunk_size(int M, int num_kv_heads, int head_dim, int max_len, int num_sms) {
  if (M < 1 || num_kv_heads < 1 || max_len < 1) return -KVS_ERR_DIMS;
  if (!head_dim_supported(head_dim)) return -KVS_ERR_UNSUPPORTED;
  const int sms = num_sms > 0 ? num_sms : kvs::device_sm_count();
  if (sms <= 0) return -KVS_ERR_LAUNCH;
  // Chunks are the scheduling atoms of the persistent chunk kernel: a block's
  // range starts and ends on chunk boundaries, so the chunk size is the
  // granularity of the load balance (a block holds its 1/P share of the live
  // rows to within one chunk).  Partials are kept per run of chunks, so small
  // chunks cost no extra partial traffic.  Aim for about 1/128 of a block's
  // share of a full cache, as a power of two in [16, 64].
  const int64_t blocks = 2ll * sms;
  const int64_t share = (int64_t)M * num_kv_heads * max_len / blocks;
  int c = 16;
  while (c < 64 && 2ll * c * 128 <= share) c <<= 1;
  return c;
}

size_t kvs_flash_decode_workspace_bytes(int M, int num_heads, int num_kv_heads, int head_dim,
                                        int max_len, int chunk_size) {
  if (check_attention_shape(M, num_heads, num_kv_heads, head_dim, max_len, chunk_size) != KVS_OK)
    return 0;
  if (M == 0) return 0;
  // The partials are kept per run of chunks (see kvs_launch.h), so the size
  // depends on neither max_len nor the chunk size.
  return kvs::ws_layout(M, num_kv_heads, num_heads / num_kv_heads, head_dim).total;
}

// Pointer and workspace checks shared by the attention entry points.
static int check_attention_buffers(const float *q, const float *k_cache, const float *v_cache,
                                   const int32_t *positions, const float *out, int M,
                                   int num_heads, int num_kv_heads, int head_dim,
                                   const void *workspace, size_t workspace_bytes) {
  if (!q || !k_cache || !v_cache || !positions || !out) return KVS_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(positions, 4))
    return KVS_ERR_ALIGN;
  if (!workspace) return KVS_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KVS_ERR_ALIGN;
  if (workspace_bytes < kvs::ws_layout(M, num_kv_heads, num_heads / num_kv_heads, head_dim).total)
    return KVS_ERR_WORKSPACE;
  return KVS_OK;
}

int kvs_flash_decode(const float *q, const float *k_cache, const float *v_cache,
                     const int32_t *positions, float *out, int M, int num_heads,
                     int num_kv_heads, int head_dim, int max_len, int chunk_size,
                     void *workspace, size_t workspace_bytes, int *d_status,
                     kvs_stream_t stream) {
  int rc = check_attention_shape(M, num_heads, num_kv_heads, head_dim, max_len, chunk_size);
  if (rc != KVS_OK) return rc;
  if (M == 0) return KVS_OK;
  rc = check_attention_buffers(q, k_cache, v_cache, positions, out, M, num_heads, num_kv_heads,
                               head_dim, workspace, workspace_bytes);
  if (rc != KVS_OK) return rc;
  const int chunk = resolve_chunk(M, num_kv_heads, head_dim, max_len, chunk_size);
  if (chunk <= 0) return -chunk;
  // the caches are only read when no new rows are passed
  const kvs::SeqArgs seqs{positions, nullptr, nullptr, max_len, M};
  return launch_attention(q, const_cast<float *>(k_cache), const_cast<float *>(v_cache), seqs,
                          nullptr, nullptr, out, M, num_heads, num_kv_heads, head_dim, chunk,
                          workspace, d_status, reinterpret_cast<cudaStream_t>(stream));
}

int kvs_decode_step(const float *q, const float *k_rows, const float *v_rows,
                    const int32_t *positions, float *k_cache, float *v_cache, float *out, int M,
                    int num_heads, int num_kv_heads, int head_dim, int max_len, int chunk_size,
                    void *workspace, size_t workspace_bytes, int *d_status,
                    kvs_stream_t stream) {
  return kvs::decode_step(q, k_rows, v_rows, positions, k_cache, v_cache, out, M, num_heads,
                          num_kv_heads, head_dim, max_len, chunk_size, workspace,
                          workspace_bytes, d_status, stream, false);
}

}  // extern "C"

int kvs::decode_step(const float *q, const float *k_rows, const float *v_rows,
                     const int32_t *positions, float *k_cache, float *v_cache, float *out, int M,
                     int num_heads, int num_kv_heads, int head_dim, int max_len, int chunk_size,
                     void *workspace, size_t workspace_bytes, int *d_status,
                     kvs_stream_t stream, bool early) {
  int rc = check_attention_shape(M, num_heads, num_kv_heads, head_dim, max_len, chunk_size);
  if (rc != KVS_OK) return rc;
  if (M == 0) return KVS_OK;
  if (!k_rows || !v_rows) return KVS_ERR_NULL;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16)) return KVS_ERR_ALIGN;
  rc = check_attention_buffers(q, k_cache, v_cache, positions, out, M, num_heads, num_kv_heads,
                               head_dim, workspace, workspace_bytes);
  if (rc != KVS_OK) return rc;
  const int chunk = resolve_chunk(M, num_kv_heads, head_dim, max_len, chunk_size);
  if (chunk <= 0) return -chunk;
  kvs::SeqArgs seqs{positions, nullptr, nullptr, max_len, M};
  seqs.early = early;
  return launch_attention(q, k_cache, v_cache, seqs, k_rows, v_rows, out, M, num_heads,
                          num_kv_heads, head_dim, chunk, workspace, d_status,
                          reinterpret_cast<cudaStream_t>(stream));
}

extern "C" {

namespace {

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Offsets of the device copies in the io buffer of kvs_decode_step_host:
// q, k_rows, v_rows, positions, out, each 256-byte aligned.
struct IoLayout {
  size_t q, k, v, pos, out, total;
};

IoLayout io_layout(int M, int num_heads, int num_kv_heads, int head_dim) {
  const size_t qo = (size_t)M * num_heads * head_dim * sizeof(float);
  const size_t kv = (size_t)M * num_kv_heads * head_dim * sizeof(float);
  IoLayout L;
  L.q = 0;
  L.k = L.q + round256(qo);
  L.v = L.k + round256(kv);
  L.pos = L.v + round256(kv);
  L.out = L.pos + round256((size_t)M * sizeof(int32_t));
  L.total = L.out + round256(qo);
  return L;
}

}  // namespace

size_t kvs_step_io_bytes(int M, int num_heads, int num_kv_heads, int head_dim) {
  if (M < 1 || num_heads < 1 || num_kv_heads < 1 || head_dim < 1) return 0;
  return io_layout(M, num_heads, num_kv_heads, head_dim).total;
}

int kvs_decode_step_host(const float *q, const float *k_rows, const float *v_rows,
                         const int32_t *positions, float *k_cache, float *v_cache, float *out,
                         int M, int num_heads, int num_kv_heads, int head_dim, int max_len,
                         int chunk_size, void *io, size_t io_bytes, void *workspace,
                         size_t workspace_bytes, int *d_status, kvs_stream_t stream) {
  int rc = check_attention_shape(M, num_heads, num_kv_heads, head_dim, max_len, chunk_size);
  if (rc != KVS_OK) return rc;
  if (M == 0) return KVS_OK;
  if (!q || !k_rows || !v_rows || !positions || !out || !io) return KVS_ERR_NULL;
  if (!aligned(io, 256)) return KVS_ERR_ALIGN;
  const IoLayout L = io_layout(M, num_heads, num_kv_heads, head_dim);
  if (io_bytes < L.total) return KVS_ERR_WORKSPACE;
  unsigned char *base = static_cast<unsigned char *>(io);
  float *dq = reinterpret_cast<float *>(base + L.q);
  float *dk = reinterpret_cast<float *>(base + L.k);
  float *dv = reinterpret_cast<float *>(base + L.v);
  int32_t *dpos = reinterpret_cast<int32_t *>(base + L.pos);
  float *dout = reinterpret_cast<float *>(base + L.out);
  rc = check_attention_buffers(dq, k_cache, v_cache, dpos, dout, M, num_heads, num_kv_heads,
                               head_dim, workspace, workspace_bytes);
  if (rc != KVS_OK) return rc;
  const int chunk = resolve_chunk(M, num_kv_heads, head_dim, max_len, chunk_size);
  if (chunk <= 0) return -chunk;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t qo = (size_t)M * num_heads * head_dim * sizeof(float);
  const size_t kv = (size_t)M * num_kv_heads * head_dim * sizeof(float);
  if (cudaMemcpyAsync(dpos, positions, (size_t)M * sizeof(int32_t), cudaMemcpyHostToDevice,
                      st) != cudaSuccess ||
      cudaMemcpyAsync(dq, q, qo, cudaMemcpyHostToDevice, st) != cudaSuccess ||
      cudaMemcpyAsync(dk, k_rows, kv, cudaMemcpyHostToDevice, st) != cudaSuccess ||
      cudaMemcpyAsync(dv, v_rows, kv, cudaMemcpyHostToDevice, st) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  const kvs::SeqArgs seqs{dpos, nullptr, nullptr, max_len, M};
  rc = launch_attention(dq, k_cache, v_cache, seqs, dk, dv, dout, M, num_heads, num_kv_heads,
                        head_dim, chunk, workspace, d_status, st);
  if (rc != KVS_OK) return rc;
  if (cudaMemcpyAsync(out, dout, qo, cudaMemcpyDeviceToHost, st) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

int kvs_step_io_layout(int M, int num_heads, int num_kv_heads, int head_dim, size_t *offsets) {
  if (M < 1 || num_heads < 1 || num_kv_heads < 1 || head_dim < 1) return KVS_ERR_DIMS;
  if (!offsets) return KVS_ERR_NULL;
  const IoLayout L = io_layout(M, num_heads, num_kv_heads, head_dim);
  offsets[0] = L.q;
  offsets[1] = L.k;
  offsets[2] = L.v;
  offsets[3] = L.pos;
  offsets[4] = L.out;
  offsets[5] = L.total;
  return KVS_OK;
}

int kvs_decode_step_host_io(void *host_io, float *k_cache, float *v_cache, int M, int num_heads,
                            int num_kv_heads, int head_dim, int max_len, int chunk_size, void *io,
                            size_t io_bytes, void *workspace, size_t workspace_bytes,
                            int *d_status, kvs_stream_t stream) {
  int rc = check_attention_shape(M, num_heads, num_kv_heads, head_dim, max_len, chunk_size);
  if (rc != KVS_OK) return rc;
  if (M == 0) return KVS_OK;
  if (!host_io || !io) return KVS_ERR_NULL;
  if (!aligned(io, 256)) return KVS_ERR_ALIGN;
  const IoLayout L = io_layout(M, num_heads, num_kv_heads, head_dim);
  if (io_bytes < L.total) return KVS_ERR_WORKSPACE;
  unsigned char *base = static_cast<unsigned char *>(io);
  float *dq = reinterpret_cast<float *>(base + L.q);
  float *dk = reinterpret_cast<float *>(base + L.k);
  float *dv = reinterpret_cast<float *>(base + L.v);
  int32_t *dpos = reinterpret_cast<int32_t *>(base + L.pos);
  float *dout = reinterpret_cast<float *>(base + L.out);
  rc = check_attention_buffers(dq, k_cache, v_cache, dpos, dout, M, num_heads, num_kv_heads,
                               head_dim, workspace, workspace_bytes);
  if (rc != KVS_OK) return rc;
  const int chunk = resolve_chunk(M, num_kv_heads, head_dim, max_len, chunk_size);
  if (chunk <= 0) return -chunk;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t qo = (size_t)M * num_heads * head_dim * sizeof(float);
  unsigned char *host = static_cast<unsigned char *>(host_io);
  // the inputs (q, k_rows, v_rows, positions and the padding between them)
  // in one copy
  const size_t in_bytes = L.pos + (size_t)M * sizeof(int32_t);
  // Pinned host memory the GPU can address is moved by the library's copy
  // kernel; any other host memory by a copy engine.
  cudaPointerAttributes pa;
  unsigned char *mapped = nullptr;
  if (cudaPointerGetAttributes(&pa, host_io) == cudaSuccess && pa.type == cudaMemoryTypeHost &&
      pa.devicePointer != nullptr && aligned(pa.devicePointer, 16))
    mapped = static_cast<unsigned char *>(pa.devicePointer);
  else
    cudaGetLastError();
  if (mapped) {
    rc = kvs::launch_io_copy(mapped, base, in_bytes, st);
    if (rc != KVS_OK) return rc;
  } else if (cudaMemcpyAsync(base, host, in_bytes, cudaMemcpyHostToDevice, st) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  const kvs::SeqArgs seqs{dpos, nullptr, nullptr, max_len, M};
  rc = launch_attention(dq, k_cache, v_cache, seqs, dk, dv, dout, M, num_heads, num_kv_heads,
                        head_dim, chunk, workspace, d_status, st);
  if (rc != KVS_OK) return rc;
  if (mapped) return kvs::launch_io_copy(dout, mapped + L.out, qo, st);
  if (cudaMemcpyAsync(host + L.out, dout, qo, cudaMemcpyDeviceToHost, st) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

int kvs_decode_step_slots(const float *q, const float *k_rows, const float *v_rows,
                          const int32_t *positions, const int32_t *slots, const uint8_t *done,
                          float *k_pool, float *v_pool, int num_slots, float *out, int M,
                          int num_heads, int num_kv_heads, int head_dim, int max_len,
                          int chunk_size, void *workspace, size_t workspace_bytes,
                          int *d_status, kvs_stream_t stream) {
  int rc = check_attention_shape(M, num_heads, num_kv_heads, head_dim, max_len, chunk_size);
  if (rc != KVS_OK) return rc;
  if (num_slots < 1 || (!slots && num_slots < M)) return KVS_ERR_DIMS;
  if (M == 0) return KVS_OK;
  if ((k_rows == nullptr) != (v_rows == nullptr)) return KVS_ERR_NULL;
  if (k_rows && (!aligned(k_rows, 16) || !aligned(v_rows, 16))) return KVS_ERR_ALIGN;
  if (slots && !aligned(slots, 4)) return KVS_ERR_ALIGN;
  rc = check_attention_buffers(q, k_pool, v_pool, positions, out, M, num_heads, num_kv_heads,
                               head_dim, workspace, workspace_bytes);
  if (rc != KVS_OK) return rc;
  const int chunk = resolve_chunk(M, num_kv_heads, head_dim, max_len, chunk_size);
  if (chunk <= 0) return -chunk;
  const kvs::SeqArgs seqs{positions, slots, done, max_len, num_slots};
  return launch_attention(q, k_pool, v_pool, seqs, k_rows, v_rows, out, M, num_heads,
                          num_kv_heads, head_dim, chunk, workspace, d_status,
                          reinterpret_cast<cudaStream_t>(stream));
}

int kvs_argmax(const float *logits, int M, int vocab_size, int32_t *token_ids,
               kvs_stream_t stream) {
  if (M < 0 || vocab_size < 1) return KVS_ERR_DIMS;
  if (M == 0) return KVS_OK;
  if (!logits || !token_ids) return KVS_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(token_ids, 4)) return KVS_ERR_ALIGN;
  return kvs::launch_argmax(logits, M, vocab_size, token_ids,
                            reinterpret_cast<cudaStream_t>(stream));
}

size_t kvs_prefill_workspace_bytes(int num_heads, int seq_len, int head_dim) {
  if (num_heads < 1 || seq_len < 1 || num_heads > 65535 || (int64_t)seq_len > 65535ll * 128 ||
      !head_dim_supported(head_dim))
    return 0;
  return kvs::prefill_workspace_bytes(num_heads, seq_len, head_dim);
}

int kvs_prefill_attention(const float *q, const float *k, const float *v, float *out,
                          int num_heads, int seq_len, int head_dim, int causal, void *workspace,
                          size_t workspace_bytes, int *d_status, kvs_stream_t stream) {
  if (num_heads < 0 || seq_len < 0) return KVS_ERR_DIMS;
  if (!head_dim_supported(head_dim)) return KVS_ERR_UNSUPPORTED;
  if ((int64_t)num_heads > 65535 || (int64_t)seq_len > 65535ll * 128) return KVS_ERR_DIMS;
  if (num_heads == 0 || seq_len == 0) return KVS_OK;
  if (!q || !k || !v || !out) return KVS_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return KVS_ERR_ALIGN;
  if (!workspace) return KVS_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KVS_ERR_ALIGN;
  if (workspace_bytes < kvs::prefill_workspace_bytes(num_heads, seq_len, head_dim))
    return KVS_ERR_WORKSPACE;
  return kvs::launch_prefill(q, k, v, out, num_heads, seq_len, head_dim, causal ? 1 : 0,
                             workspace, d_status, reinterpret_cast<cudaStream_t>(stream));
}

// Shape checks of a paged cache and batch (no device memory is looked at).
static int check_paged(const kvs_paged_cache *cache, const kvs_paged_batch *batch, int num_heads) {
  if (!cache || !batch) return KVS_ERR_NULL;
  const int Hkv = cache->num_kv_heads;
  if (cache->num_pages < 1 || cache->page_size < 1 || Hkv < 1 || num_heads < 1 ||
      num_heads % Hkv != 0 || batch->num_seqs < 0 || batch->num_rows < 0 || batch->max_new < 1 ||
      batch->max_pages < 1)
    return KVS_ERR_DIMS;
  if (cache->dtype != KVS_F32 && cache->dtype != KVS_F16 && cache->dtype != KVS_BF16)
    return KVS_ERR_UNSUPPORTED;
  if (!head_dim_supported(cache->head_dim) || num_heads / Hkv > 8 || num_heads > 4096)
    return KVS_ERR_UNSUPPORTED;
  if (cache->page_size < 16 || (cache->page_size & (cache->page_size - 1)) != 0)
    return KVS_ERR_UNSUPPORTED;
  // (a block walks the sequences one after the other, empty ones too: 2^20 of them in about half a
  // second, within its waits' bound)
  if (batch->num_seqs > (1 << 20)) return KVS_ERR_UNSUPPORTED;
  // rows of the pages and of one sequence are counted in 32 bits
  if ((int64_t)cache->num_pages * Hkv > 0x7fffffffll / cache->page_size ||
      (int64_t)batch->max_pages > 0x7fffffffll / cache->page_size)
    return KVS_ERR_DIMS;
  return KVS_OK;
}

// Pointers of a paged cache and batch with work in it.
static int check_paged_pointers(const kvs_paged_cache *cache, const kvs_paged_batch *batch) {
  if (!cache->k_pages || !cache->v_pages || !batch->positions || !batch->row_offsets ||
      !batch->page_table)
    return KVS_ERR_NULL;
  if (!aligned(cache->k_pages, 16) || !aligned(cache->v_pages, 16) ||
      !aligned(batch->positions, 4) || !aligned(batch->row_offsets, 4) ||
      !aligned(batch->page_table, 4))
    return KVS_ERR_ALIGN;
  return KVS_OK;
}

// Rows of `row` elements of `dtype`, `stride` elements apart.
static int check_rows(const void *p, int64_t stride, int64_t row, int dtype) {
  if (!p) return KVS_ERR_NULL;
  if (stride < row) return KVS_ERR_DIMS;
  if (!aligned(p, 16) || stride * (dtype == KVS_F32 ? 4 : 2) % 16 != 0) return KVS_ERR_ALIGN;
  return KVS_OK;
}

// `n` rows of `len` bytes, `stride` bytes apart (stride >= len).
struct RowSpan {
  uintptr_t at;
  int64_t stride, len;
};
static RowSpan row_span(const void *p, int64_t stride, int64_t row, int dtype) {
  const int64_t size = dtype == KVS_F32 ? 4 : 2;
  return RowSpan{reinterpret_cast<uintptr_t>(p), stride * size, row * size};
}

// Whether some row of a shares a byte with some row of b, n rows each.  Blocks
// of columns of one matrix do not, although their spans lie in each other.
static bool rows_overlap(const RowSpan &a, const RowSpan &b, int64_t n) {
  const int64_t d = (int64_t)(b.at - a.at);  // row j of b starts d + j b.stride behind a
  if (d >= (n - 1) * a.stride + a.len || -d >= (n - 1) * b.stride + b.len) return false;
  auto div_up = [](int64_t x, int64_t y) { return x > 0 ? (x + y - 1) / y : -(-x / y); };
  if (a.stride == b.stride || n == 1) {
    // rows i and i + k: apart unless -b.len < d + k stride < a.len
    const int64_t k = std::max(div_up(1 - b.len - d, a.stride), 1 - n);
    return k < n && d + k * a.stride < a.len;
  }
  for (int64_t i = 0; i < n; ++i) {
    const int64_t j = std::max<int64_t>(div_up(i * a.stride + 1 - b.len - d, b.stride), 0);
    if (j < n && d + j * b.stride < i * a.stride + a.len) return true;
  }
  return false;
}
// The same rows: an operator that may work in place does.
static bool same_rows(const RowSpan &a, const RowSpan &b, int64_t n) {
  return a.at == b.at && (a.stride == b.stride || n == 1);
}

static kvs::PagedArgs paged_args(const kvs_paged_cache *cache, const kvs_paged_batch *batch) {
  int shift = 0;
  while ((1 << shift) < cache->page_size) ++shift;
  return kvs::PagedArgs{batch->positions, batch->row_offsets, batch->page_table,
                        batch->num_seqs,  batch->num_rows,    batch->max_new,
                        batch->max_pages, shift,              cache->num_pages};
}

int kvs_rope_scatter_paged(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                           const void *v, int64_t v_stride, void *q_out, int64_t q_out_stride,
                           const kvs_paged_cache *cache, const kvs_paged_batch *batch,
                           const float *inv_freq, int num_heads, int rot_dim, int interleaved,
                           float scale, int *d_status, kvs_stream_t stream) {
  int rc = check_paged(cache, batch, num_heads);
  if (rc != KVS_OK) return rc;
  const int D = cache->head_dim, Hkv = cache->num_kv_heads, dtype = cache->dtype;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0) return KVS_ERR_DIMS;
  if (batch->num_seqs == 0 || batch->num_rows == 0) return KVS_OK;
  rc = check_paged_pointers(cache, batch);
  if (rc == KVS_OK) rc = check_rows(q, q_stride, (int64_t)num_heads * D, dtype);
  if (rc == KVS_OK) rc = check_rows(k, k_stride, (int64_t)Hkv * D, dtype);
  if (rc == KVS_OK) rc = check_rows(v, v_stride, (int64_t)Hkv * D, dtype);
  if (rc == KVS_OK) rc = check_rows(q_out, q_out_stride, (int64_t)num_heads * D, dtype);
  if (rc != KVS_OK) return rc;
  if (rot_dim > 0 && !inv_freq) return KVS_ERR_NULL;
  if (!aligned(inv_freq, 4)) return KVS_ERR_ALIGN;
  const int64_t n = batch->num_rows;
  const RowSpan to = row_span(q_out, q_out_stride, (int64_t)num_heads * D, dtype);
  const RowSpan from = row_span(q, q_stride, (int64_t)num_heads * D, dtype);
  if ((!same_rows(from, to, n) && rows_overlap(from, to, n)) ||
      rows_overlap(row_span(k, k_stride, (int64_t)Hkv * D, dtype), to, n) ||
      rows_overlap(row_span(v, v_stride, (int64_t)Hkv * D, dtype), to, n))
    return KVS_ERR_OVERLAP;
  return kvs::launch_rope_scatter(q, q_stride, k, k_stride, v, v_stride, q_out, q_out_stride,
                                  cache->k_pages, cache->v_pages, paged_args(cache, batch),
                                  inv_freq, num_heads, Hkv, D, dtype, rot_dim, interleaved ? 1 : 0,
                                  scale, d_status, reinterpret_cast<cudaStream_t>(stream));
}

int kvs_rope_frequencies(int rot_dim, double base, int kind, double factor, double original_len,
                         double slow, double fast, float *inv_freq, float *scale) {
  const bool ramp = kind == KVS_ROPE_YARN || kind == KVS_ROPE_BANDS;
  if (rot_dim < 2 || rot_dim % 2 != 0 || kind < KVS_ROPE_PLAIN || kind > KVS_ROPE_BANDS ||
      !(base > 0.0) || (kind != KVS_ROPE_PLAIN && !(factor >= 1.0)) ||
      (ramp && (!(original_len > 0.0) || !(slow > 0.0) || !(fast > slow))) ||
      (kind == KVS_ROPE_NTK && rot_dim < 4) || (kind == KVS_ROPE_YARN && !(base > 1.0)) ||
      !std::isfinite(base) || (kind != KVS_ROPE_PLAIN && !std::isfinite(factor)) ||
      (ramp && (!std::isfinite(original_len) || !std::isfinite(fast))))
    return KVS_ERR_DIMS;
  if (!inv_freq) return KVS_ERR_NULL;
  const double two_pi = 6.28318530717958647693;
  if (kind == KVS_ROPE_NTK) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  // YARN's ramp runs over the pair index, from the (fractional) pair that
  // turns `fast` times over original_len positions to the one that turns
  // `slow` times, both rounded outwards and kept inside the head
  auto pair_of = [&](double turns) {
    return rot_dim * std::log(original_len / (turns * two_pi)) / (2.0 * std::log(base));
  };
  double first = 0.0, last = 0.0;
  bool none = false;  // not even pair 0 turns `slow` times
  if (kind == KVS_ROPE_YARN) {
    none = pair_of(slow) < 0.0;
    first = std::max(0.0, std::floor(pair_of(fast)));
    last = std::min(rot_dim - 1.0, std::ceil(pair_of(slow)));
    if (last <= first) last = first + 0.001;
  }
  // (the largest entry is the first, or with a base below 1 the last)
  const double fastest = std::max(1.0, std::pow(base, 2.0 / rot_dim - 1.0));
  if (!(fastest <= 1e6)) return KVS_ERR_DIMS;
  for (int j = 0; j < rot_dim / 2; ++j) {
    double w = std::pow(base, -2.0 * j / rot_dim);
    double keep = 1.0;  // share of w kept, the rest is w / factor
    if (kind == KVS_ROPE_LINEAR) keep = 0.0;
    if (kind == KVS_ROPE_YARN)
      keep = none ? 0.0 : 1.0 - std::min(1.0, std::max(0.0, (j - first) / (last - first)));
    if (kind == KVS_ROPE_BANDS)
      keep = std::min(1.0, std::max(0.0, (original_len * w / two_pi - slow) / (fast - slow)));
    if (kind == KVS_ROPE_LINEAR || ramp) w = keep * w + (1.0 - keep) * w / factor;
    inv_freq[j] = (float)w;
  }
  if (scale) *scale = kind == KVS_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return KVS_OK;
}

size_t kvs_paged_attention_workspace_bytes(int num_heads, int num_kv_heads, int head_dim,
                                           int max_new) {
  if (num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 || max_new < 1 ||
      !head_dim_supported(head_dim) || num_heads / num_kv_heads > 8)
    return 0;
  return kvs::paged_attention_workspace_bytes(num_heads, num_kv_heads, head_dim, max_new);
}

int kvs_paged_attention(const void *q, int64_t q_stride, const kvs_paged_cache *cache,
                        const kvs_paged_batch *batch, void *out, int64_t out_stride,
                        int num_heads, void *workspace, size_t workspace_bytes, int *d_status,
                        kvs_stream_t stream) {
  int rc = check_paged(cache, batch, num_heads);
  if (rc != KVS_OK) return rc;
  // The kernels count a sequence's keys and what they look ahead (a tile, a
  // unit's fixed price, 32 tiles of pages: all under 2048 keys) in 32 bits.
  if ((int64_t)batch->max_pages * cache->page_size > KVS_PAGED_MAX_KEYS) return KVS_ERR_DIMS;
  if (batch->num_seqs == 0 || batch->num_rows == 0) return KVS_OK;
  const int D = cache->head_dim;
  rc = check_paged_pointers(cache, batch);
  if (rc == KVS_OK) rc = check_rows(q, q_stride, (int64_t)num_heads * D, cache->dtype);
  if (rc == KVS_OK) rc = check_rows(out, out_stride, (int64_t)num_heads * D, cache->dtype);
  if (rc != KVS_OK) return rc;
  if (!workspace) return KVS_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KVS_ERR_ALIGN;
  if (workspace_bytes < kvs::paged_attention_workspace_bytes(num_heads, cache->num_kv_heads, D,
                                                             batch->max_new))
    return KVS_ERR_WORKSPACE;
  if (rows_overlap(row_span(q, q_stride, (int64_t)num_heads * D, cache->dtype),
                   row_span(out, out_stride, (int64_t)num_heads * D, cache->dtype),
                   batch->num_rows))
    return KVS_ERR_OVERLAP;
  return kvs::launch_paged_attention(q, q_stride, *cache, paged_args(cache, batch), out,
                                     out_stride, num_heads, workspace, d_status,
                                     reinterpret_cast<cudaStream_t>(stream));
}

int kvs_process_logits(const void *logits, int64_t logits_stride, void *out, int64_t out_stride,
                       int dtype, int M, int vocab_size, const kvs_logit_rules *rules,
                       int32_t *token_ids, int *d_status, kvs_stream_t stream) {
  if (M < 0 || vocab_size < 1) return KVS_ERR_DIMS;
  if (dtype != KVS_F32 && dtype != KVS_F16 && dtype != KVS_BF16) return KVS_ERR_UNSUPPORTED;
  if (vocab_size > (1 << 19)) return KVS_ERR_UNSUPPORTED;
  if (M > (1 << 30)) return KVS_ERR_UNSUPPORTED;  // (the kernel steps past M by a grid's rows)
  if (M == 0) return KVS_OK;
  if (!logits || !rules || (!out && !token_ids)) return KVS_ERR_NULL;
  if (logits_stride < vocab_size || (out && out_stride < vocab_size)) return KVS_ERR_DIMS;
  const uintptr_t size = dtype == KVS_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(out, size) || !aligned(token_ids, 4)) return KVS_ERR_ALIGN;
  const kvs_logit_rules &r = *rules;
  if (r.history && !r.history_offsets) return KVS_ERR_NULL;
  if (r.bias_ids && (!r.bias_values || !r.bias_offsets)) return KVS_ERR_NULL;
  if (r.history_len < 0 || r.history_len > (1 << 29) || r.bias_len < 0 ||
      r.bias_len > (1 << 29) ||
      (r.mask && r.mask_count < (r.mask_rows ? 1 : M)))
    return KVS_ERR_DIMS;
  for (const void *p : {(const void *)r.history, (const void *)r.history_offsets,
                        (const void *)r.prompt_lens, (const void *)r.repetition,
                        (const void *)r.presence, (const void *)r.frequency,
                        (const void *)r.bias_ids, (const void *)r.bias_values,
                        (const void *)r.bias_offsets, (const void *)r.mask,
                        (const void *)r.mask_rows})
    if (!aligned(p, 4)) return KVS_ERR_ALIGN;
  if (out) {
    const RowSpan from = row_span(logits, logits_stride, vocab_size, dtype);
    const RowSpan to = row_span(out, out_stride, vocab_size, dtype);
    if (!same_rows(from, to, M) && rows_overlap(from, to, M)) return KVS_ERR_OVERLAP;
  }
  return kvs::launch_logits(logits, logits_stride, out, out_stride, dtype, M, vocab_size, r,
                            token_ids, d_status, reinterpret_cast<cudaStream_t>(stream));
}

int kvs_set_schedule(int schedule) {
  if (schedule != KVS_SCHEDULE_AUTO && schedule != KVS_SCHEDULE_PERSISTENT &&
      schedule != KVS_SCHEDULE_CLUSTER)
    return -KVS_ERR_DIMS;
  return g_schedule.exchange(schedule);
}

int kvs_get_schedule(void) { return g_schedule.load(); }

int kvs_set_wait_limit_ns(uint64_t ns, uint64_t *previous) {
  if (ns > KVS_WAIT_LIMIT_DEFAULT_NS) return KVS_ERR_DIMS;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxLimitDevices) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  std::lock_guard<std::mutex> lk(g_limit_mu);
  int rc = kvs::set_wait_limit_step(ns);
  if (rc == KVS_OK) rc = kvs::set_wait_limit_cluster(ns);
  if (rc == KVS_OK) rc = kvs::set_wait_limit_prefill(ns);
  if (rc == KVS_OK) rc = kvs::set_wait_limit_paged(ns);
  if (rc == KVS_OK) rc = kvs::set_wait_limit_decode(ns);
  if (rc == KVS_OK) rc = kvs::set_wait_limit_chunk(ns);
  if (rc != KVS_OK) return rc;
  if (previous) *previous = g_limit[dev].load();
  g_limit[dev].store(ns);
  return KVS_OK;
}

int kvs_schedule_for(int M, int num_heads, int num_kv_heads, int head_dim, int max_len) {
  const int rc = check_attention_shape(M, num_heads, num_kv_heads, head_dim, max_len, 0);
  if (rc != KVS_OK) return -rc;
  if (M < 1) return -KVS_ERR_DIMS;
  return use_cluster(M, num_heads, num_kv_heads, head_dim, max_len) ? KVS_SCHEDULE_CLUSTER
                                                                    : KVS_SCHEDULE_PERSISTENT;
}

int kvs_prepare(int num_heads, int num_kv_heads, int head_dim) {
  if (num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0) return KVS_ERR_DIMS;
  if (!head_dim_supported(head_dim)) return KVS_ERR_UNSUPPORTED;
  if (num_heads / num_kv_heads > 8) return KVS_ERR_UNSUPPORTED;
  const int rc = kvs::prepare_step_kernel(num_heads, num_kv_heads, head_dim);
  if (rc != KVS_OK) return rc;
  return kvs::prepare_cluster_kernel(num_heads, num_kv_heads, head_dim);
}

}  // extern "C"
