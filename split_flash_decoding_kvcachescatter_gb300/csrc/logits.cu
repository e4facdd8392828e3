// logits.cu -- penalties for repeated tokens, biases and a grammar mask on
// each of M logit rows, and the greedy token of the result, in one launch.
//
// Bound: bytes (a row is read once and written once).  What stands in the
// way is the history: a token's count decides what happens to its logit, and
// the counts of a row are needed before its first logit is final.  One
// thread-block cluster takes a row; block r owns an equal slice of the
// vocabulary and keeps one 32-bit word a token in shared memory (how often
// generated, whether seen, whether biased).  The blocks share the row's
// history: each reads its part of the list once and adds every token to the
// word in its owner's shared memory (distributed shared memory atomics, the
// equal tokens of a warp combined first, since histories repeat a few tokens
// often).  After one cluster barrier each block streams its slice with
// 16-byte loads and stores, and the (value, index) maxima meet as in the
// batched argmax.  Integer atomics only: the result does not depend on their
// order.
//
// Arithmetic is one IEEE operation at a time (no fused multiply-add), so a
// logit is the same whichever variant or alignment handles it.

#include <mutex>

#include "kvs_paged.cuh"

namespace kvs {

namespace {

constexpr int kLogitThreads = 512;
constexpr int kLogitMaxDevices = 64;
constexpr unsigned kSeen = 1u << 31;    // in the prompt (generated tokens have a count)
constexpr unsigned kBiased = 1u << 30;  // in the bias list
constexpr unsigned kCount = kBiased - 1;

struct LogitArgs {
  const void *logits;
  void *out;
  long long logits_stride, out_stride;
  int M, V, slice;
  kvs_logit_rules r;
  int32_t *ids;
  int *d_status;
};

__device__ __forceinline__ void red_add_cluster(uint32_t addr, unsigned v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v)
               : "memory");
}
__device__ __forceinline__ void red_or_cluster(uint32_t addr, unsigned v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v)
               : "memory");
}

// [lo, hi) of row m in a ragged list, or an empty range when the offsets are
// bad (`report`: this thread records that).
__device__ __forceinline__ int2 list_range(const int32_t *offsets, int m, int len, bool report,
                                           int *d_status) {
  const int a = __ldca(offsets + m), e = __ldca(offsets + m + 1);
  if (a < 0 || e < a || e > len) {
    if (report) record_status(d_status, KVS_ERR_ROWS);
    return make_int2(0, 0);
  }
  return make_int2(a, e);
}

struct RowRules {
  float rep, pres, freq;
  const uint32_t *mask;  // this row's words, or nullptr
  int2 bias;
};

// One logit: the rules in their order.  `w` is the token's word.
__device__ __forceinline__ float apply_rules(float x, unsigned w, int id, const RowRules &rr,
                                             const kvs_logit_rules &r) {
  if (w != 0u) {
    const unsigned c = w & kCount;
    if ((w & kSeen) || c) x = x > 0.f ? __fdiv_rn(x, rr.rep) : __fmul_rn(x, rr.rep);
    if (c) {
      x = __fsub_rn(x, __fmul_rn(rr.freq, (float)c));
      x = __fsub_rn(x, rr.pres);
    }
    if (w & kBiased)  // few: walk the list, so that equal ids add up in its order
      for (int e = rr.bias.x; e < rr.bias.y; ++e)
        if (__ldca(r.bias_ids + e) == id) x = __fadd_rn(x, __ldca(r.bias_values + e));
  }
  return x;
}

// 32 mask bits from token id on (bit 0: id).
__device__ __forceinline__ unsigned mask_bits(const uint32_t *mask, int id, int V) {
  const int w = id >> 5;
  const unsigned lo = __ldca(mask + w);
  const unsigned hi = (w + 1) * 32 < V ? __ldca(mask + w + 1) : 0u;
  return __funnelshift_r(lo, hi, id & 31);
}

struct Best {
  float v;
  int i;
};
__device__ __forceinline__ void take(Best &b, float x, int i) {
  const float v = (x == x) ? x : neg_inf_f();
  if (v > b.v || (v == b.v && i < b.i)) {
    b.v = v;
    b.i = i;
  }
}
__device__ __forceinline__ Best warp_best(Best b) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, b.v, o);
    const int i = __shfl_xor_sync(0xffffffffu, b.i, o);
    take(b, v, i);
  }
  return b;
}

// grid (CS, rows), clusters of (CS, 1, 1); rows past gridDim.y loop.
template <typename T>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(LogitArgs a) {
  constexpr int VE = 16 / sizeof(T);
  extern __shared__ unsigned words[];  // [slice]
  __shared__ Best s_warp[kLogitThreads / 32];
  __shared__ float s_v;
  __shared__ int s_i;
  const int t = threadIdx.x;
  const int lane = t & 31;
  const int cs = (int)gridDim.x;
  const int rank = (int)cluster_rank();
  const int V = a.V;
  const int lo = min(V, rank * a.slice), hi = min(V, lo + a.slice);
  const bool counts = a.r.history != nullptr || a.r.bias_ids != nullptr;
  grid_dependency_wait();
  allow_dependent_launch();
  for (int m = blockIdx.y; m < a.M; m += gridDim.y) {  // same trip count in a cluster
    const bool report = rank == 0 && t == 0;
    RowRules rr;
    rr.rep = a.r.repetition ? __ldca(a.r.repetition + m) : 1.f;
    rr.pres = a.r.presence ? __ldca(a.r.presence + m) : 0.f;
    rr.freq = a.r.frequency ? __ldca(a.r.frequency + m) : 0.f;
    rr.bias = make_int2(0, 0);
    rr.mask = nullptr;
    if (a.r.mask) {
      const int k = a.r.mask_rows ? __ldca(a.r.mask_rows + m) : m;
      if (k >= a.r.mask_count) {
        if (report) record_status(a.d_status, KVS_ERR_PAGE);
      } else if (k >= 0) {
        rr.mask = a.r.mask + (size_t)k * ((V + 31) / 32);
      }
    }
    if (counts) {
      for (int j = t; j < hi - lo; j += kLogitThreads) words[j] = 0u;
      cluster_sync_all();  // every block's words are zero
      const uint32_t base = smem_addr(words);
      if (a.r.history) {
        const int2 h = list_range(a.r.history_offsets, m, a.r.history_len, report, a.d_status);
        const int n = h.y - h.x;
        const int prompt = a.r.prompt_lens ? __ldca(a.r.prompt_lens + m) : 0;
        for (int e0 = rank * kLogitThreads + (t & ~31); e0 < n; e0 += cs * kLogitThreads) {
          const int e = e0 + lane;
          const int id = e < n ? __ldca(a.r.history + h.x + e) : -1;
          const bool made = e >= prompt;
          const bool ok = id >= 0 && id < V;
          // equal (token, kind) of the warp become one update by their first lane
          const unsigned peers = __match_any_sync(0xffffffffu, ok ? (id << 1) | (int)made : -1);
          if (ok && lane == __ffs(peers) - 1) {
            const int owner = id / a.slice;
            uint32_t at;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(at)
                         : "r"(base + 4u * (uint32_t)(id - owner * a.slice)), "r"(owner));
            if (made)
              red_add_cluster(at, (unsigned)__popc(peers));
            else
              red_or_cluster(at, kSeen);
          }
        }
      }
      if (a.r.bias_ids) {
        rr.bias = list_range(a.r.bias_offsets, m, a.r.bias_len, report, a.d_status);
        for (int e = rr.bias.x + t; e < rr.bias.y; e += kLogitThreads) {
          const int id = __ldca(a.r.bias_ids + e);  // every block marks its own slice
          if (id >= lo && id < hi) atomicOr(&words[id - lo], kBiased);
        }
      }
      cluster_sync_all();  // every update has landed
    }
    const T *x = static_cast<const T *>(a.logits) + (long long)m * a.logits_stride;
    T *y = a.out ? static_cast<T *>(a.out) + (long long)m * a.out_stride : nullptr;
    Best b{neg_inf_f(), 0x7fffffff};
    auto one = [&](int id) {
      float f = to_f32(x[id]);
      if (counts) f = apply_rules(f, words[id - lo], id, rr, a.r);
      if (rr.mask && !((__ldca(rr.mask + (id >> 5)) >> (id & 31)) & 1u)) f = neg_inf_f();
      const T o = from_f32<T>(f);
      if (y) y[id] = o;
      take(b, to_f32(o), id);
    };
    // [lo, va) and [vb, hi) one by one, [va, vb) in aligned 16-byte vectors
    // where logits and out are aligned alike
    const int mis = (int)((reinterpret_cast<uintptr_t>(x + lo) & 15u) / sizeof(T));
    const bool alike = !y || ((reinterpret_cast<uintptr_t>(y + lo) & 15u) / sizeof(T)) == (unsigned)mis;
    const int va = alike ? min(hi, lo + (mis ? VE - mis : 0)) : hi;
    const int vb = va + (hi - va) / VE * VE;
    for (int id = lo + t; id < va; id += kLogitThreads) one(id);
    for (int id = vb + t; id < hi; id += kLogitThreads) one(id);
    for (int id0 = va + VE * t; id0 < vb; id0 += VE * kLogitThreads) {
      Vec<T, VE> v = vec_load<T, VE>(x + id0);
      const unsigned bits = rr.mask ? mask_bits(rr.mask, id0, V) : ~0u;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        float f = to_f32(v.e[e]);
        if (counts) f = apply_rules(f, words[id0 - lo + e], id0 + e, rr, a.r);
        if (!((bits >> e) & 1u)) f = neg_inf_f();
        v.e[e] = from_f32<T>(f);
        take(b, to_f32(v.e[e]), id0 + e);
      }
      if (y) vec_store<T, VE>(y + id0, v);
    }
    b = warp_best(b);
    if (lane == 0) s_warp[t >> 5] = b;
    __syncthreads();
    if (t < 32) {
      Best c = (t < kLogitThreads / 32) ? s_warp[t] : Best{neg_inf_f(), 0x7fffffff};
      c = warp_best(c);
      if (t == 0) {
        s_v = c.v;
        s_i = c.i;
      }
    }
    cluster_sync_all();  // every block's maximum is in its shared memory
    if (rank == 0 && t < 32 && a.ids) {
      Best c{neg_inf_f(), 0x7fffffff};
      if (t < cs) {
        c.v = ld_dsmem_f32(dsmem_addr(&s_v, t));
        c.i = ld_dsmem_s32(dsmem_addr(&s_i, t));
      }
      c = warp_best(c);
      if (t == 0) a.ids[m] = c.v == neg_inf_f() ? 0 : c.i;
    }
    cluster_sync_all();  // block 0 has read them: they, and the words, may be overwritten
  }
}

struct LogitInfo {
  int active[5] = {0};  // resident clusters of 1, 2, 4, 8, 16 blocks with no words
  int top = 0;          // index of the largest cluster size
  int smem = 0;         // bytes of words a block may have
  bool configured = false;
};

template <typename T>
const LogitInfo *logit_info(int dev) {
  static LogitInfo info[kLogitMaxDevices];
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (!info[dev].configured) {
    LogitInfo rec;
    int optin = 0;
    if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
        cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    rec.smem = optin - 1024;
    if (cudaFuncSetAttribute(logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             rec.smem) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    int top = 4;
    if (cudaFuncSetAttribute(logits_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1) != cudaSuccess) {
      cudaGetLastError();
      top = 3;
    }
    for (int k = 0; k <= top; ++k) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1u << k, 1, 1);
      cfg.blockDim = dim3(kLogitThreads, 1, 1);
      cfg.dynamicSmemBytes = 32 << 10;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1u << k;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, logits_kernel<T>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      if (n <= 0) break;
      rec.active[k] = n;
      rec.top = k;
    }
    if (rec.active[0] < 1) return nullptr;
    rec.configured = true;
    info[dev] = rec;
  }
  return &info[dev];
}

template <typename T>
int launch_logits_impl(LogitArgs a, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kLogitMaxDevices)
    return KVS_ERR_LAUNCH;
  const LogitInfo *li = logit_info<T>(dev);
  if (!li) return KVS_ERR_LAUNCH;
  // The largest cluster whose clusters for all M rows are resident at once
  // (one wave) with slices of 8 KB or more; then larger ones until a slice's
  // words fit a block's shared memory.
  const long long row_bytes = (long long)a.V * sizeof(T);
  auto slice_of = [&](int k) { return ((a.V + (1 << k) - 1) / (1 << k) + 31) / 32 * 32; };
  const bool counts = a.r.history != nullptr || a.r.bias_ids != nullptr;
  auto words_of = [&](int k) { return counts ? (long long)slice_of(k) * 4 : 0ll; };
  int k = li->top;
  while (k > 0 && (a.M > li->active[k] || (row_bytes >> k) < (8 << 10))) --k;
  while (k < li->top && words_of(k) > li->smem) ++k;
  if (words_of(k) > li->smem) return KVS_ERR_UNSUPPORTED;
  a.slice = slice_of(k);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1u << k, (unsigned)(a.M < 65535 ? a.M : 65535), 1);
  cfg.blockDim = dim3(kLogitThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)words_of(k);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << k;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logits_kernel<T>, a);
  if (e != cudaSuccess) {
    cudaGetLastError();  // leave no stale error for the caller's next check
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

}  // namespace

int launch_logits(const void *logits, long long logits_stride, void *out, long long out_stride,
                  int dtype, int M, int V, const kvs_logit_rules &rules, int32_t *ids,
                  int *d_status, cudaStream_t stream) {
  const LogitArgs a{logits, out, logits_stride, out_stride, M, V, 0, rules, ids, d_status};
  if (dtype == KVS_F32) return launch_logits_impl<float>(a, stream);
  if (dtype == KVS_F16) return launch_logits_impl<__half>(a, stream);
  return launch_logits_impl<__nv_bfloat16>(a, stream);
}

}  // namespace kvs
