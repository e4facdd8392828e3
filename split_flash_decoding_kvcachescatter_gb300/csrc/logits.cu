// logits.cu -- penalties for repeated tokens, biases and a grammar mask on
// each of M logit rows, and the greedy token of the result, in one launch.
//
// Bound: bytes (a row is read once and written once).  What stands in the
// way is the history: a token's count decides what happens to its logit, and
// the counts of a row are needed before its first logit is final.  One
// thread-block cluster takes a row; block r owns an equal slice of the
// vocabulary and keeps one 32-bit word a token in shared memory (how often
// generated, whether seen, whether biased).  Every block reads the whole
// history (it comes from L2) and counts the tokens of its own slice with
// shared-memory atomics; the slice's logits are on their way meanwhile, in
// 16-byte loads.  (Sharing the list out, each entry sent once to its owner's
// shared memory, took 24.4 us where this takes 15.9 for 32 rows of 152,064 with
// 4,096 entries: the frequent tokens' updates queue at one block.)  The
// (value, index) maxima meet in block 0's shared memory.  Integer atomics
// only: the result does not depend on their order.
//
// Measured: 32 float32 rows of 152,064 tokens, 4,096 history entries, half of
// them masked: 16.0 us (39.6 MB, 2.5 TB/s; 5.8 us at the copy peak); one row
// 6.3 us; 67 bfloat16 rows of 32,001: 9.8 us.  The chain of launch, counting,
// row and maxima is what takes the time, not the bytes.
//
// Arithmetic is one IEEE operation at a time (no fused multiply-add), so a
// logit is the same whichever variant or alignment handles it.

#include <mutex>

#include "kvs_cluster.cuh"
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

// One logit under the penalties.  `w` is the token's word.
__device__ __forceinline__ float penalised(float x, unsigned w, const RowRules &rr) {
  const unsigned c = w & kCount;
  if ((w & kSeen) || c) x = x > 0.f ? __fdiv_rn(x, rr.rep) : __fmul_rn(x, rr.rep);
  if (c) {
    x = __fsub_rn(x, __fmul_rn(rr.freq, (float)c));
    x = __fsub_rn(x, rr.pres);
  }
  return x;
}

// 32 mask bits from token id on (bit 0: id).
__device__ __forceinline__ unsigned mask_bits(const uint32_t *mask, int id, int V) {
  const int w = id >> 5;
  const unsigned lo = __ldca(mask + w);
  const unsigned hi = (id & 31) && (w + 1) * 32 < V ? __ldca(mask + w + 1) : 0u;
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

// Token id's logit before the mask, f, becomes its result.
template <typename T>
__device__ __forceinline__ void put(T *y, const uint32_t *mask, int id, float f, Best &b) {
  if (mask && !((__ldca(mask + (id >> 5)) >> (id & 31)) & 1u)) f = neg_inf_f();
  const T o = from_f32<T>(f);
  if (y) y[id] = o;
  take(b, to_f32(o), id);
}

// The biased tokens of [lo, hi) of a list that names some of them more than once.
// A token's word becomes its penalised logit, one warp adds the list's values in
// order (32 entries at a time, those of one token one after the other), and
// whoever first takes a token's sum puts it in its place.  Linear in the list: a
// scan of it for every entry took 21 ms for 20,000 entries with one repeated
// (4 rows of 152,064), this takes 0.13 ms.  (wl[id]: the word of token id; a sum
// is never kTaken, since an addition's NaN is 0x7fffffff.)
template <typename T>
__device__ __noinline__ Best add_repeated(int lo, int hi, const T *x, T *y, unsigned *wl,
                                          RowRules rr, const int32_t *ids, const float *values) {
  constexpr unsigned kTaken = 0xffffffffu;
  constexpr int kBatch = 4;  // groups of 32 entries in flight
  const int t = threadIdx.x, lane = t & 31;
  __syncthreads();  // the words have been read
  for (int id = lo + t; id < hi; id += kLogitThreads) {
    const unsigned w = wl[id];
    if (w & kBiased) wl[id] = __float_as_uint(penalised(to_f32(x[id]), w, rr));
  }
  __syncthreads();
  if (t < 32) {
    for (int e0 = rr.bias.x; e0 < rr.bias.y; e0 += 32 * kBatch) {
      int id[kBatch];
      float v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int e = e0 + 32 * j + lane;
        id[j] = e < rr.bias.y ? __ldca(ids + e) : -1;
        v[j] = e < rr.bias.y ? __ldca(values + e) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const bool mine = id[j] >= lo && id[j] < hi;
        // how many entries of the group name this one's token before it
        const unsigned same = __match_any_sync(0xffffffffu, mine ? id[j] : -1);
        const int before = mine ? __popc(same & ((1u << lane) - 1u)) : -1;
        const int most = __reduce_max_sync(0xffffffffu, before);
        for (int k = 0; k <= most; ++k) {
          if (before == k) wl[id[j]] = __float_as_uint(__fadd_rn(__uint_as_float(wl[id[j]]), v[j]));
          __syncwarp();
        }
      }
    }
  }
  __syncthreads();
  Best b{neg_inf_f(), 0x7fffffff};
  for (int e = rr.bias.x + t; e < rr.bias.y; e += kLogitThreads) {
    const int id = __ldca(ids + e);
    if (id < lo || id >= hi) continue;
    const unsigned sum = atomicExch(&wl[id], kTaken);
    if (sum != kTaken) put(y, rr.mask, id, __uint_as_float(sum), b);
  }
  return b;
}

// grid (CS, rows), clusters of (CS, 1, 1); rows past gridDim.y loop.  A
// thread's first kAhead vectors are loaded before the history is counted, so
// that the row streams in behind the counting.
template <typename T>
__global__ void __launch_bounds__(kLogitThreads, 2) logits_kernel(LogitArgs a) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int kAhead = 3;
  constexpr int kStep = VE * kLogitThreads;
  constexpr unsigned kAll = (1u << VE) - 1u;
  extern __shared__ __align__(16) unsigned words[];  // [slice + 4]
  __shared__ Best s_warp[kLogitThreads / 32];
  __shared__ float s_v[2][16];  // of the cluster's blocks, in block 0; by row parity
  __shared__ int s_i[2][16];
  __shared__ int s_twice;  // m + 1: the bias list of row m has an id of this slice twice
  const int t = threadIdx.x;
  const int lane = t & 31;
  const int cs = (int)gridDim.x;
  const int rank = (int)cluster_rank();
  const int V = a.V;
  const int lo = min(V, rank * a.slice), hi = min(V, lo + a.slice);
  const bool counts = a.r.history != nullptr || a.r.bias_ids != nullptr;
  if (t == 0) s_twice = 0;
  if (a.ids) cluster_arrive_relaxed();  // waited for before the first remote store
  grid_dependency_wait();
  allow_dependent_launch();
  int parity = 0;
  for (int m = blockIdx.y; m < a.M; m += gridDim.y, parity ^= 1) {  // same trip count in a cluster
    const T *x = static_cast<const T *>(a.logits) + (long long)m * a.logits_stride;
    T *y = a.out ? static_cast<T *>(a.out) + (long long)m * a.out_stride : nullptr;
    // [lo, va) and [vb, hi) one by one, [va, vb) in aligned 16-byte vectors
    // where logits and out are aligned alike
    const int mis = (int)((reinterpret_cast<uintptr_t>(x + lo) & 15u) / sizeof(T));
    const bool alike = !y || ((reinterpret_cast<uintptr_t>(y + lo) & 15u) / sizeof(T)) == (unsigned)mis;
    const int va = alike ? min(hi, lo + (mis ? VE - mis : 0)) : hi;
    const int vb = va + (hi - va) / VE * VE;
    // token id's word: words[id - lo + pad], so that a vector's words are
    // 16-byte aligned (slices are whole multiples of 16 bytes: the same pad
    // in every block)
    const int pad = mis ? mis & 3 : 0;
    unsigned *const wl = words + pad - lo;
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
    Vec<T, VE> v[kAhead];
    unsigned bits[kAhead];  // the vectors' mask bits
    auto load = [&](int j, int id0) {
      if (id0 < vb) v[j] = vec_load<T, VE>(x + id0);
    };
    auto load_bits = [&](int j, int id0) {
      if (rr.mask && id0 < vb)  // (aligned vectors lie in one word)
        bits[j] = mis == 0 ? __ldca(rr.mask + (id0 >> 5)) >> (id0 & 31) : mask_bits(rr.mask, id0, V);
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) load(j, va + VE * t + j * kStep);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) load_bits(j, va + VE * t + j * kStep);
    if (counts) {
      constexpr int kBatch = 4;  // history entries of a thread in flight
      int2 h = make_int2(0, 0);
      int prompt = 0;
      if (a.r.history) {
        h = list_range(a.r.history_offsets, m, a.r.history_len, report, a.d_status);
        if (a.r.prompt_lens) prompt = __ldca(a.r.prompt_lens + m);
      }
      const int n = h.y - h.x;
      int id[kBatch];
      auto fetch = [&](int e0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int e = e0 + j * kLogitThreads;
          id[j] = e < n ? __ldca(a.r.history + h.x + e) : -1;
        }
      };
      fetch(t);
      for (int j = 4 * t; j < a.slice + 4; j += 4 * kLogitThreads)
        *reinterpret_cast<uint4 *>(words + j) = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();  // the words are zero
      for (int e0 = t; e0 < n; e0 += kBatch * kLogitThreads) {
        if (e0 != t) fetch(e0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (id[j] >= lo && id[j] < hi) {
            if (e0 + j * kLogitThreads >= prompt)
              atomicAdd(&wl[id[j]], 1u);
            else
              atomicOr(&wl[id[j]], kSeen);
          }
        }
      }
      if (a.r.bias_ids) {
        rr.bias = list_range(a.r.bias_offsets, m, a.r.bias_len, report, a.d_status);
        for (int e = rr.bias.x + t; e < rr.bias.y; e += kLogitThreads) {
          const int bid = __ldca(a.r.bias_ids + e);
          if (bid >= lo && bid < hi && (atomicOr(&wl[bid], kBiased) & kBiased)) s_twice = m + 1;
        }
      }
      __syncthreads();  // every update has landed
    }
    Best b{neg_inf_f(), 0x7fffffff};
    auto scalar = [&](int id) {
      const unsigned w = counts ? wl[id] : 0u;
      if (!(w & kBiased)) put(y, rr.mask, id, penalised(to_f32(x[id]), w, rr), b);
    };
    // The biased tokens, a thread an entry of the list: nothing else touches
    // them, so this may run beside the rest.  An entry is its token's only one
    // (the usual list); lists with an id of this slice twice come last.
    if (counts && s_twice != m + 1) {
      for (int e = rr.bias.x + t; e < rr.bias.y; e += kLogitThreads) {
        const int id = __ldca(a.r.bias_ids + e);
        if (id >= lo && id < hi)
          put(y, rr.mask, id,
              __fadd_rn(penalised(to_f32(x[id]), wl[id], rr), __ldca(a.r.bias_values + e)), b);
      }
    }
    for (int id = lo + t; id < va; id += kLogitThreads) scalar(id);
    for (int id = vb + t; id < hi; id += kLogitThreads) scalar(id);
    for (int i0 = va + VE * t; i0 < vb; i0 += kAhead * kStep) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int id0 = i0 + j * kStep;
        if (id0 >= vb) break;
        Vec<T, VE> u = v[j];
        const unsigned mb = bits[j];
        load(j, id0 + kAhead * kStep);  // the slot's next vector
        load_bits(j, id0 + kAhead * kStep);
        unsigned biased = 0u;  // elements that the loop above has
        if (counts) {
          uint4 w[VE / 4];
          unsigned any = 0u;
#pragma unroll
          for (int k = 0; k < VE / 4; ++k) {
            w[k] = *reinterpret_cast<const uint4 *>(wl + id0 + 4 * k);
            any |= w[k].x | w[k].y | w[k].z | w[k].w;
          }
          if (any != 0u) {  // few vectors hold a token with a word
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              const uint4 q = w[e / 4];
              const unsigned word = e % 4 == 0 ? q.x : e % 4 == 1 ? q.y : e % 4 == 2 ? q.z : q.w;
              u.e[e] = from_f32<T>(penalised(to_f32(u.e[e]), word, rr));
              if (word & kBiased) biased |= 1u << e;
            }
          }
        }
        if (rr.mask && (mb & kAll) != kAll) {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (!((mb >> e) & 1u)) u.e[e] = from_f32<T>(neg_inf_f());
        }
        if (biased) {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (!((biased >> e) & 1u)) {
              if (y) y[id0 + e] = u.e[e];
              take(b, to_f32(u.e[e]), id0 + e);
            }
          continue;
        }
        if (y) vec_store<T, VE>(y + id0, u);
        // the vector's maximum (fmaxf passes over NaN) and the first element
        // that holds it; a thread's vectors come in ascending order, so a
        // later one wins only if it is larger (or if the biased tokens, which
        // came before, hold the same value at a larger index)
        float mx = to_f32(u.e[VE - 1]);
        int at = VE - 1;
#pragma unroll
        for (int e = VE - 2; e >= 0; --e) {
          const float f = to_f32(u.e[e]);
          at = f >= mx || mx != mx ? e : at;
          mx = fmaxf(mx, f);
        }
        const bool better = mx > b.v || (mx == b.v && id0 + at < b.i);
        b.i = better ? id0 + at : b.i;
        b.v = better ? mx : b.v;
      }
    }
    if (counts && s_twice == m + 1) {
      const Best c = add_repeated(lo, hi, x, y, wl, rr, a.r.bias_ids, a.r.bias_values);
      take(b, c.v, c.i);
    }
    if (!a.ids) {
      __syncthreads();  // the words may be cleared for the next row
      continue;
    }
    b = warp_best(b);
    if (lane == 0) s_warp[t >> 5] = b;
    __syncthreads();
    if (m == (int)blockIdx.y) cluster_wait();  // block 0 runs: its shared memory may be written
    if (t < 32) {
      Best c = (t < kLogitThreads / 32) ? s_warp[t] : Best{neg_inf_f(), 0x7fffffff};
      c = warp_best(c);
      if (t == 0) {
        st_dsmem_f32(dsmem_addr(&s_v[parity][rank], 0), c.v);
        st_dsmem_s32(dsmem_addr(&s_i[parity][rank], 0), c.i);
      }
    }
    cluster_sync_all();  // every block's maximum is in block 0
    if (rank == 0 && t < 32) {
      Best c{neg_inf_f(), 0x7fffffff};
      if (t < cs) {
        c.v = s_v[parity][t];
        c.i = s_i[parity][t];
      }
      c = warp_best(c);
      if (t == 0) a.ids[m] = c.v == neg_inf_f() ? 0 : c.i;
    }
  }
}

struct LogitInfo {
  // resident clusters of 1, 2, 4, 8, 16 blocks, with one block an SM and with two
  int active[2][5] = {{0}, {0}};
  int top = 0;          // index of the largest cluster size
  int smem = 0;         // bytes of words a block may have
  int two = 0;          // ... of which an SM holds two
  bool configured = false;
};

template <typename T>
const LogitInfo *logit_info(int dev) {
  static LogitInfo info[kLogitMaxDevices];
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (!info[dev].configured) {
    LogitInfo rec;
    int optin = 0, of_sm = 0;
    if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&of_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) !=
            cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    rec.smem = optin - 1024;
    rec.two = of_sm / 2 - 2048;  // (1 KB reserved a block, and its static arrays)
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
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1u << k;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      for (int of = 0; of < 2; ++of) {
        cfg.dynamicSmemBytes = of ? rec.two : rec.smem;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, logits_kernel<T>, &cfg) != cudaSuccess) {
          cudaGetLastError();
          n = 0;
        }
        rec.active[of][k] = n;
      }
      if (rec.active[0][k] <= 0) break;
      rec.top = k;
    }
    if (rec.active[0][0] < 1) return nullptr;
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
  const long long row_bytes = (long long)a.V * sizeof(T);
  auto slice_of = [&](int k) { return ((a.V + (1 << k) - 1) / (1 << k) + 31) / 32 * 32; };
  const bool counts = a.r.history != nullptr || a.r.bias_ids != nullptr;
  auto words_of = [&](int k) { return counts ? (long long)(slice_of(k) + 4) * 4 : 0ll; };
  // The largest cluster whose clusters for all M rows are resident at once (one
  // wave; words past `two` leave an SM one block) with slices of 8 KB or more.
  // Where none is: the smallest whose words let an SM hold two blocks, or else
  // the smallest whose words fit.  With history and
  // biases, us at clusters of 1, 2, 4, 8, 16 (-: does not fit), * chosen:
  //   48 rows of 152,064, float32     -     -    31.0  24.4*  33.6
  //   300 rows of 152,064, float32    -     -     138  108*   177
  //   128 rows of 128,256, bfloat16   -     -    60.2  47.8*  80.8
  //   67 rows of 32,001, bfloat16   16.7  12.1   10.9* 16.5   34.2
  //   300 rows of 32,001, bfloat16  36.7  30.1*  46.1  71.3   160
  //   304 rows of 50,000, float32   43.2  34.8*  50.0  70.6   138
  //   15 rows of 262,144, bfloat16    -     -      -   16.5*  21.1
  auto resident = [&](int k) { return words_of(k) > li->smem ? 0 : li->active[words_of(k) <= li->two][k]; };
  int k = li->top;
  while (k >= 0 && (a.M > resident(k) || (row_bytes >> k) < (8 << 10))) --k;
  for (const int most : {li->two, li->smem})
    if (k < 0)
      for (int c = li->top; c >= 0; --c)
        if (words_of(c) <= most) k = c;
  if (k < 0) return KVS_ERR_UNSUPPORTED;
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
