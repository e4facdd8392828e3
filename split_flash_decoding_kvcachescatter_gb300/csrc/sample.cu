// sample.cu -- a token drawn from each of M rows of logits under temperature,
// top-k, top-p and min-p, with given random numbers, in one launch.
//
// Mathematics.  A row's tokens in order of falling logit (of equal ones the lower id
// first) have the weights w = e^((x - max) / T).  Top-k keeps the first k; top-p, of
// those, the shortest run from the front with p of their weight; min-p those with at
// least min_p of the largest weight.  What is kept is so always a run from the front:
// the tokens above some logit and the first few that equal it.  No row is sorted: the
// logit is found by counting, digit by digit of its bits (an order-preserving integer),
// how many tokens (top-k) or how much weight (top-p) lie above.  The token drawn is the
// first id at which the running sum of kept weights, in the order of ids, exceeds u
// times their sum.
//
// Weights are integers, w 2^44 rounded, computed to 2^-41 of themselves (below), so
// sums are exact whatever their order, and a token is drawn wrongly only where u falls
// within about 2^-40 of a border between two tokens.
//
// A thread-block cluster takes a row; block r owns an equal slice of the ids and keeps
// their logits in shared memory.  Histograms of a digit are gathered with
// shared-memory atomics, summed over the cluster a share of the bins a block, and
// scanned by every block.
//
// Bound: bytes (a row is read once).

#include <mutex>

#include "kvs_cluster.cuh"
#include "kvs_exp2_table.cuh"
#include "kvs_paged.cuh"

namespace kvs {

namespace {

constexpr int kSThreads = 512;
constexpr int kSBins = 2048;
constexpr int kSMaxDevices = 64;
typedef unsigned long long u64;

struct SampleArgs {
  const void *logits;
  long long logits_stride;
  float *probs;
  long long probs_stride;
  int M, V, slice;
  const float *uniforms;
  kvs_sample_rules r;
  int32_t *ids;
  float *token_probs;
};

// An integer that orders logits: larger for larger ones, equal for equal ones; 0 for
// NaN and -inf, which are never chosen.
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned u = __float_as_uint(x + 0.f);  // (-0 equals 0)
  if (!(x > neg_inf_f())) return 0u;
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(unsigned key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Weights of a row: largest logit and log2(e) / T in two parts.
struct Weigher {
  float top, ch, cl;
  const u64 *table;  // 2^(i / 256) 2^44

  // e^((x - top) / T) 2^44.  y = (x - top) log2(e) / T as a sum of two floats
  // (off by 2^-46 of it); y = n + i / 256 + r with |r| <= 2^-9; 2^r - 1 = e^(r ln 2) - 1
  // by its series, whose first term is kept in two floats; all but the leading parts
  // are below 2^-17, so float arithmetic is off by 2^-41 there.
  __device__ __forceinline__ u64 operator()(unsigned key) const {
    if (key == 0u) return 0ull;
    const float x = logit_of(key);
    if (!(top < __uint_as_float(0x7f800000u))) return x == top ? 1ull << 44 : 0ull;
    const float d = fmaxf(__fsub_rn(x, top), -3.4e38f);
    const float b = __fsub_rn(d, x);
    const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-top, b));
    const float p = __fmul_rn(d, ch);
    if (!(p > -46.f)) return 0ull;
    const float e = __fadd_rn(__fmaf_rn(d, ch, -p), __fmaf_rn(d, cl, __fmul_rn(dl, ch)));
    const float t = rintf(__fmul_rn(p, 256.f));
    const float rr = __fmaf_rn(t, -1.f / 256.f, p);  // exact
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Low = -1.904654323148236e-09f;
    const float zh = __fmul_rn(rr, kLn2);
    const float zl = __fadd_rn(__fmaf_rn(rr, kLn2, -zh), __fmaf_rn(rr, kLn2Low, __fmul_rn(e, kLn2)));
    const float sq = __fmul_rn(zh, zh);
    const float poly = __fmul_rn(sq, __fmaf_rn(zh, __fmaf_rn(zh, 1.f / 24.f, 1.f / 6.f), 0.5f));
    const float rest = __fadd_rn(poly, __fmaf_rn(zh, zl, zl));  // e^z - 1 = zh + rest
    const int ti = (int)t;
    const u64 tab = table[ti & 255];
    const float th = (float)(unsigned)(tab >> 21) * 1.1920928955078125e-07f;  // 2^(i / 256), 24 bits
    const float tl = (float)((int)(tab & 0x1fffffu)) * 5.684341886080802e-14f;  // and what is left
    const float hi = __fmul_rn(th, zh);
    const float lo = __fadd_rn(__fmaf_rn(th, zh, -hi), __fmaf_rn(tl, zh, __fmul_rn(th, rest)));
    // hi + lo in units of 2^-44, in two steps
    const float h1 = rintf(__fmul_rn(hi, 2147483648.f));
    const float left = __fadd_rn(__fmaf_rn(h1, -4.656612873077393e-10f, hi), lo);
    const long long w = (long long)tab + (long long)(int)h1 * 8192 +
                        (long long)(int)rintf(__fmul_rn(left, 17592186044416.f));
    const int n = -(ti >> 8);  // 0 .. 46
    return n == 0 ? (u64)w : ((u64)w + (1ull << (n - 1))) >> n;
  }
};

// floor(f x) for 0 <= f < 1 as the float it is, and whether something was left.
__device__ __forceinline__ u64 share_of(float f, u64 x, bool &left) {
  const unsigned u = __float_as_uint(f);
  const int ex = max((int)(u >> 23), 1);
  const u64 mant = (u >> 23) ? (u & 0x7fffffu) | 0x800000u : (u & 0x7fffffu);
  const int s = 150 - ex;  // f = mant 2^-s, s >= 24
  const u64 lo = mant * x, hi = __umul64hi(mant, x);
  if (s >= 128) {
    left = (lo | hi) != 0ull;
    return 0ull;
  }
  if (s >= 64) {
    left = lo != 0ull || (s > 64 && (hi & ((1ull << (s - 64)) - 1ull)) != 0ull);
    return s == 64 ? hi : hi >> (s - 64);
  }
  left = (lo & ((1ull << s) - 1ull)) != 0ull;
  return (lo >> s) | (hi << (64 - s));
}

struct SampleShared {
  unsigned count[kSBins];   // of this block's tokens
  unsigned tcount[kSBins];  // of the row's
  u64 mass[kSBins];
  u64 tmass[kSBins];
  u64 table[256];
  unsigned top[16];         // of the cluster's blocks
  unsigned ties[16];
  u64 above[16];
  u64 wmass[32];
  unsigned wcount[32];
  int bin;
  unsigned before_count;
  u64 before_mass;
  int cut;
};

// The bin, from the top, in which a running number passes `need`, over the row's
// counts (kCount) or weights; leaves it in s.bin with what lies above it (s.bin = -1:
// all of them do not reach it).  By the whole block.
template <bool kCount>
__device__ __forceinline__ void find_bin(SampleShared &s, u64 need) {
  constexpr int kPer = kSBins / kSThreads;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  unsigned c[kPer], csum = 0u;
  u64 m[kPer], msum = 0ull;
  // thread t takes bins from the top: kSBins - 1 - (kPer t + j)
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    c[j] = s.tcount[kSBins - 1 - (kPer * t + j)];
    m[j] = s.tmass[kSBins - 1 - (kPer * t + j)];
    csum += c[j];
    msum += m[j];
  }
  unsigned ci = csum;
  u64 mi = msum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned cv = __shfl_up_sync(0xffffffffu, ci, o);
    const u64 mv = __shfl_up_sync(0xffffffffu, mi, o);
    if (lane >= o) {
      ci += cv;
      mi += mv;
    }
  }
  if (lane == 31) {
    s.wcount[warp] = ci;
    s.wmass[warp] = mi;
  }
  if (t == 0) s.bin = -1;
  __syncthreads();
  unsigned cb = ci - csum;
  u64 mb = mi - msum;
  for (int w = 0; w < warp; ++w) {
    cb += s.wcount[w];
    mb += s.wmass[w];
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const u64 lo = kCount ? (u64)cb : mb, hi = lo + (kCount ? (u64)c[j] : m[j]);
    if (lo < need && need <= hi) {  // (one bin at most)
      s.bin = kSBins - 1 - (kPer * t + j);
      s.before_count = cb;
      s.before_mass = mb;
    }
    cb += c[j];
    mb += m[j];
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kSThreads) sample_kernel(SampleArgs a) {
  constexpr int VE = 16 / sizeof(T);
  extern __shared__ __align__(16) unsigned char raw[];
  SampleShared &s = *reinterpret_cast<SampleShared *>(raw);
  unsigned *keys = reinterpret_cast<unsigned *>(raw + sizeof(SampleShared));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int cs = (int)gridDim.x, rank = (int)cluster_rank();
  const int lo = min(a.V, rank * a.slice), hi = min(a.V, lo + a.slice), n = hi - lo;
  if (t < 256) s.table[t] = kExp2Table[t];
  grid_dependency_wait();
  allow_dependent_launch();
  // a histogram of digit `shift` of the keys whose bits from `from` up are `prefix`
  auto histogram = [&](const Weigher &weigh, int shift, int from, unsigned prefix, bool with_mass) {
    for (int j = t; j < kSBins; j += kSThreads) {
      s.count[j] = 0u;
      s.mass[j] = 0ull;
    }
    __syncthreads();
    for (int j = t; j < n; j += kSThreads) {
      const unsigned k = keys[j];
      if (k == 0u || (from < 32 && (k >> from) != prefix)) continue;
      const unsigned bin = (k >> shift) & (kSBins - 1);
      atomicAdd(&s.count[bin], 1u);
      if (with_mass) atomicAdd(&s.mass[bin], weigh(k));
    }
    cluster_sync_all();  // every block's histogram is there
    const int per = kSBins / cs;
    for (int j = t; j < per; j += kSThreads) {
      const int bin = rank * per + j;
      unsigned c = 0u;
      u64 m = 0ull;
      for (int r = 0; r < cs; ++r) {
        c += (unsigned)ld_dsmem_s32(dsmem_addr(&s.count[bin], r));
        m += ld_dsmem_u64(dsmem_addr(&s.mass[bin], r));
      }
      for (int r = 0; r < cs; ++r) {
        st_dsmem_s32(dsmem_addr(&s.tcount[bin], r), (int)c);
        st_dsmem_u64(dsmem_addr(&s.tmass[bin], r), m);
      }
    }
    cluster_sync_all();  // the row's histogram is in every block
  };
  constexpr int kShift[3] = {21, 10, 0};
  for (int m = blockIdx.y; m < a.M; m += gridDim.y) {  // same trip count in a cluster
    const T *x = static_cast<const T *>(a.logits) + (long long)m * a.logits_stride + lo;
    const float temp = a.r.temperature ? __ldca(a.r.temperature + m) : 1.f;
    const bool greedy = !(temp >= 1.1754943508222875e-38f);
    int k = a.r.top_k ? __ldca(a.r.top_k + m) : 0;
    if (greedy) k = 1;
    const float p = !greedy && a.r.top_p ? __ldca(a.r.top_p + m) : 1.f;
    const float least = !greedy && a.r.min_p ? __ldca(a.r.min_p + m) : 0.f;
    const float u = __ldca(a.uniforms + m);
    // ---- the slice's logits ----
    unsigned most = 0u;
    const int mis = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int va = min(n, mis ? VE - mis : 0), vb = va + (n - va) / VE * VE;
    auto put = [&](int j, float f) {
      const unsigned key = key_of(f);
      keys[j] = key;
      most = max(most, key);
    };
    for (int j = t; j < va; j += kSThreads) put(j, to_f32(x[j]));
    for (int j = vb + t; j < n; j += kSThreads) put(j, to_f32(x[j]));
    for (int j = va + VE * t; j < vb; j += VE * kSThreads) {
      const Vec<T, VE> v = vec_load<T, VE>(x + j);
#pragma unroll
      for (int e = 0; e < VE; ++e) put(j + e, to_f32(v.e[e]));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s.wcount[warp] = most;
    __syncthreads();
    cluster_sync_all();  // every block runs, and is done with the row before
    if (t < cs) {
      unsigned w = 0u;
      for (int j = 0; j < kSThreads / 32; ++j) w = max(w, s.wcount[j]);
      st_dsmem_s32(dsmem_addr(&s.top[rank], t), (int)w);
    }
    cluster_sync_all();
    unsigned top = 0u;
    for (int r = 0; r < cs; ++r) top = max(top, s.top[r]);
    if (top == 0u) {  // nothing above -inf
      if (rank == 0 && t == 0) {
        if (a.ids) a.ids[m] = 0;
        if (a.token_probs) a.token_probs[m] = 0.f;
      }
      if (a.probs)
        for (int j = t; j < n; j += kSThreads) a.probs[(long long)m * a.probs_stride + lo + j] = 0.f;
      continue;
    }
    Weigher weigh{logit_of(top), 0.f, 0.f, s.table};
    {
      const double c = 1.4426950408889634074 / (double)(greedy ? 1.f : temp);
      weigh.ch = (float)c;
      weigh.cl = (float)(c - (double)weigh.ch);
    }
    // ---- the last logit that is kept, and how many tokens that equal it ----
    unsigned thr = 0u, kept = 0u;  // (nothing equals key 0)
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.f;
    u64 sum = 0ull;  // weight of what top-k keeps
    if (by_k && k == 1) {
      thr = top;
      kept = 1u;
      sum = 1ull << 44;
    } else if (by_k) {
      unsigned prefix = 0u;
      u64 need = (u64)k;
      int from = 32;
      for (int pass = 0; pass < 3; ++pass) {
        histogram(weigh, kShift[pass], from, prefix, by_p);
        find_bin<true>(s, need);
        if (s.bin < 0) break;  // fewer tokens than k
        need -= s.before_count;
        sum += s.before_mass;
        from = kShift[pass];
        prefix = pass == 0 ? (unsigned)s.bin : prefix << (kShift[pass - 1] - kShift[pass]) | (unsigned)s.bin;
        __syncthreads();
      }
      if (from == 0) {
        thr = prefix;
        kept = (unsigned)need;
        sum += need * weigh(thr);
      }
    }
    if (by_p && !(by_k && k == 1)) {
      unsigned prefix = 0u;
      int from = 32;
      u64 need = 0ull;
      for (int pass = 0; pass < 3; ++pass) {
        histogram(weigh, kShift[pass], from, prefix, true);
        if (pass == 0) {
          if (thr == 0u) {  // all of the row
            sum = 0ull;
            for (int j = lane; j < kSBins; j += 32) sum += s.tmass[j];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          }
          bool left;
          need = p > 0.f ? share_of(p, sum, left) : 0ull;
          if (p > 0.f && left) ++need;
          if (need == 0ull) need = 1ull;
        }
        find_bin<false>(s, need);
        need -= s.before_mass;
        from = kShift[pass];
        prefix = pass == 0 ? (unsigned)s.bin : prefix << (kShift[pass - 1] - kShift[pass]) | (unsigned)s.bin;
        __syncthreads();
      }
      thr = prefix;
      const u64 w = weigh(thr);
      kept = (unsigned)((need + w - 1ull) / w);
    }
    // ---- min-p: a weight that is kept at the least ----
    const u64 floor_w = least > 0.f ? (least >= 1.f ? 1ull << 44 : [&] {
      bool left;
      const u64 w = share_of(least, 1ull << 44, left);
      return w + (left ? 1ull : 0ull);
    }()) : 0ull;
    const u64 thr_w = thr ? weigh(thr) : 0ull;
    if (thr_w < floor_w) kept = 0u;
    // ---- this block's share: a run of ids a thread ----
    const int run = ((n + kSThreads - 1) / kSThreads) | 1;  // (odd: no bank conflicts)
    const int j0 = min(n, t * run), j1 = min(n, j0 + run);
    u64 above = 0ull;
    unsigned ties = 0u;
    for (int j = j0; j < j1; ++j) {
      const unsigned key = keys[j];
      if (key > thr) {
        const u64 w = weigh(key);
        if (w >= floor_w) above += w;
      } else if (key == thr && key) {
        ++ties;
      }
    }
    u64 ai = above;
    unsigned ci = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 av = __shfl_up_sync(0xffffffffu, ai, o);
      const unsigned cv = __shfl_up_sync(0xffffffffu, ci, o);
      if (lane >= o) {
        ai += av;
        ci += cv;
      }
    }
    if (lane == 31) {
      s.wmass[warp] = ai;
      s.wcount[warp] = ci;
    }
    __syncthreads();
    u64 ab = ai - above, atot = 0ull;  // before this thread, of the block
    unsigned cb = ci - ties, ctot = 0u;
    for (int w = 0; w < kSThreads / 32; ++w) {
      if (w < warp) {
        ab += s.wmass[w];
        cb += s.wcount[w];
      }
      atot += s.wmass[w];
      ctot += s.wcount[w];
    }
    if (t < cs) {
      st_dsmem_u64(dsmem_addr(&s.above[rank], t), atot);
      st_dsmem_s32(dsmem_addr(&s.ties[rank], t), (int)ctot);
    }
    if (t == 0) s.cut = -1;
    cluster_sync_all();
    u64 total = 0ull, first = 0ull;  // of the row; before this block
    unsigned seen = 0u, seen_first = 0u;
    for (int r = 0; r < cs; ++r) {
      const unsigned c = min(s.ties[r], kept - min(kept, seen));
      const u64 w = s.above[r] + (u64)c * thr_w;
      if (r < rank) first += w;
      if (r == rank) seen_first = seen;
      total += w;
      seen += s.ties[r];
    }
    bool left;
    u64 mark = !(u > 0.f) ? 0ull : u < 1.f ? share_of(u, total, left) : total - 1ull;
    if (mark >= total) mark = total - 1ull;
    // (ties of the row before this thread's run, and how many of them are kept)
    const unsigned tb = seen_first + cb;
    const u64 before = first + ab + (u64)(min(tb, kept) - min(seen_first, kept)) * thr_w;
    const u64 own = above + (u64)(min(tb + ties, kept) - min(tb, kept)) * thr_w;
    const bool here = before <= mark && mark < before + own;
    const bool cut_here = tb < kept && kept <= tb + ties;  // the last kept one of the ties
    if (here || cut_here) {
      u64 at = before;
      unsigned tie = tb;
      for (int j = j0; j < j1; ++j) {
        const unsigned key = keys[j];
        u64 w = 0ull;
        if (key > thr) {
          w = weigh(key);
          if (w < floor_w) w = 0ull;
        } else if (key == thr && key) {
          if (tie < kept) w = thr_w;
          if (++tie == kept) s.cut = j;
        }
        if (here && at <= mark && mark < at + w) {
          if (a.ids) a.ids[m] = lo + j;
          if (a.token_probs) a.token_probs[m] = (float)((double)w / (double)total);
        }
        at += w;
      }
    }
    if (a.probs) {
      __syncthreads();  // cut is there
      // ties up to position `cut` of the slice are kept; all of them where the last kept
      // one lies in a later block
      const int cut = s.cut >= 0 ? s.cut : seen_first + ctot <= kept ? n : -1;
      const float inv = (float)(1.0 / (double)total);
      float *to = a.probs + (long long)m * a.probs_stride + lo;
      for (int j = t; j < n; j += kSThreads) {
        const unsigned key = keys[j];
        u64 w = 0ull;
        if (key > thr) {
          w = weigh(key);
          if (w < floor_w) w = 0ull;
        } else if (key == thr && key && j <= cut) {
          w = kept ? thr_w : 0ull;
        }
        to[j] = __ull2float_rn(w) * inv;
      }
    }
    __syncthreads();  // the keys may be replaced
  }
  // (a cluster barrier follows every access to another block's memory)
}

struct SampleInfo {
  int active[2][5] = {{0}, {0}};  // resident clusters of 1, 2, 4, 8, 16 blocks, with one block an SM and with two
  int top = 0;                    // index of the largest cluster size
  int smem = 0, two = 0;          // bytes a block may have, and of which an SM holds two
  bool configured = false;
};

template <typename T>
const SampleInfo *sample_info(int dev) {
  static SampleInfo info[kSMaxDevices];
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (!info[dev].configured) {
    SampleInfo rec;
    int optin = 0, of_sm = 0;
    if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&of_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    rec.smem = optin;
    rec.two = of_sm / 2 - 1024;  // (1 KB reserved a block)
    if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, rec.smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    int top = 4;
    if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
        cudaSuccess) {
      cudaGetLastError();
      top = 3;
    }
    for (int k = 0; k <= top; ++k) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1u << k, 1, 1);
      cfg.blockDim = dim3(kSThreads, 1, 1);
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
        if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<T>, &cfg) != cudaSuccess) {
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
int launch_sample_impl(SampleArgs a, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kSMaxDevices) return KVS_ERR_LAUNCH;
  const SampleInfo *si = sample_info<T>(dev);
  if (!si) return KVS_ERR_LAUNCH;
  auto slice_of = [&](int k) { return ((a.V + (1 << k) - 1) / (1 << k) + 31) / 32 * 32; };
  auto bytes_of = [&](int k) { return (long long)sizeof(SampleShared) + 4ll * slice_of(k); };
  // The largest cluster whose clusters for all M rows are resident at once, with
  // slices of 2048 ids or more; where none is, the smallest whose slices fit.
  auto resident = [&](int k) { return bytes_of(k) > si->smem ? 0 : si->active[bytes_of(k) <= si->two][k]; };
  int k = si->top;
  while (k >= 0 && (a.M > resident(k) || (a.V >> k) < 2048)) --k;
  if (k < 0)
    for (int c = si->top; c >= 0; --c)
      if (bytes_of(c) <= si->smem) k = c;
  if (k < 0) return KVS_ERR_UNSUPPORTED;
  a.slice = slice_of(k);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1u << k, (unsigned)(a.M < 65535 ? a.M : 65535), 1);
  cfg.blockDim = dim3(kSThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)bytes_of(k);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
  if (e != cudaSuccess) {
    cudaGetLastError();  // leave no stale error for the caller's next check
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

}  // namespace

int launch_sample(const void *logits, long long logits_stride, int dtype, int M, int V,
                  const float *uniforms, const kvs_sample_rules &rules, int32_t *ids,
                  float *token_probs, float *probs, long long probs_stride, cudaStream_t stream) {
  const SampleArgs a{logits, logits_stride, probs, probs_stride, M, V, 0, uniforms, rules, ids, token_probs};
  if (dtype == KVS_F32) return launch_sample_impl<float>(a, stream);
  if (dtype == KVS_F16) return launch_sample_impl<__half>(a, stream);
  return launch_sample_impl<__nv_bfloat16>(a, stream);
}

}  // namespace kvs
