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
// Weights are integers, w 2^44 computed to 2^-37 of itself (below) and rounded, so
// sums are exact whatever their order, and a token is drawn wrongly only where u falls
// within 2^-36 + V 2^-44 of a border between two tokens: the sum up to a border and that of
// the row are each off by 2^-37 of themselves and by V roundings of 2^-45 of the largest
// weight.  (More bits a weight would not fit: 2^19 tokens of 2^44 make 2^63.)
//
// A thread-block cluster takes a row; block r owns an equal slice of the ids and keeps
// their logits in shared memory.  One histogram over the distance from the largest
// logit, 64 bins a unit of (x - max) / T, says in which bin the last kept token lies
// (amounts by shared-memory atomics, summed over the cluster a share of the bins a
// block, scanned by every block); the bin's tokens, or all down to it where they are at
// most 1024, go to block 0, which sorts them.  Few tokens are then finished there, and
// the row's 150,000 have been looked at twice.  Where the bin holds more (rows of nearly
// equal logits) or lies 32 units down, the logit is found digit by digit of its bits.
// For a small k each block bounds the row's k-th logit by the k-th of its threads' maxima;
// what reaches the largest of these bounds goes to block 0 without the row's histogram.
//
// Bound: bytes (a row is read once); what it takes is a chain of short phases (a cluster
// barrier each 0.6 us) and, without a top-k, the instructions of a weight for every token.
// Measured: one row of 152,064 in float32 17 us (23 by other rules), 32 rows 56, 67 of 32,001 in
// bfloat16 36, 24 of 152,064 in float16 with all probabilities 55.  By digits of the bits alone, 64-bit atomics
// for the weights 73 (one row) and 229 (32), pairs of 32-bit ones 39 and 77; the histogram over
// the distance 19 and 65; weights in fewer steps, one thread for 1 / T and bounds that spare
// the counting 18 and 58.  (Small k by the row's histogram: one row 18.)

#include <mutex>
#include <type_traits>

#include "kvs_cluster.cuh"
#include "kvs_exp2_table.cuh"
#include "kvs_paged.cuh"

namespace kvs {

namespace {

constexpr int kSThreads = 512;
constexpr int kSBins = 2048;  // of a digit of 11 bits, and of 32 units of distance
constexpr int kSMost = 1024;  // tokens that block 0 sorts
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

// An integer of the type's size that orders its numbers: larger for larger ones, equal
// for equal ones; 0 for NaN and -inf, which are never chosen.
template <typename T>
struct Keys {  // the 16-bit types
  using Key = uint16_t;
  static constexpr int kPasses = 2;
  static constexpr bool kHalf = std::is_same<T, __half>::value;
  static __host__ __device__ constexpr int shift(int pass) { return pass == 0 ? 5 : 0; }
  static __device__ __forceinline__ Key of(T x) {
    const unsigned u = *reinterpret_cast<const uint16_t *>(&x), inf = kHalf ? 0x7c00u : 0x7f80u;
    if ((u & 0x7fffu) > inf || u == (inf | 0x8000u)) return 0;
    if ((u & 0x7fffu) == 0u) return 0x8000;  // (-0 equals 0)
    return (Key)(u ^ ((u & 0x8000u) ? 0xffffu : 0x8000u));
  }
  static __device__ __forceinline__ float logit(unsigned key) {
    const uint16_t u = (uint16_t)(key ^ ((key & 0x8000u) ? 0x8000u : 0xffffu));
    return to_f32(*reinterpret_cast<const T *>(&u));
  }
};
template <>
struct Keys<float> {
  using Key = uint32_t;
  static constexpr int kPasses = 3;
  static __host__ __device__ constexpr int shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
  static __device__ __forceinline__ Key of(float x) {
    const unsigned u = __float_as_uint(x + 0.f);  // (-0 equals 0)
    if (!(x > neg_inf_f())) return 0u;
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  }
  static __device__ __forceinline__ float logit(unsigned key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
  }
};

// Weights of a row: largest logit and log2(e) / T in two parts.
template <typename T>
struct Weigher {
  float top, ch, cl;
  const u64 *table;  // 2^(i / 256) 2^44

  // e^((x - top) / T) 2^44.  y = (x - top) log2(e) / T as a sum of two floats (off by
  // 2^-46 of it); y = n + i / 256 + r with |r| <= 2^-9; z = 2^r - 1 = e^(r ln 2) - 1 by its
  // series: the first term in two floats, the others, below 2^-19, in one; then 2^(i / 256)
  // (1 + z) in integers, z in units of 2^-40.  Off by 2^-37 of itself at most, and the last
  // shift by half a unit.
  __device__ __forceinline__ u64 operator()(unsigned key) const {
    if (key == 0u) return 0ull;
    const float x = Keys<T>::logit(key);
    if (!(top < __uint_as_float(0x7f800000u))) return x == top ? 1ull << 44 : 0ull;
    const float d = fmaxf(__fsub_rn(x, top), -3.4e38f);
    const float b = __fsub_rn(d, x);
    const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-top, b));
    const float p = __fmul_rn(d, ch);
    if (!(p > -46.f)) return 0ull;
    const float e = __fadd_rn(__fmaf_rn(d, ch, -p), __fmaf_rn(d, cl, __fmul_rn(dl, ch)));
    const int t = __float2int_rn(__fmul_rn(p, 256.f));
    const float rr = __fmaf_rn((float)t, -1.f / 256.f, p);  // exact
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Low = -1.904654323148236e-09f;
    const float zh = __fmul_rn(rr, kLn2);
    const float zl = __fadd_rn(__fmaf_rn(rr, kLn2, -zh), __fmaf_rn(rr, kLn2Low, __fmul_rn(e, kLn2)));
    const float rest = __fmaf_rn(__fmul_rn(zh, zh), __fmaf_rn(zh, 1.f / 6.f, 0.5f), __fmaf_rn(zh, zl, zl));
    const int z = __float2int_rn(__fmul_rn(zh, 1099511627776.f)) + __float2int_rn(__fmul_rn(rest, 1099511627776.f));
    const u64 tab = table[t & 255];
    // tab z 2^-40, from tab's upper 32 bits
    const u64 w = tab + (u64)(((long long)(int)(unsigned)(tab >> 14) * (long long)z) >> 26);
    const int n = -(t >> 8);  // 0 .. 46
    return (w + ((1ull << n) >> 1)) >> n;
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

// w / total for w <= 2^45, total < 2^64, to a rounding of float32 (2^-24 and 2^-44 of itself):
// the reciprocal and w as sums of two floats, the product's first term exact.
struct Divider {
  float ih, il;
  __device__ __forceinline__ explicit Divider(u64 total) {
    const float th = __ull2float_rn(total);
    const float tl = __ll2float_rn((long long)(total - (u64)th));  // (total <= 2^63: th is, too)
    ih = __frcp_rn(th);
    il = __fmul_rn(ih, __fmaf_rn(-ih, tl, __fmaf_rn(-ih, th, 1.f)));
  }
  __device__ __forceinline__ float operator()(u64 w) const {
    const float a = __fmul_rn(__uint2float_rn((unsigned)(w >> 22)), 4194304.f);
    const float b = __uint2float_rn((unsigned)w & 0x3fffffu);  // (both exact)
    const float wh = __fadd_rn(a, b), wl = __fsub_rn(b, __fsub_rn(wh, a));
    const float p = __fmul_rn(wh, ih);
    return __fadd_rn(p, __fmaf_rn(wl, ih, __fmaf_rn(wh, il, __fmaf_rn(wh, ih, -p))));
  }
};

struct alignas(16) SampleShared {  // (the keys lie behind it)
  // this block's amounts (tokens or weight), by bin; or the tokens it sends to block 0
  union {
    struct {
      unsigned low[kSBins], high[kSBins];
    };
    u64 out[kSMost];
  };
  // the row's; or in block 0 the tokens to sort (key, then ~id), and their weights
  union {
    u64 amount[kSBins];
    struct {
      u64 item[kSMost], weight[kSMost];
    };
  };
  u64 table[256];
  unsigned top[2][16];  // of the cluster's blocks, by row parity
  int bound[16];
  unsigned ties[16];
  u64 above[16];
  u64 wsum[32];
  unsigned wcount[32];
  int bin, cut;
  u64 before, inside;
  unsigned sent, total[2];       // tokens in out; in block 0: in item, by gather parity
  unsigned found_key, found_kept;  // the last kept logit, and how many tokens that equal it
  u64 found_cut;                 // weight of those that equal it and are not kept
  float rate[2];                 // log2(e) / T in two parts
};
static_assert(sizeof(SampleShared) % 16 == 0 && kSBins % 4 == 0, "vectors of keys and of bins");
static_assert(kSMost <= 2 * kSThreads && kSMost * 16 <= kSBins * 8, "two tokens a thread, where the amounts were");

// The row's amounts from the cluster's blocks': (bin, block) pairs, four a thread, the
// pairs of a bin side by side: four loads in flight, sums over the threads of a bin,
// and each pair's thread stores the bin's sum to the pair's block.
__device__ __forceinline__ void sum_bins(SampleShared &s, int rank, int cs) {
  const int log = __ffs(cs) - 1, per = kSBins >> log;
  u64 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int pair = 4 * (int)threadIdx.x + u, bin = rank * per + (pair >> log), r = pair & (cs - 1);
    v[u] = (u64)(unsigned)ld_dsmem_s32(dsmem_addr(&s.high[bin], r)) << 32;
    v[u] += (unsigned)ld_dsmem_s32(dsmem_addr(&s.low[bin], r));
  }
  if (cs >= 4) {
    u64 t = v[0] + v[1] + v[2] + v[3];
    for (int o = cs / 8; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    v[0] = v[1] = v[2] = v[3] = t;
  } else if (cs == 2) {
    v[0] = v[1] = v[0] + v[1];
    v[2] = v[3] = v[2] + v[3];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int pair = 4 * (int)threadIdx.x + u, bin = rank * per + (pair >> log), r = pair & (cs - 1);
    st_dsmem_u64(dsmem_addr(&s.amount[bin], r), v[u]);
  }
}

// The bin, from the top, in which the running amount reaches need(all of it); leaves it
// in s.bin with what lies above it and in it (s.bin = -1: all of them do not reach it),
// and returns the whole amount.  By the whole block.  kOwn: of this block's counts.
template <bool kOwn = false, typename Need>
__device__ __forceinline__ u64 find_bin(SampleShared &s, Need need) {
  constexpr int kPer = kSBins / kSThreads;
  static_assert(kPer == 4, "two 16-byte loads");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  // thread t takes bins from the top: kSBins - 1 - (4 t + j)
  u64 m[4];
  if constexpr (kOwn) {
    const uint4 c = *reinterpret_cast<const uint4 *>(&s.low[kSBins - 4 - 4 * t]);
    m[0] = c.w, m[1] = c.z, m[2] = c.y, m[3] = c.x;
  } else {
    const ulonglong2 hi = *reinterpret_cast<const ulonglong2 *>(&s.amount[kSBins - 2 - 4 * t]);
    const ulonglong2 lo = *reinterpret_cast<const ulonglong2 *>(&s.amount[kSBins - 4 - 4 * t]);
    m[0] = hi.y, m[1] = hi.x, m[2] = lo.y, m[3] = lo.x;
  }
  const u64 mine = m[0] + m[1] + m[2] + m[3];
  u64 inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.wsum[warp] = inc;
  if (t == 0) s.bin = -1;
  __syncthreads();
  u64 before = inc - mine, all = 0ull;
#pragma unroll
  for (int w = 0; w < kSThreads / 32; ++w) {
    const u64 x = s.wsum[w];
    if (w < warp) before += x;
    all += x;
  }
  const u64 n = need(all);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (before < n && n <= before + m[j]) {  // (one bin at most)
      s.bin = kSBins - 1 - (kPer * t + j);
      s.before = before;
      s.inside = m[j];
    }
    before += m[j];
  }
  __syncthreads();
  return all;
}

__device__ __forceinline__ int power_of_two(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// The first n of x (all different, above 0; n <= kSMost) in falling order; by the block.  What
// lies behind them up to a power of two may be overwritten.
__device__ __forceinline__ void sort_falling(u64 *x, int n) {
  const int t = threadIdx.x;
  const int n2 = power_of_two(n);
  if (n2 <= 256) {
    // An item's place is the number of larger ones, counted by kSThreads / n2 threads side by
    // side (32 at most): for 50 items some 200 cycles where the network below takes 1300.
    const int parts = min(kSThreads / n2, 32), i = t / parts, part = t & (parts - 1);
    const u64 mine = i < n ? x[i] : 0ull;
    int place = 0;
    if (i < n)
      for (int j = part; j < n; j += parts) place += x[j] > mine;
    for (int o = parts >> 1; o >= 1; o >>= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    __syncthreads();
    if (i < n && part == 0) x[place] = mine;
    __syncthreads();
    return;
  }
  for (int i = n + t; i < n2; i += kSThreads) x[i] = 0ull;
  __syncthreads();
  // (Steps of 32 and less stay within the 64 places of a warp's threads.)
  for (int size = 2; size <= n2; size <<= 1) {
    for (int step = size >> 1; step >= 1; step >>= 1) {
      if (2 * t < n2) {
        const int i = 2 * t - (t & (step - 1)), j = i + step;
        const u64 p = x[i], q = x[j];
        if ((p < q) == ((i & size) == 0)) {
          x[i] = q;
          x[j] = p;
        }
      }
      // the next step, of this size or of the next one
      if ((step > 1 ? step >> 1 : size) >= 64 || step >= 64)
        __syncthreads();
      else
        __syncwarp();
    }
  }
  __syncthreads();
}

// Sums of x[0 .. i] in place, i < n <= kSMost; by the block.
__device__ __forceinline__ void running_sums(SampleShared &s, u64 *x, int n) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  u64 p = 2 * t < n ? x[2 * t] : 0ull, q = 2 * t + 1 < n ? x[2 * t + 1] : 0ull;
  u64 inc = p + q;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.wsum[warp] = inc;
  __syncthreads();
  u64 before = inc - p - q;
  for (int w = 0; w < warp; ++w) before += s.wsum[w];
  if (2 * t < n) x[2 * t] = before + p;
  if (2 * t + 1 < n) x[2 * t + 1] = before + p + q;
  __syncthreads();
}

// How many of x[0 .. n), which do not fall, are below `need`; by every thread.
__device__ __forceinline__ int first_reaching(const u64 *x, int n, u64 need) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (x[mid] < need)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

template <typename T>
__global__ void __launch_bounds__(kSThreads, 2) sample_kernel(SampleArgs a) {
  using Key = typename Keys<T>::Key;
  constexpr int VE = 16 / sizeof(T);  // logits, and keys, of a vector
  extern __shared__ __align__(16) unsigned char raw[];
  SampleShared &s = *reinterpret_cast<SampleShared *>(raw);
  Key *keys = reinterpret_cast<Key *>(raw + sizeof(SampleShared));  // [slice], 0 behind the last id
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int cs = (int)gridDim.x, rank = (int)cluster_rank();
  const int lo = min(a.V, rank * a.slice), hi = min(a.V, lo + a.slice), n = hi - lo;
  const int vecs = a.slice / VE;  // (slices are multiples of 32)
  cluster_arrive_relaxed();  // waited for before the first remote store
  if (t < 256) s.table[t] = kExp2Table[t];
  if (t < 2) s.total[t] = 0u;
  grid_dependency_wait();
  allow_dependent_launch();
  int parity = 0, gathers = 0;
  auto clear = [&]() {
    for (int j = 4 * t; j < kSBins; j += 4 * kSThreads) {
      *reinterpret_cast<uint4 *>(&s.low[j]) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4 *>(&s.high[j]) = make_uint4(0u, 0u, 0u, 0u);
    }
  };
  clear();
  for (int m = blockIdx.y; m < a.M; m += gridDim.y, parity ^= 1) {  // same trip count in a cluster
    const T *x = static_cast<const T *>(a.logits) + (long long)m * a.logits_stride + lo;
    const float temp = a.r.temperature ? __ldca(a.r.temperature + m) : 1.f;
    const bool greedy = !(temp >= 1.1754943508222875e-38f);
    const int k = greedy ? 1 : a.r.top_k ? __ldca(a.r.top_k + m) : 0;
    const float p = !greedy && a.r.top_p ? __ldca(a.r.top_p + m) : 1.f;
    const float least = !greedy && a.r.min_p ? __ldca(a.r.min_p + m) : 0.f;
    const float u = __ldca(a.uniforms + m);
    if (t == kSThreads - 1) {  // (one thread: all of them would take 4 us for it)
      const double c = 1.4426950408889634074 / (double)(greedy ? 1.f : temp);
      s.rate[0] = (float)c;
      s.rate[1] = (float)(c - (double)(float)c);
    }
    // ---- the slice's logits ----
    unsigned most = 0u;
    if ((reinterpret_cast<uintptr_t>(x) & 15u) == 0u) {
      for (int j = t; j < vecs; j += kSThreads) {
        Vec<Key, VE> kv;
        if (j * VE + VE <= n) {
          const Vec<T, VE> v = vec_load<T, VE>(x + j * VE);
#pragma unroll
          for (int e = 0; e < VE; ++e) kv.e[e] = Keys<T>::of(v.e[e]);
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) kv.e[e] = j * VE + e < n ? Keys<T>::of(x[j * VE + e]) : (Key)0;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) most = max(most, (unsigned)kv.e[e]);
        *reinterpret_cast<Vec<Key, VE> *>(keys + j * VE) = kv;
      }
    } else {
      for (int j = t; j < a.slice; j += kSThreads) {
        const Key key = j < n ? Keys<T>::of(x[j]) : (Key)0;
        keys[j] = key;
        most = max(most, (unsigned)key);
      }
    }
    const unsigned own_most = most;
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s.wcount[warp] = most;
    __syncthreads();
    if (m == (int)blockIdx.y) cluster_wait();  // every block runs
    if (t < cs) {
      unsigned w = 0u;
      for (int j = 0; j < kSThreads / 32; ++j) w = max(w, s.wcount[j]);
      st_dsmem_s32(dsmem_addr(&s.top[parity][rank], t), (int)w);
    }
    cluster_sync_all();
    unsigned top = 0u;
    for (int r = 0; r < cs; ++r) top = max(top, s.top[parity][r]);
    if (top == 0u) {  // nothing above -inf
      if (rank == 0 && t == 0) {
        if (a.ids) a.ids[m] = 0;
        if (a.token_probs) a.token_probs[m] = 0.f;
      }
      if (a.probs)
        for (int j = t; j < n; j += kSThreads) a.probs[(long long)m * a.probs_stride + lo + j] = 0.f;
      __syncthreads();  // the keys may be replaced
      continue;
    }
    const Weigher<T> weigh{Keys<T>::logit(top), s.rate[0], s.rate[1], s.table};
    // ---- min-p: a weight that is kept at the least ----
    const u64 floor_w = least > 0.f ? (least >= 1.f ? 1ull << 44 : [&] {
      bool left;
      const u64 w = share_of(least, 1ull << 44, left);
      return w + (left ? 1ull : 0ull);
    }()) : 0ull;
    // ---- the last logit that is kept, and how many tokens that equal it ----
    // The bin of a key by its distance from the top, the largest bin nearest; the least bin
    // holds all from 32 units down.  (Rounding keeps the order, so bins fall as keys do.)
    const float x_top = Keys<T>::logit(top);
    const float per_unit = fminf(64.f / (greedy ? 1.f : temp), 1e30f);
    auto near_bin = [&](unsigned key) {
      return kSBins - 1 - (int)fminf((x_top - Keys<T>::logit(key)) * per_unit, (float)(kSBins - 1));
    };
    // The least key of a bin or a higher one (1 or more); by a warp, 32 looks at a time.
    auto first_key = [&](int bin) {
      unsigned low = 1u, high = top;  // of [low, high], high's bin is the largest
      while (low < high) {
        const unsigned step = (high - low) / 32u + 1u;
        const unsigned at = min(high, low + step * (unsigned)lane + (step - 1u));  // the end of a part
        const unsigned hit = __ballot_sync(0xffffffffu, near_bin(at) >= bin);      // (lane 31's at the least)
        const int part = __ffs(hit) - 1;
        const unsigned end = min(high, low + step * (unsigned)part + (step - 1u));
        low += step * (unsigned)part;
        high = end;
        if (step == 1u) break;
      }
      return high;
    };
    // Amounts by bin, summed over the cluster, of the keys from `least_key` up: by distance
    // (pass < 0), or by digit `pass` of those whose higher digits are `prefix`.
    auto pass_over = [&](bool weights, int pass, unsigned prefix, unsigned least_key) {
      const int shift = pass < 0 ? 0 : Keys<T>::shift(pass), above = pass <= 0 ? 31 : Keys<T>::shift(pass - 1);
      auto bin_of = [&](unsigned key) {  // negative: not of this pass
        if (key < least_key || (pass > 0 && (key >> above) != prefix)) return -1;
        if (pass < 0) return near_bin(key);
        return (int)((key >> shift) & ((pass == 0 ? kSBins : 1u << (above - shift)) - 1u));
      };
      if (weights) {  // (key by key: the code of a weight is long)
#pragma unroll 2
        for (int j = t; j < a.slice; j += kSThreads) {
          const unsigned key = keys[j];
          const int bin = bin_of(key);
          if (bin < 0) continue;
          const u64 w = weigh(key);
          const unsigned wl = (unsigned)w, old = atomicAdd(&s.low[bin], wl);
          const unsigned carry = (unsigned)(w >> 32) + (old + wl < old ? 1u : 0u);
          if (carry) atomicAdd(&s.high[bin], carry);
        }
      } else {
        for (int j = t; j < vecs; j += kSThreads) {
          const Vec<Key, VE> v = *reinterpret_cast<const Vec<Key, VE> *>(keys + j * VE);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const int bin = bin_of(v.e[e]);
            if (bin >= 0) atomicAdd(&s.low[bin], 1u);
          }
        }
      }
      cluster_sync_all();  // every block's amounts are there
      sum_bins(s, rank, cs);
      cluster_sync_all();  // the row's are in every block
      clear();
    };
    unsigned thr = 0u, kept = 0u;  // (nothing equals key 0)
    u64 cut_off = 0ull;            // weight of the tokens that equal thr and are not kept
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.f;
    const bool near = x_top < __uint_as_float(0x7f800000u);  // (from +inf there is no distance)
    // p times the weight of what top-k keeps, rounded up; one token at the least
    auto p_need = [&](u64 all) {
      bool left = false;
      const u64 w = p > 0.f ? share_of(p, all, left) : 0ull;
      return max(w + (left ? 1ull : 0ull), 1ull);
    };
    // Sends to block 0 the keys from `least_key` up in bin `bin` of the distances, and
    // above it where `whole`.  All blocks call it, after find_bin() (settled: and after a
    // barrier of the cluster).
    auto gather = [&](int bin, bool whole, unsigned least_key, bool settled) {
      if (!settled) cluster_arrive_release();  // this block is done with the row's amounts
      if (t == 0) s.sent = 0u;
      __syncthreads();
      const unsigned from = max(least_key, first_key(bin));
      const unsigned upto = whole || bin == kSBins - 1 ? top : first_key(bin + 1) - 1u;
      for (int j = t; j < vecs; j += kSThreads) {
        const Vec<Key, VE> v = *reinterpret_cast<const Vec<Key, VE> *>(keys + j * VE);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const unsigned key = v.e[e];
          if (key >= from && key <= upto) {
            const unsigned i = atomicAdd(&s.sent, 1u);
            if (i < (unsigned)kSMost) s.out[i] = (u64)key << 32 | (unsigned)~(lo + j * VE + e);
          }
        }
      }
      __syncthreads();
      if (!settled) cluster_wait_acquire();  // and so is block 0
      const unsigned sent = s.sent;
      if (t == 0 && sent) s.cut = (int)atom_dsmem_add(dsmem_addr(&s.total[gathers & 1], 0), sent);
      __syncthreads();
      const unsigned at = (unsigned)s.cut;
      for (unsigned j = t; j < min(sent, (unsigned)kSMost); j += kSThreads)
        if (at + j < (unsigned)kSMost) st_dsmem_u64(dsmem_addr(&s.item[at + j], 0), s.out[j]);
      cluster_sync_all();  // block 0 has them
      clear();             // (the amounts' place)
      ++gathers;
      if (t == 0) s.total[gathers & 1] = 0u;  // of the gather after this one
    };
    // Block 0: its n tokens in falling order, and the sums of their weights.
    auto sort_items = [&](int n, bool weights) {
      __syncthreads();
      sort_falling(s.item, n);
      if (weights) {
        for (int i = t; i < n; i += kSThreads) s.weight[i] = weigh((unsigned)(s.item[i] >> 32));
        __syncthreads();
        running_sums(s, s.weight, n);
      }
    };
    // How many of the sorted tokens [from, to) have this key; by block 0.
    auto equal_in = [&](int from, int to, unsigned key) {
      int c = 0;
      for (int i = from + t; i < to; i += kSThreads) c += (unsigned)(s.item[i] >> 32) == key;
      c = __reduce_add_sync(0xffffffffu, c);
      if (t == 0) s.sent = 0u;
      __syncthreads();
      if (lane == 0 && c) atomicAdd(&s.sent, (unsigned)c);
      __syncthreads();
      const unsigned r = s.sent;
      __syncthreads();
      return r;
    };
    // Block 0 tells all (it alone gives the values); by all blocks.
    auto tell = [&](unsigned key, unsigned count, u64 cut) {
      if (rank == 0 && t < cs) {
        st_dsmem_s32(dsmem_addr(&s.found_key, t), (int)key);
        st_dsmem_s32(dsmem_addr(&s.found_kept, t), (int)count);
        st_dsmem_u64(dsmem_addr(&s.found_cut, t), cut);
      }
      cluster_sync_all();
      thr = s.found_key;
      kept = s.found_kept;
      cut_off = s.found_cut;
    };
    bool k_open = by_k, p_open = by_p;
    if (by_k && k == 1) {
      thr = top;
      kept = 1u;
      k_open = p_open = false;
    }
    if (k_open && near) {
      // Where this block alone has k maxima of its threads' tokens, the k-th of those is at
      // most the row's k-th logit: what lies in lower bins than it need not be counted.
      // (Each count is a shared-memory atomic on a place of its own, some 17 cycles a warp.
      // For larger k the maxima of vectors bound it too, but cost more than they spare: one row
      // of 152,064, k = 300 26.3 us with them, 24.4 without.)
      const bool by_thread = 2 * k <= kSThreads;
      int bound = 0;
      if (by_thread) {
        if (own_most) atomicAdd(&s.low[near_bin(own_most)], 1u);
        __syncthreads();
        find_bin<true>(s, [&](u64) { return (u64)k; });
        bound = max(s.bin, 0);
        __syncthreads();
        clear();
      }
      bool have = false, whole = false;  // block 0 has the tokens that matter: all of them from a bin up
      int n = 0;
      u64 before = 0ull;
      if (by_thread && k * cs <= kSMost) {
        // Few tokens reach the largest of the blocks' bounds (some 10 a block for k = 20, 40 for
        // 50): they go to block 0 at once, without counts of the whole row.
        if (t < cs) st_dsmem_s32(dsmem_addr(&s.bound[rank], t), bound);
        cluster_sync_all();
        for (int r = 0; r < cs; ++r) bound = max(bound, s.bound[r]);
        if (bound > 0) {
          gather(bound, true, 1u, true);
          n = (int)min((unsigned)ld_dsmem_s32(dsmem_addr(&s.total[(gathers - 1) & 1], 0)), (unsigned)kSMost + 1u);
          have = whole = n <= kSMost;
          // (128 and less are sorted as they are.  One row of 152,064, k = 20 and 50: 12.0 and 12.6
          // us from 65 or from 129 on, 14.6 and 12.7 from 257 on, 14.7 and 18.5 never.)
          if (have && rank == 0 && n > 128) {  // those of the bins above the k-th's and of its own
            const u64 v0 = t < n ? s.item[t] : 0ull, v1 = t + kSThreads < n ? s.item[t + kSThreads] : 0ull;
            __syncthreads();  // (the counts' place is clear)
            const int b0 = v0 ? near_bin((unsigned)(v0 >> 32)) : -1, b1 = v1 ? near_bin((unsigned)(v1 >> 32)) : -1;
            if (b0 >= 0) atomicAdd(&s.low[b0], 1u);
            if (b1 >= 0) atomicAdd(&s.low[b1], 1u);
            if (t == 0) s.sent = 0u;
            __syncthreads();
            find_bin<true>(s, [&](u64) { return (u64)k; });
            const int bin = s.bin;
            n = (int)(s.before + s.inside);
            if (b0 >= bin) s.item[atomicAdd(&s.sent, 1u)] = v0;
            if (b1 >= bin) s.item[atomicAdd(&s.sent, 1u)] = v1;
            __syncthreads();
            clear();
          }
        }
      }
      if (!have) {
        __syncthreads();  // the counts' place is clear
        pass_over(false, -1, 0u, bound > 0 ? first_key(bound) : 1u);
        find_bin(s, [&](u64) { return (u64)k; });
        const int bin = s.bin;
        const u64 inside = s.inside;
        before = s.before;
        if (bin < 0) {  // fewer tokens than k
          k_open = false;
        } else if (bin > 0 && inside <= (u64)kSMost) {
          have = true;
          whole = before + inside <= (u64)kSMost;
          n = (int)(whole ? before + inside : inside);
          gather(bin, whole, 1u, false);
        }
      }
      if (have) {
        k_open = false;
        unsigned key = 0u, count = 0u;
        u64 cut = 0ull;
        if (whole && !a.probs) {
          if (rank == 0) {  // the rest of the row is block 0's
            sort_items(n, true);
            int c = k;
            if (by_p) c = min(c, first_reaching(s.weight, c, p_need(s.weight[c - 1])) + 1);
            int heavy = 0;
            for (int i = t; i < c; i += kSThreads)
              heavy += s.weight[i] - (i ? s.weight[i - 1] : 0ull) >= floor_w;
            heavy = __reduce_add_sync(0xffffffffu, heavy);
            if (t == 0) s.sent = 0u;
            __syncthreads();
            if (lane == 0 && heavy) atomicAdd(&s.sent, (unsigned)heavy);
            __syncthreads();
            c = (int)s.sent;
            const u64 total = s.weight[c - 1];
            // the kept ones in the order of ids, with the sums of their weights
            for (int i = t; i < c; i += kSThreads) s.out[i] = s.item[i] << 32 | (unsigned)i;
            __syncthreads();
            sort_falling(s.out, c);
            for (int i = t; i < c; i += kSThreads) {
              const int r = (int)(unsigned)s.out[i];
              s.item[i] = s.weight[r] - (r ? s.weight[r - 1] : 0ull);
            }
            __syncthreads();
            running_sums(s, s.item, c);
            bool left;
            u64 mark = !(u > 0.f) ? 0ull : u < 1.f ? share_of(u, total, left) : total - 1ull;
            if (mark >= total) mark = total - 1ull;
            const int i = first_reaching(s.item, c, mark + 1ull);
            if (t == 0) {
              const u64 w = s.item[i] - (i ? s.item[i - 1] : 0ull);
              if (a.ids) a.ids[m] = (int)~(unsigned)(s.out[i] >> 32);
              if (a.token_probs) a.token_probs[m] = Divider(total)(w);
            }
            __syncthreads();
            clear();
          }
          __syncthreads();  // the keys may be replaced
          continue;
        }
        if (rank == 0) {
          sort_items(n, whole);
          int c = whole ? k : (int)((u64)k - before);
          if (whole && by_p) c = min(c, first_reaching(s.weight, c, p_need(s.weight[c - 1])) + 1);
          key = (unsigned)(s.item[c - 1] >> 32);
          count = equal_in(0, c, key);
          // (all that equal the key lie in the bin)
          if (!whole) cut = equal_in(c, n, key) * weigh(key);
        }
        tell(key, count, cut);
        if (whole) p_open = false;
      }
    }
    if (k_open) {  // digit by digit
      unsigned prefix = 0u, need = (unsigned)k;
      bool reached = true;
      u64 ties = 0ull;
      for (int pass = 0; pass < Keys<T>::kPasses && reached; ++pass) {
        pass_over(false, pass, prefix, 1u);
        find_bin(s, [&](u64) { return (u64)need; });
        reached = s.bin >= 0;  // (else fewer tokens than k)
        if (reached) {
          need -= (unsigned)s.before;
          ties = s.inside;
          prefix = pass == 0 ? (unsigned)s.bin
                             : prefix << (Keys<T>::shift(pass - 1) - Keys<T>::shift(pass)) | (unsigned)s.bin;
        }
      }
      if (reached) {
        thr = prefix;
        kept = need;
        cut_off = (ties - need) * weigh(thr);
      }
    }
    if (p_open && near) {
      pass_over(true, -1, 0u, max(thr, 1u));
      u64 need = 0ull;
      find_bin(s, [&](u64 all) { return need = p_need(all - cut_off); });
      const int bin = s.bin;
      const u64 before = s.before;
      if (bin > 0) {
        gather(bin, false, max(thr, 1u), false);
        const unsigned n = (unsigned)ld_dsmem_s32(dsmem_addr(&s.total[(gathers - 1) & 1], 0));
        if (n <= (unsigned)kSMost) {
          p_open = false;
          unsigned key = 0u, count = 0u;
          if (rank == 0) {
            sort_items((int)n, true);
            const int c = first_reaching(s.weight, (int)n, need - before) + 1;
            key = (unsigned)(s.item[c - 1] >> 32);
            count = equal_in(0, c, key);
          }
          tell(key, count, 0ull);
        }
      }
    }
    if (p_open) {
      unsigned prefix = 0u;
      u64 need = 0ull;
      const unsigned least_key = max(thr, 1u);
      for (int pass = 0; pass < Keys<T>::kPasses; ++pass) {
        pass_over(true, pass, prefix, least_key);
        find_bin(s, [&](u64 all) {
          if (pass == 0) need = p_need(all - cut_off);
          return need;
        });
        need -= s.before;
        prefix = pass == 0 ? (unsigned)s.bin
                           : prefix << (Keys<T>::shift(pass - 1) - Keys<T>::shift(pass)) | (unsigned)s.bin;
      }
      thr = prefix;
      const u64 w = weigh(thr);
      kept = (unsigned)((need + w - 1ull) / w);
    }
    const u64 thr_w = thr ? weigh(thr) : 0ull;
    if (thr_w < floor_w) kept = 0u;
    // ---- this block's share: a run of ids a thread ----
    const int run = ((n + kSThreads - 1) / kSThreads) | 1;  // (odd: no bank conflicts)
    const int j0 = min(n, t * run), j1 = min(n, j0 + run);
    u64 above = 0ull;
    unsigned ties = 0u;
#pragma unroll 2
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
      s.wsum[warp] = ai;
      s.wcount[warp] = ci;
    }
    __syncthreads();
    u64 ab = ai - above, atot = 0ull;  // before this thread, of the block
    unsigned cb = ci - ties, ctot = 0u;
    for (int w = 0; w < kSThreads / 32; ++w) {
      if (w < warp) {
        ab += s.wsum[w];
        cb += s.wcount[w];
      }
      atot += s.wsum[w];
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
          if (a.token_probs) a.token_probs[m] = Divider(total)(w);
        }
        at += w;
      }
    }
    if (a.probs) {
      __syncthreads();  // cut is there
      // ties up to position `cut` of the slice are kept; all of them where the last kept
      // one lies in a later block
      const int cut = s.cut >= 0 ? s.cut : seen_first + ctot <= kept ? n : -1;
      const Divider share(total);
      float *to = a.probs + (long long)m * a.probs_stride + lo;
      auto prob = [&](int j, unsigned key) {
        u64 w = 0ull;
        if (key > thr) {
          w = weigh(key);
          if (w < floor_w) w = 0ull;
        } else if (key == thr && key && j <= cut) {
          w = kept ? thr_w : 0ull;
        }
        return w ? share(w) : 0.f;
      };
      if ((reinterpret_cast<uintptr_t>(to) & 15u) == 0u) {
        for (int j = 4 * t; j < n; j += 4 * kSThreads) {
          const Vec<Key, 4> v = *reinterpret_cast<const Vec<Key, 4> *>(keys + j);
          Vec<float, 4> o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o.e[e] = prob(j + e, v.e[e]);
          if (j + 4 <= n) {
            vec_store<float, 4>(to + j, o);
          } else {
            for (int e = 0; j + e < n; ++e) to[j + e] = o.e[e];
          }
        }
      } else {
        for (int j = t; j < n; j += kSThreads) to[j] = prob(j, keys[j]);
      }
    }
    __syncthreads();  // the keys may be replaced
  }
  // Where a small k sent the tokens to block 0 at once, every block has read their number there
  // with no barrier behind it; a cluster barrier follows every other access to another block's
  // memory.  No block leaves before all have read.  (Block 0, which finishes such a row, is last.)
  cluster_sync_all();
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
  auto bytes_of = [&](int k) {
    return (long long)sizeof(SampleShared) + (long long)sizeof(typename Keys<T>::Key) * slice_of(k);
  };
  // The largest cluster whose clusters for all M rows are resident at once, with
  // slices of 2048 ids or more; where none is, the smallest whose slices fit.
  // Slices, us at least 512, 1024, 2048, 4096, 8192 ids under top-p 0.9: one row of 9000
  // 15.3, 14.5, 15.9, 19.1, 25.1, of 32,001 17.1, 17.1, 18.7, 23.2, 34.1; nine of 32,001
  // 23.3, 23.3, 19.5, 24.4, 35.9.
  // More rows than are resident: few large blocks keep more of the SM's shared memory busy
  // where the vocabulary lets two a block be, and lose where a block takes an SM for itself.
  // us by the rule and by clusters of 8, 152,064 in float32, top-p 0.95, a top-k for every
  // other row: 36 rows 64 and 64, 38 83 and 66, 64 136 and 102, 128 212 and 171; top_k 50
  // for all: 38 35 and 30, 128 92 and 78; in bfloat16 without a top-k: 38 107 and 95, 64 110
  // and 127, 100 253 and 186; 32,001 in bfloat16: 38 35 and 41, 64 37 and 54, 128 55 and 100.
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
