// paged_decode.cu -- attention of single tokens (and of the few tokens whose
// rows with all G query heads are 16 at most) over a paged KV cache.
//
// Bound: HBM, which has to deliver every live K and V row once.  Mathematics,
// units and ranges as in paged_attention.cu.  Two kernels around the same
// block: one equal range of the line of cost rows a block, or, where no unit
// is long, a cluster of blocks a unit.
//
// Block: 4 consumer warps of the same 16 rows (the keys are split over the
// warps, each with a ring of stages: K and V of one tile) and 4 producer
// warps, one a ring (tensor-map copies of 16 rows, each looked up in the page
// table).  Producers run ahead over the ends of units, so the copies go on
// while the consumers join a unit's four states in shared memory and write
// the output or a partial.
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

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "kvs_paged.cuh"
#include "kvs_rows_mma.cuh"
#include "kvs_tags.cuh"
#include "kvs_tma.cuh"

namespace kvs {

namespace {

constexpr int kDW = 4;     // rings: consumer and producer warps
constexpr int kDRows = 16; // rows of a unit
constexpr int kDThreads = 2 * kDW * 32;
// A unit's fixed price (its start, the joining of its four states, its output)
// in bytes of K and V: 32 sequences of up to 8192 keys, H 32 / 8, D 128,
// bfloat16, took 104 us at 32 KB, 98 at 96, 94 at 128, 92.7 at 192, 93.0 at
// 256; 32 of up to 4500 62, 55, 48.6, 45.6 and 44.7 us (float32: 134, 123,
// 121, 123, 125).
constexpr int kDFixBytes = 192 << 10;
constexpr int kDMaxDevices = 64;
// Rules for clusters: the K and V bytes of a block, and those of a unit that
// halves the block, all counted as if every page of a table were in use.
constexpr long long kDBlockBytes = 1 << 20;
constexpr long long kDShortBytes16 = 512 << 10;
constexpr long long kDShortBytes32 = 128 << 10;

template <typename T, int D_, int W_>
struct DGeo {
  static constexpr int W = W_;                         // rings: consumer and producer warps
  static constexpr int D = D_;
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int KT = WarpRows<T, D>::KT;        // keys of a tile
  static constexpr int GB = 16 * D * (int)sizeof(T);   // bytes of a 16-row copy
  static constexpr int BLK = 2048;                     // one of its column blocks
  static constexpr int TILE = KT / 16 * GB;            // K (or V) of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int THREADS = 2 * W * 32;
  static constexpr int STATE = W * 16 * (D + 4) * 4;  // the consumers' accumulators
  static constexpr int BUDGET = (W == 4 ? 227 : 113) * 1024 - 2048 - STATE;
  static constexpr int S0 = BUDGET / (W * STAGE);
  static constexpr int S = S0 > 8 ? 8 : S0;            // stages of a ring
  static constexpr int OFF_STATE = W * S * STAGE;
  static constexpr int OFF_ML = OFF_STATE + STATE;     // float2 [W][16]
  static constexpr int OFF_BAR = OFF_ML + W * 16 * 8;
  static constexpr int OFF_BAD = OFF_BAR + (2 * W * S + 1) * 8;  // int [W][S]
  static constexpr int OFF_MISC = OFF_BAD + W * S * 4;           // abort, last
  static constexpr int SMEM = OFF_MISC + 8;
  static_assert(S >= 2, "two stages at least");
  static_assert(SMEM <= (W == 4 ? 227 : 113) * 1024, "one block per SM must fit");
};

// The barriers and bookkeeping of a block's rings.
struct Rings {
  uint64_t *full, *empty;  // [W][S]
  int *bad;                // [W][S] the stage's tile has a bad page
  volatile int *abort;
  unsigned char *smem;
};

// Fills a ring with its tiles of [t_lo, t_hi) (tile t goes to ring (t - t_lo) %
// W); by one warp.  n: tiles put in the ring so far.
template <typename T, int D, int W, bool kPoll>
__device__ __forceinline__ bool fill_ring(const Rings &rg, const PagedArgs &pa,
                                          const CUtensorMap *kmap, const CUtensorMap *vmap, int ring,
                                          int i, int g, int Hkv, int t_lo, int t_hi, int keys,
                                          uint32_t &n, uint64_t policy, int *d_status) {
  using C = DGeo<T, D, W>;
  constexpr int NP = C::KT / 16;  // 16-row pieces of a tile
  constexpr int AHEAD = 32 / NP;  // tiles whose pages one look-up finds
  const int lane = threadIdx.x & 31;
  const int piece = lane % NP;    // lanes 0..NP-1: K pieces, NP..2NP-1: V pieces
  const int32_t *table = pa.page_table + (size_t)i * pa.max_pages;
  int page = 0, k = 0;  // lane: the page of piece `piece` of the ring's tile k + lane / NP
  for (int t = t_lo + ring; t < t_hi; t += W, ++n, ++k) {
    if (k % AHEAD == 0) {
      const long long r0 = (long long)(t + W * (lane / NP)) * C::KT + 16 * piece;
      page = r0 < keys ? __ldca(table + (r0 >> pa.page_shift)) : 0;
    }
    const int pg = __shfl_sync(0xffffffffu, page, (k % AHEAD) * NP + piece);
    const int npieces = min(NP, (keys - t * C::KT + 15) / 16);
    const bool mine = lane < 2 * NP && piece < npieces;
    const bool wrong = mine && (unsigned)pg >= (unsigned)pa.num_pages;
    const unsigned any_bad = __ballot_sync(0xffffffffu, wrong);
    const int st = ring * C::S + (int)(n % C::S);
    if (!__all_sync(0xffffffffu,
                    mbar_wait<kPoll>(&rg.empty[st], ((n / C::S) & 1u) ^ 1u, rg.abort)))
      return false;
    if (lane == 0) {
      rg.bad[st] = any_bad != 0u;
      if (any_bad) record_status(d_status, KVS_ERR_PAGE);
      mbar_arrive_expect_tx(&rg.full[st], 2u * (uint32_t)npieces * C::GB);
    }
    __syncwarp();
    if (mine) {
      const int r0 = t * C::KT + 16 * piece;
      const int row = ((wrong ? 0 : pg) * Hkv + g) * (1 << pa.page_shift) +
                      (r0 & ((1 << pa.page_shift) - 1));
      unsigned char *dst = rg.smem + st * C::STAGE + (lane >= NP ? C::TILE : 0) + piece * C::GB;
      tma_rows(dst, lane >= NP ? vmap : kmap, row, &rg.full[st], policy);
    }
  }
  return true;
}

// Every copy of a ring lands before the block exits (one thread).
template <typename T, int D, int W>
__device__ __forceinline__ void drain_ring(const Rings &rg, int ring, uint32_t n) {
  using C = DGeo<T, D, W>;
  for (uint32_t j = n > (uint32_t)C::S ? n - C::S : 0u; j < n; ++j)
    mbar_wait_drain(&rg.full[ring * C::S + j % C::S], (j / C::S) & 1u);
}

// The ring's tiles of [t_lo, t_hi) against the warp's rows; n as in
// fill_ring.  False when a wait ran out; poison: a bad page was among them.
template <typename T, int D, int W, bool kPoll, bool kFew>
__device__ __forceinline__ bool consume_tiles(WarpRows<T, D> &w, const Rings &rg, int ring, int t_lo,
                                             int t_hi, int keys, const int (&reach)[2], float sl2,
                                             uint32_t &n, bool &poison) {
  using C = DGeo<T, D, W>;
  const int lane = threadIdx.x & 31;
  for (int t = t_lo + ring; t < t_hi; t += W, ++n) {
    const int st = ring * C::S + (int)(n % C::S);
    if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&rg.full[st], (n / C::S) & 1u, rg.abort)))
      return false;
    poison |= rg.bad[st] != 0;
    unsigned char *sk = rg.smem + st * C::STAGE;
    const int left = keys - t * C::KT;  // keys of the tile that exist
    if (left < C::KT) {
      // rows past the last key hold anything: V's become zero (their weights
      // are zero, but 0 x NaN is not)
      for (int e = lane; e < (C::KT - left) * (D * (int)sizeof(T) / 16); e += 32) {
        const int row = left + e % (C::KT - left), pc = e / (C::KT - left);
        *reinterpret_cast<uint4 *>(sk + C::TILE + (row >> 4) * C::GB + (pc >> 3) * C::BLK +
                                   (row & 15) * 128 + (pc & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_shared();
      __syncwarp();
    }
    const int lim[2] = {reach[0] - t * C::KT, reach[1] - t * C::KT};
    w.template tile<kFew>(smem_addr(sk), smem_addr(sk + C::TILE), sl2, lim);
    __syncwarp();
    if (lane == 0) mbar_arrive(&rg.empty[st]);
  }
  return true;
}

// The same for a unit of `rows` rows, with the row sums finished.
template <typename T, int D, int W, bool kPoll>
__device__ __forceinline__ bool consume_ring(WarpRows<T, D> &w, const Rings &rg, int ring, int rows,
                                             int t_lo, int t_hi, int keys, const int (&reach)[2],
                                             float sl2, uint32_t &n, bool &poison) {
  bool ok;
  if (!std::is_same<T, float>::value && rows <= 8) {
    constexpr bool kFew = !std::is_same<T, float>::value;
    ok = consume_tiles<T, D, W, kPoll, kFew>(w, rg, ring, t_lo, t_hi, keys, reach, sl2, n, poison);
    w.template finish<kFew>();
  } else {
    ok = consume_tiles<T, D, W, kPoll, false>(w, rg, ring, t_lo, t_hi, keys, reach, sl2, n, poison);
    w.finish();
  }
  return ok;
}

// A warp's state into shared memory: [16][D + 4] accumulators, [16] (m, l).
template <typename T, int D>
__device__ __forceinline__ void put_state(const WarpRows<T, D> &w, float *acc, float2 *ml) {
  const int lane = threadIdx.x & 31;
  w.each([&](int hh, int d, const float(&v)[4]) {
    float *p = acc + (lane / 4 + 8 * hh) * (D + 4) + d;
    if constexpr (std::is_same<T, float>::value)
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  });
  if ((lane & 3) == 0) {
    ml[lane / 4] = make_float2(w.m[0], w.l[0]);
    ml[lane / 4 + 8] = make_float2(w.m[1], w.l[1]);
  }
}

// Columns d .. d + 3 of row r joined over the W warps' states.
template <int D, int W>
__device__ __forceinline__ void join_states(const float *acc0, const float2 *ml0, int r, int d,
                                            float4 &acc, float &mx, float &ls) {
  mx = neg_inf_f();
#pragma unroll
  for (int k = 0; k < W; ++k) mx = fmaxf(mx, ml0[k * 16 + r].x);
  const float mz = mx == neg_inf_f() ? 0.f : mx;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  ls = 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const float2 ml = ml0[k * 16 + r];
    const float wgt = ex2f(ml.x - mz);
    const float4 v = *reinterpret_cast<const float4 *>(acc0 + (k * 16 + r) * (D + 4) + d);
    acc.x = fmaf(wgt, v.x, acc.x);
    acc.y = fmaf(wgt, v.y, acc.y);
    acc.z = fmaf(wgt, v.z, acc.z);
    acc.w = fmaf(wgt, v.w, acc.w);
    ls = fmaf(wgt, ml.y, ls);  // (a NaN sum stays one also under a zero weight)
  }
}

template <typename T, int D, bool kPoll>
__global__ void __launch_bounds__(kDThreads, 1)
    paged_decode_kernel(const T *__restrict__ q, long long q_stride, T *__restrict__ out,
                        long long out_stride, PagedArgs pa,
                        const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int G, int Hkv, float sl2,
                        int min_column, unsigned char *ws, unsigned host_tag, int *d_status) {
  using C = DGeo<T, D, kDW>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [kDW][S]
  uint64_t *empty = full + kDW * C::S;
  uint64_t *cbar = empty + kDW * C::S;  // all consumer warps
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  volatile int *s_last = abort + 1;
  const Rings rg{full, empty, reinterpret_cast<int *>(smem + C::OFF_BAD), abort, smem};
  unsigned *epoch = reinterpret_cast<unsigned *>(ws);
  unsigned long long *counters = reinterpret_cast<unsigned long long *>(ws + 256);
  float *slots = reinterpret_cast<float *>(ws + 256 + (size_t)kPagedMaxBlocks * 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const Line ln{Hkv, kDRows / G, kDFixBytes / (2 * D * (int)sizeof(T)), C::KT, min_column};
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int s = 0; s < kDW * C::S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(cbar, kDW);
    *abort = 0;
    *s_last = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  // bad sequences: status, and NaN rows where the rows are known
  for (int i = b; i < pa.M; i += gridDim.x) {
    const PagedSeq s = paged_seq(pa, i);
    if (s.err != KVS_OK) {
      if (threadIdx.x == 0) record_status(d_status, s.err);
      const T nan = from_f32<T>(__int_as_float(0x7fc00000));
      for (int r = 0; r < s.n; ++r)
        for (int e = threadIdx.x; e < Hkv * G * D; e += kDThreads)
          out[(long long)(s.row0 + r) * out_stride + e] = nan;
    }
  }
  const unsigned tag = launch_tag(host_tag, __ldcg(epoch));
  __syncthreads();
  allow_dependent_launch();
  const Cuts cut = equal_cuts(warp_line_total(pa, ln, lane), ln, gridDim.x);
  if (cut.R == 0 || b >= cut.NS) return;
  const long long x0 = cut.start(b), x1 = cut.start(b + 1);
  Unit u = warp_unit_at(pa, ln, x0, lane);

  if (warp >= kDW) {
    // ======================= producer of a ring ==============================
    const uint64_t policy = policy_evict_first();  // a row is read once
    const int ring = warp - kDW;
    uint32_t n = 0;
    bool ok = true;
    do {
      const UnitInfo f = unit_info(pa, u, ln, x0, x1);
      ok = fill_ring<T, D, kDW, kPoll>(rg, pa, &kmap, &vmap, ring, u.i, u.g, Hkv, f.t_lo, f.t_hi, f.keys,
                                  n, policy, d_status);
      if (!ok) break;
      if (!next_unit(pa, u, f, ln)) break;
    } while (u.base < x1);
    if (lane == 0) {
      if (!ok) give_up(abort, d_status, epoch);
      drain_ring<T, D, kDW>(rg, ring, n);
    }
    return;
  }

  // ========================= consumers ======================================
  uint32_t n = 0, cphase = 0;
  auto consumers_barrier = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(cbar);
    bool got = mbar_wait<kPoll>(cbar, cphase, abort);
    got = __all_sync(0xffffffffu, got);
    if (!got) {
      if (lane == 0) give_up(abort, d_status, epoch);
      return false;
    }
    cphase ^= 1u;
    return true;
  };
  const float nan = __int_as_float(0x7fc00000);
  WarpRows<T, D> w;
  do {
    const UnitInfo f = unit_info(pa, u, ln, x0, x1);
    if (f.t_lo < f.t_hi) {
      const int rows = f.ntok * G;
      w.start(q, q_stride, 0, rows, G, f, u.g);
      // keys that this lane's two rows attend
      int reach[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        reach[hh] = f.s.p + f.tok0 + min(lane / 4 + 8 * hh, rows - 1) / G + 1;
      bool poison = false;
      if (!consume_ring<T, D, kDW, kPoll>(w, rg, warp, rows, f.t_lo, f.t_hi, f.keys, reach, sl2, n,
                                         poison)) {
        if (lane == 0) give_up(abort, d_status, epoch);
        return;
      }
      if (poison) w.l[0] = w.l[1] = nan;
      const bool whole = f.t_hi - f.t_lo == f.nt;
      const size_t slot = 2 * (size_t)b + (f.t_lo == 0 ? 1 : 0);
      float *sl = slots + slot * paged_slot_floats(kDRows, D);
      float *sacc = sl + 2 * kDRows;
      T *orow = out + (long long)(f.s.row0 + f.tok0) * out_stride + (long long)u.g * G * D;
      // the key groups' states merge in shared memory
      float *macc = reinterpret_cast<float *>(smem + C::OFF_STATE);  // [kDW][16][D + 4]
      float2 *mml = reinterpret_cast<float2 *>(smem + C::OFF_ML);    // [kDW][16]
      put_state<T, D>(w, macc + warp * 16 * (D + 4), mml + warp * 16);
      if (!consumers_barrier()) return;
      for (int e = threadIdx.x; e < rows * (D / 4); e += kDW * 32) {
        const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
        float4 acc;
        float mx, ls;
        join_states<D, kDW>(macc, mml, r, d, acc, mx, ls);
        if (whole) {
          const float inv = 1.f / ls;
          const int tok = r / G;
          store4<T>(orow + (long long)tok * out_stride + (r - tok * G) * D + d,
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        } else {
          __stcg(reinterpret_cast<float4 *>(sacc + (size_t)r * D + d), acc);
          if (d == 0) __stcg(reinterpret_cast<float2 *>(sl) + r, make_float2(mx, ls));
        }
      }
      if (!whole) __threadfence();  // the partial is visible GPU-wide before it counts
      if (!consumers_barrier()) return;  // (also: the states may be written again)
      if (!whole) {
        // the blocks of the unit's first and last tile; every block between has some
        const int b1 = cut.at(f.k0);
        const int b2 = cut.at(f.k0 + (long long)(f.nt - 1) * C::KT);
        if (threadIdx.x == 0) {
          const unsigned add = (unsigned)(f.t_hi - f.t_lo);
          const unsigned before = tagged_add(counters + b1, add, tag, d_status, epoch);
          const bool last = before != 0xffffffffu && before + add == (unsigned)f.nt;
          if (last) counters[b1] = 0ull;  // a replayed graph uses the same tag again
          *s_last = last;
        }
        if (!consumers_barrier()) return;
        if (*s_last) {
          __threadfence();
          for (int e = threadIdx.x; e < rows * (D / 4); e += kDW * 32) {
            const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
            float4 acc;
            float ls;
            merge_pieces(slots, paged_slot_floats(kDRows, D), 2 * kDRows + r * D + d, r, b1, b2, acc, ls);
            const float inv = 1.f / ls;
            const int tok = r / G;
            store4<T>(orow + (long long)tok * out_stride + (r - tok * G) * D + d,
                      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
          }
        }
      }
    }
    if (!next_unit(pa, u, f, ln)) break;
  } while (u.base < x1);
}

// ---- a thread-block cluster a unit ----------------------------------------------
// grid (CS, M * Hkv), clusters of CS (1 to 16): block r of a cluster takes
// tiles [nt r / CS, nt (r + 1) / CS) of its (sequence, kv head).  No line of
// cost rows to walk, no partials in global memory and no counters: the
// blocks' states meet in distributed shared memory, where block r joins its
// share of the output elements.
//
// Measured against the equal ranges (us; H 32 / 8, D 128, float16, 16-key
// pages, replayed, so that up to 100 MB come from L2):
//   sequences x keys       1 x 256   1 x 4096   4 x 1024   32 x 2048   1 x 32768   8 x 32768
//   full cache a block       16 KB     256 KB     128 KB        1 MB        2 MB        8 MB
//   clusters                  5.2        7.7        6.5        46.5        26.8       158.7
//   equal ranges              9.9       13.2       11.1        49.2        32.8       163.5
//   lengths of 1/8 to all     9.5       13.4       11.0        31.5        25.3       125.9
//   the same, clusters        5.4        7.2        6.5        31.8        21.2       123.2
// A block reads about 45 KB/us, so 1 MB bounds what a call can lose by one
// long sequence among short ones at 20 us; past it the equal ranges run.
//
// With W = 2 rings a block, two blocks an SM: one starts and joins while the
// other streams.  For many short units: 128 x 256 keys, 8 kv heads 39.5 us
// (W = 4: 44.1), 256 x 128, one head 7.9 (9.7); but float32, whose products
// weigh more, 32 x 512, D 64 23.3 (19.4).
template <typename T, int D, int W, bool kPoll>
__global__ void __launch_bounds__(2 * W * 32, 4 / W)
    paged_decode_cluster_kernel(const T *__restrict__ q, long long q_stride, T *__restrict__ out,
                                long long out_stride, PagedArgs pa,
                                const __grid_constant__ CUtensorMap kmap,
                                const __grid_constant__ CUtensorMap vmap, int G, int Hkv, float sl2,
                                int *d_status) {
  using C = DGeo<T, D, W>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [W][S]
  uint64_t *empty = full + W * C::S;
  uint64_t *cbar = empty + W * C::S;  // all consumer warps
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  const Rings rg{full, empty, reinterpret_cast<int *>(smem + C::OFF_BAD), abort, smem};
  float *macc = reinterpret_cast<float *>(smem + C::OFF_STATE);  // [W][16][D + 4]
  float2 *mml = reinterpret_cast<float2 *>(smem + C::OFF_ML);    // [W][16]
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cs = (int)gridDim.x, rank = (int)cluster_rank();
  const int i = (int)blockIdx.y / Hkv, g = (int)blockIdx.y - i * Hkv;
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int s = 0; s < W * C::S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(cbar, W);
    *abort = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  const PagedSeq s = paged_seq(pa, i);
  __syncthreads();
  allow_dependent_launch();
  if (s.err != KVS_OK) {  // (the whole cluster leaves)
    if (threadIdx.x == 0) record_status(d_status, s.err);
    const T nan = from_f32<T>(__int_as_float(0x7fc00000));
    for (int r = rank; r < s.n; r += cs)
      for (int e = threadIdx.x; e < G * D; e += C::THREADS)
        out[(long long)(s.row0 + r) * out_stride + (long long)g * G * D + e] = nan;
    return;
  }
  if (s.n == 0) return;
  const int keys = s.p + s.n;
  const int nt = (keys + C::KT - 1) / C::KT;
  const int t_lo = (int)((long long)nt * rank / cs), t_hi = (int)((long long)nt * (rank + 1) / cs);
  const int rows = s.n * G;
  bool ok = true;
  uint32_t n = 0;
  if (warp >= W) {
    ok = fill_ring<T, D, W, kPoll>(rg, pa, &kmap, &vmap, warp - W, i, g, Hkv, t_lo, t_hi, keys, n,
                                policy_evict_first(), d_status);
    if (lane == 0) {
      if (!ok) {
        *abort = 1;
        record_status(d_status, KVS_ERR_TIMEOUT);
      }
      drain_ring<T, D, W>(rg, warp - W, n);
    }
  } else {
    WarpRows<T, D> w;
    UnitInfo f{};
    f.s = s;
    f.ntok = s.n;
    w.start(q, q_stride, 0, rows, G, f, g);
    int reach[2];  // keys that this lane's two rows attend
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) reach[hh] = s.p + min(lane / 4 + 8 * hh, rows - 1) / G + 1;
    bool poison = false;
    ok = consume_ring<T, D, W, kPoll>(w, rg, warp, rows, t_lo, t_hi, keys, reach, sl2, n, poison);
    if (poison) w.l[0] = w.l[1] = __int_as_float(0x7fc00000);
    put_state<T, D>(w, macc + warp * 16 * (D + 4), mml + warp * 16);
    __syncwarp();
    if (lane == 0) mbar_arrive(cbar);
    ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(cbar, 0u, abort)) && ok;
    if (!ok && lane == 0) {
      *abort = 1;
      record_status(d_status, KVS_ERR_TIMEOUT);
    }
    // the block's joined state over the first warp's (each thread rewrites
    // only elements it has read)
    for (int e = threadIdx.x; e < rows * (D / 4); e += W * 32) {
      const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
      float4 acc;
      float mx, ls;
      join_states<D, W>(macc, mml, r, d, acc, mx, ls);
      *reinterpret_cast<float4 *>(macc + r * (D + 4) + d) = acc;
      if (d == 0) *reinterpret_cast<float2 *>(smem + r * 8) = make_float2(mx, ls);
    }
  }
  // (every block of the cluster comes here, also when a wait ran out)
  cluster_sync_all();
  const int total = rows * (D / 4);
  const int e0 = (int)((long long)total * rank / cs), e1 = (int)((long long)total * (rank + 1) / cs);
  for (int e = e0 + (int)threadIdx.x; e < e1; e += C::THREADS) {
    const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
    float2 ml[16];
    float4 v[16];
    float mx = neg_inf_f();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < cs) {
        ml[k] = ld_dsmem_f2(dsmem_addr(smem + r * 8, k));
        v[k] = ld_dsmem_f4(dsmem_addr(macc + r * (D + 4) + d, k));
        mx = fmaxf(mx, ml[k].x);
      }
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < cs) {
        const float wgt = ex2f(ml[k].x - mx);  // (some block has attended keys: mx is finite)
        acc.x = fmaf(wgt, v[k].x, acc.x);
        acc.y = fmaf(wgt, v[k].y, acc.y);
        acc.z = fmaf(wgt, v[k].z, acc.z);
        acc.w = fmaf(wgt, v[k].w, acc.w);
        ls = fmaf(wgt, ml[k].y, ls);
      }
    }
    const float inv = 1.f / ls;
    const int tok = r / G;
    store4<T>(out + (long long)(s.row0 + tok) * out_stride + (long long)(g * G + r - tok * G) * D + d,
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
  cluster_sync_all();  // the other blocks have read this one's state
}

// Resident clusters of 2, 4, 8, 16 blocks on the device, by log2 - 1.
struct ClusterInfo {
  int active[4] = {0};
  bool configured = false;
};

template <typename T, int D, int W>
const ClusterInfo *cluster_info(int dev) {
  using C = DGeo<T, D, W>;
  static ClusterInfo info[kDMaxDevices];
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (!info[dev].configured) {
    ClusterInfo rec;
    int top = 4;
    for (auto kern : {paged_decode_cluster_kernel<T, D, W, false>, paged_decode_cluster_kernel<T, D, W, true>}) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
          cudaSuccess) {
        cudaGetLastError();
        return nullptr;
      }
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess) {
        cudaGetLastError();
        top = 3;
      }
    }
    for (int k = 1; k <= top; ++k) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1u << k, 1, 1);
      cfg.blockDim = dim3(C::THREADS, 1, 1);
      cfg.dynamicSmemBytes = C::SMEM;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1u << k;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, paged_decode_cluster_kernel<T, D, W, false>, &cfg) !=
          cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      rec.active[k - 1] = n;
    }
    rec.configured = true;
    info[dev] = rec;
  }
  return &info[dev];
}

template <typename T, int D, int W>
int launch_clusters(unsigned cs, const void *q, long long q_stride, const PagedArgs &pa, void *out,
                    long long out_stride, int G, int Hkv, float sl2, const CUtensorMap &kmap,
                    const CUtensorMap &vmap, int *d_status, cudaStream_t stream) {
  using C = DGeo<T, D, W>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, (unsigned)(pa.M * Hkv), 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, poll_waits() ? paged_decode_cluster_kernel<T, D, W, true>
                         : paged_decode_cluster_kernel<T, D, W, false>,
      static_cast<const T *>(q), q_stride, static_cast<T *>(out), out_stride,
      pa, kmap, vmap, G, Hkv, sl2, d_status);
  if (e != cudaSuccess) {
    cudaGetLastError();  // leave no stale error for the caller's next check
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

template <typename T, int D>
int launch_decode(const void *q, long long q_stride, const kvs_paged_cache &cache,
                  const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                  int *d_status, cudaStream_t stream) {
  using C = DGeo<T, D, kDW>;
  static bool configured[kDMaxDevices] = {false};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDMaxDevices)
    return KVS_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      for (auto kern : {paged_decode_kernel<T, D, false>,
                        paged_decode_kernel<T, D, true>}) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
            cudaSuccess) {
          cudaGetLastError();
          return KVS_ERR_LAUNCH;
        }
      }
      configured[dev] = true;
    }
  }
  const int sms = device_sm_count();
  if (sms <= 0) return KVS_ERR_LAUNCH;
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)cache.num_pages * cache.num_kv_heads * cache.page_size;
  int rc = make_row_map(&kmap, cache.k_pages, rows, D, cache.dtype, 16,
                        D * (int)sizeof(T) / 128);
  if (rc == KVS_OK) rc = make_row_map(&vmap, cache.v_pages, rows, D, cache.dtype, 16,
                        D * (int)sizeof(T) / 128);
  if (rc != KVS_OK) return rc;
  const int Hkv = cache.num_kv_heads;
  const int grid = sms < kPagedMaxBlocks ? sms : kPagedMaxBlocks;
  const float sl2 = (float)(1.4426950408889634074 / std::sqrt((double)D));
  // the shortest range worth a block: a step of 4 x 1500 keys, 2 kv heads, in
  // float32 took 16.2 us at 48 cost rows, 15.4 at 96, 16.5 at 192, 18.9 at 384
  const int min_column = 3 * 32;
  // Clusters where no block of theirs can have much to do even if every page
  // of the table is in use; else equal ranges, which stay even however the
  // lengths differ.
  const long long units = (long long)pa.M * Hkv;
  const long long unit_bytes = ((long long)pa.max_pages << pa.page_shift) * D * 2 * (long long)sizeof(T);
  const ClusterInfo *ci = cluster_info<T, D, kDW>(dev);
  if (!ci) return KVS_ERR_LAUNCH;
  int k = 4;  // clusters of 2^k blocks: all resident at once, no block without a tile
  while (k > 0 && (units > ci->active[k - 1] || unit_bytes < (long long)C::STAGE << k)) --k;
  if (units <= 65535 && unit_bytes <= kDBlockBytes << k) {
    if (units > sms && unit_bytes <= (C::F32 ? kDShortBytes32 : kDShortBytes16)) {
      if (!cluster_info<T, D, 2>(dev)) return KVS_ERR_LAUNCH;
      return launch_clusters<T, D, 2>(1, q, q_stride, pa, out, out_stride, H / Hkv, Hkv, sl2, kmap,
                                      vmap, d_status, stream);
    }
    return launch_clusters<T, D, kDW>(1u << k, q, q_stride, pa, out, out_stride, H / Hkv, Hkv, sl2,
                                      kmap, vmap, d_status, stream);
  }
  const cudaError_t e = launch_pdl(
      poll_waits() ? paged_decode_kernel<T, D, true>
                   : paged_decode_kernel<T, D, false>,
      dim3(grid), dim3(kDThreads), C::SMEM, stream, static_cast<const T *>(q), q_stride,
      static_cast<T *>(out), out_stride, pa, kmap, vmap, H / Hkv, Hkv, sl2, min_column,
      static_cast<unsigned char *>(workspace), fresh_tag(), d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
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
             ? launch_decode<T, 64>(q, q_stride, cache, pa, out, out_stride, H, workspace,      \
                                    d_status, stream)                                           \
             : launch_decode<T, 128>(q, q_stride, cache, pa, out, out_stride, H, workspace,     \
                                     d_status, stream)
  if (cache.dtype == KVS_F32) KVS_DECODE(float);
  if (cache.dtype == KVS_F16) KVS_DECODE(__half);
  KVS_DECODE(__nv_bfloat16);
#undef KVS_DECODE
}

}  // namespace kvs
