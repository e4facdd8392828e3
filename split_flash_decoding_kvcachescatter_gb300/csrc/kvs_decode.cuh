// kvs_decode.cuh -- attention of single tokens (and of the few tokens whose
// rows with all G query heads are 16 at most) over a paged KV cache: the two
// kernels and their launch, for the plain pages of paged_decode.cu and the
// 8-bit ones of paged_decode_q8.cu.
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
// the output or a partial.  Where a byte of the pages brings more products (8
// bits under few rows) 8 consumer warps, whose rings 4 producers fill two each
// and give registers to.
#pragma once

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

constexpr int kDRows = 16; // rows of a unit
// Registers a thread of a block with 8 consumer and 4 producer warps: at launch, and shares.
constexpr int kLaunchRegs = 168, kConsumerRegs = 208, kProducerRegs = 88;
static_assert(2 * kConsumerRegs + kProducerRegs == 3 * kLaunchRegs, "what the launch has");
constexpr int kDMaxDevices = 64;

// What a kernel of this file needs to know of the pages is its policy P: the type
// T of q and out, the head size D, the bytes kElem of an element of the pages, the
// warp's rows (WarpRows or a class like it), whether 16 keys share a scale
// (kScaled), the rings of a block where ranges are equal (kRings: as many consumer
// warps), whether units have 8 rows at most (kOnlyFew), and what a launch passes beside the
// tensor maps (Extra).
template <class P, int W_>
struct DGeo {
  static constexpr int W = W_;                         // rings: consumer and producer warps
  static constexpr int D = P::D;
  static constexpr int KT = P::Rows::KT;               // keys of a tile
  static constexpr int GB = 16 * D * P::kElem;         // bytes of a 16-row copy
  static constexpr int TILE = KT / 16 * GB;            // K (or V) of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int SCALES = P::kScaled ? 2 * KT / 16 * 4 : 0;  // bytes of a stage's scales
  static constexpr int PW = W > 4 ? W / 2 : W;        // producer warps
  static constexpr int THREADS = (W + PW) * 32;
  static constexpr int ROWS = P::kOnlyFew ? 8 : 16;   // of a unit
  static constexpr int STATE = W * ROWS * (D + 4) * 4;  // the consumers' accumulators
  static constexpr int BUDGET = (W >= 4 ? 227 : 113) * 1024 - 2048 - STATE;
  static constexpr int S0 = BUDGET / (W * (STAGE + SCALES));
  static constexpr int S = S0 > 8 ? 8 : S0;            // stages of a ring
  static constexpr int OFF_STATE = W * S * STAGE;
  static constexpr int OFF_ML = OFF_STATE + STATE;     // float2 [W][ROWS]
  static constexpr int OFF_SCALE = OFF_ML + W * ROWS * 8;  // float [W][S][2][KT / 16]
  static constexpr int OFF_BAR = OFF_SCALE + W * S * SCALES;
  static constexpr int OFF_BAD = OFF_BAR + (2 * W * S + 1) * 8;  // int [W][S]
  static constexpr int OFF_MISC = OFF_BAD + W * S * 4;           // abort, last
  static constexpr int SMEM = OFF_MISC + 8;
  static_assert(S >= 2, "two stages at least");
  static_assert(SMEM <= (W >= 4 ? 227 : 113) * 1024, "one block per SM must fit");
  // arrivals that fill a stage: the one that expects the copies, and with scales
  // each lane's, made when its part of them has landed
  static constexpr int FULL = P::kScaled ? 33 : 1;
};

// The barriers and bookkeeping of a block's rings.
struct Rings {
  uint64_t *full, *empty;  // [W][S]
  int *bad;                // [W][S] the stage's tile has a bad page
  volatile int *abort;
  unsigned char *smem;
};

// Fills the rings of producer `part` with their tiles of [t_lo, t_hi) (tile t goes to
// ring (t - t_lo) % W; a producer has ring `part`, or that and ring part + PW in turn); by
// one warp.  n: tiles put in each of them so far.
template <class P, int W, bool kPoll>
__device__ __forceinline__ bool fill_rings(const Rings &rg, const PagedArgs &pa,
                                          const typename P::Extra &extra,
                                          const CUtensorMap *kmap, const CUtensorMap *vmap, int part,
                                          int i, int g, int Hkv, int t_lo, int t_hi, int keys,
                                          uint32_t (&n)[2], uint64_t policy, int *d_status) {
  using C = DGeo<P, W>;
  constexpr int NP = C::KT / 16;  // 16-row pieces of a tile
  constexpr int AHEAD = 32 / NP;  // tiles whose pages one look-up finds
  const int lane = threadIdx.x & 31;
  const int piece = lane % NP;    // lanes 0..NP-1: K pieces, NP..2NP-1: V pieces
  const int32_t *table = pa.page_table + (size_t)i * pa.max_pages;
  constexpr int PW = C::PW;
  int page = 0, k = 0;  // lane: the page of piece `piece` of the producer's tile k + lane / NP
  for (int t = t_lo + part; t < t_hi; t += PW, ++k) {
    if (k % AHEAD == 0) {
      const long long r0 = (long long)(t + PW * (lane / NP)) * C::KT + 16 * piece;
      page = r0 < keys ? __ldca(table + (r0 >> pa.page_shift)) : 0;
    }
    const int pg = __shfl_sync(0xffffffffu, page, (k % AHEAD) * NP + piece);
    const int npieces = min(NP, (keys - t * C::KT + 15) / 16);
    const bool mine = lane < 2 * NP && piece < npieces;
    const bool wrong = mine && (unsigned)pg >= (unsigned)pa.num_pages;
    const unsigned any_bad = __ballot_sync(0xffffffffu, wrong);
    const int second = PW < W ? k & 1 : 0;
    const uint32_t nr = second ? n[1]++ : n[0]++;
    const int st = (part + second * PW) * C::S + (int)(nr % C::S);
    if (!__all_sync(0xffffffffu,
                    mbar_wait<kPoll>(&rg.empty[st], ((nr / C::S) & 1u) ^ 1u, rg.abort))) {
      if (second) --n[1];
      else --n[0];
      return false;
    }
    [[maybe_unused]] float *scales = reinterpret_cast<float *>(rg.smem + C::OFF_SCALE + st * C::SCALES);
    if constexpr (P::kScaled) {  // (groups behind the last key: any scale that is a number)
      if (lane < 2 * NP && !mine) scales[lane] = 1.f;
      __syncwarp();
    }
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
      tma_rows(dst, lane >= NP ? vmap : kmap, P::map_row(row), &rg.full[st], policy);
      if constexpr (P::kScaled)
        copy_async4(&scales[lane], (lane >= NP ? extra.v_scales : extra.k_scales) + (row >> 4));
    }
    if constexpr (P::kScaled) arrive_when_copied(&rg.full[st]);
  }
  return true;
}

// Every copy of a ring lands before the block exits (one thread).
template <class P, int W>
__device__ __forceinline__ void drain_ring(const Rings &rg, int ring, uint32_t n) {
  using C = DGeo<P, W>;
  for (uint32_t j = n > (uint32_t)C::S ? n - C::S : 0u; j < n; ++j)
    mbar_wait_drain(&rg.full[ring * C::S + j % C::S], (j / C::S) & 1u);
}

// The ring's tiles of [t_lo, t_hi) against the warp's rows; n as in
// fill_rings.  False when a wait ran out; poison: a bad page was among them.
template <class P, int W, bool kPoll, bool kFew>
__device__ __forceinline__ bool consume_tiles(typename P::Rows &w, const Rings &rg, int ring, int t_lo,
                                             int t_hi, int keys, const int (&reach)[2], float sl2,
                                             uint32_t &n, bool &poison) {
  using C = DGeo<P, W>;
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
      P::clear_rows(sk + C::TILE, left);
      fence_proxy_async_shared();
      __syncwarp();
    }
    const int lim[2] = {reach[0] - t * C::KT, reach[1] - t * C::KT};
    if constexpr (P::kScaled)
      w.template tile<kFew>(smem_addr(sk), smem_addr(sk + C::TILE),
                            reinterpret_cast<const float *>(rg.smem + C::OFF_SCALE + st * C::SCALES),
                            sl2, lim);
    else
      w.template tile<kFew>(smem_addr(sk), smem_addr(sk + C::TILE), sl2, lim);
    __syncwarp();
    if (lane == 0) mbar_arrive(&rg.empty[st]);
  }
  return true;
}

// The same for a unit of `rows` rows, with the row sums finished.
template <class P, int W, bool kPoll>
__device__ __forceinline__ bool consume_ring(typename P::Rows &w, const Rings &rg, int ring, int rows,
                                             int t_lo, int t_hi, int keys, const int (&reach)[2],
                                             float sl2, uint32_t &n, bool &poison) {
  bool ok;
  if (P::kFewForm && (P::kOnlyFew || rows <= 8)) {
    constexpr bool kFew = P::kFewForm;
    ok = consume_tiles<P, W, kPoll, kFew>(w, rg, ring, t_lo, t_hi, keys, reach, sl2, n, poison);
    w.template finish<kFew>();
  } else if constexpr (!P::kOnlyFew) {
    ok = consume_tiles<P, W, kPoll, false>(w, rg, ring, t_lo, t_hi, keys, reach, sl2, n, poison);
    w.finish();
  }
  return ok;
}

// A warp's state into shared memory: [16][D + 4] accumulators, [16] (m, l).
template <class P>
__device__ __forceinline__ void put_state(const typename P::Rows &w, float *acc, float2 *ml) {
  constexpr int D = P::D;
  const int lane = threadIdx.x & 31;
  w.each([&](int hh, int d, const float(&v)[4]) {
    if (P::kOnlyFew && hh == 1) return;
    float *p = acc + (lane / 4 + 8 * hh) * (D + 4) + d;
    if constexpr (P::Rows::kEach == 4)
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  });
  if ((lane & 3) == 0) {
    ml[lane / 4] = make_float2(w.m[0], w.l[0]);
    if (!P::kOnlyFew) ml[lane / 4 + 8] = make_float2(w.m[1], w.l[1]);
  }
}

// Columns d .. d + 3 of row r joined over the W warps' states.
template <int D, int W, int ROWS, bool kFar>
__device__ __forceinline__ void join_states(const float *acc0, const float2 *ml0, int r, int d,
                                            float4 &acc, float &mx, float &ls) {
  mx = neg_inf_f();
#pragma unroll
  for (int k = 0; k < W; ++k) mx = fmaxf(mx, ml0[k * ROWS + r].x);
  const float mz = mx == neg_inf_f() ? 0.f : mx;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  ls = 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const float2 ml = ml0[k * ROWS + r];
    const float wgt = ex2f(ml.x - mz);
    const float4 v = *reinterpret_cast<const float4 *>(acc0 + (k * ROWS + r) * (D + 4) + d);
    acc.x = fmaf(wgt, v.x, acc.x);
    acc.y = fmaf(wgt, v.y, acc.y);
    acc.z = fmaf(wgt, v.z, acc.z);
    acc.w = fmaf(wgt, v.w, acc.w);
    ls = add_sum<kFar>(ls, ml.y, ml.x - mz, wgt);  // (a NaN sum stays one also under a zero weight)
  }
}

template <class P, bool kPoll>
__global__ void __launch_bounds__((DGeo<P, P::kRings>::THREADS), 1)
    paged_decode_kernel(const typename P::T *__restrict__ q, long long q_stride,
                        typename P::T *__restrict__ out,
                        long long out_stride, PagedArgs pa,
                        const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int G, int Hkv, float sl2,
                        int min_column, unsigned char *ws, unsigned host_tag,
                        typename P::Extra extra, int *d_status) {
  using T = typename P::T;
  constexpr int D = P::D;
  constexpr int W = P::kRings;
  using C = DGeo<P, W>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [W][S]
  uint64_t *empty = full + W * C::S;
  uint64_t *cbar = empty + W * C::S;  // all consumer warps
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  volatile int *s_last = abort + 1;
  const Rings rg{full, empty, reinterpret_cast<int *>(smem + C::OFF_BAD), abort, smem};
  unsigned *epoch = reinterpret_cast<unsigned *>(ws);
  unsigned long long *counters = reinterpret_cast<unsigned long long *>(ws + 256);
  float *slots = reinterpret_cast<float *>(ws + 256 + (size_t)kPagedMaxBlocks * 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const Line ln{Hkv, kDRows / G, P::kFixBytes / (2 * D * P::kElem), C::KT, min_column};
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int s = 0; s < W * C::S; ++s) {
      mbar_init(&full[s], C::FULL);
      mbar_init(&empty[s], 1);
    }
    mbar_init(cbar, W);
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
        for (int e = threadIdx.x; e < Hkv * G * D; e += C::THREADS)
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

  // With more consumers than producers, warpgroups of both: the producers' registers go to
  // the consumers (the shares' sum is the launch's, kLaunchRegs for each of three).
  constexpr bool kShares = C::PW < W;
  if (warp >= W) {
    // ======================= producer ========================================
    if constexpr (kShares) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    const uint64_t policy = policy_evict_first();  // a row is read once
    const int part = warp - W;
    uint32_t n[2] = {0, 0};
    bool ok = true;
    do {
      const UnitInfo f = unit_info(pa, u, ln, x0, x1);
      ok = fill_rings<P, W, kPoll>(rg, pa, extra, &kmap, &vmap, part, u.i, u.g, Hkv, f.t_lo, f.t_hi,
                                   f.keys, n, policy, d_status);
      if (!ok) break;
      if (!next_unit(pa, u, f, ln)) break;
    } while (u.base < x1);
    if (lane == 0) {
      if (!ok) give_up(abort, d_status, epoch);
      drain_ring<P, W>(rg, part, n[0]);
      if (kShares) drain_ring<P, W>(rg, part + C::PW, n[1]);
    }
    return;
  }
  if constexpr (kShares) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));

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
  typename P::Rows w;
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
      if (!consume_ring<P, W, kPoll>(w, rg, warp, rows, f.t_lo, f.t_hi, f.keys, reach, sl2, n,
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
      float *macc = reinterpret_cast<float *>(smem + C::OFF_STATE);  // [W][ROWS][D + 4]
      float2 *mml = reinterpret_cast<float2 *>(smem + C::OFF_ML);    // [W][ROWS]
      put_state<P>(w, macc + warp * C::ROWS * (D + 4), mml + warp * C::ROWS);
      if (!consumers_barrier()) return;
      for (int e = threadIdx.x; e < rows * (D / 4); e += W * 32) {
        const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
        float4 acc;
        float mx, ls;
        join_states<D, W, C::ROWS, P::kScaled>(macc, mml, r, d, acc, mx, ls);
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
          for (int e = threadIdx.x; e < rows * (D / 4); e += W * 32) {
            const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
            float4 acc;
            float ls;
            merge_pieces<P::kScaled>(slots, paged_slot_floats(kDRows, D), 2 * kDRows + r * D + d, r, b1,
                                     b2, acc, ls);
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
template <class P, int W, bool kPoll>
__global__ void __launch_bounds__(2 * W * 32, 4 / W)
    paged_decode_cluster_kernel(const typename P::T *__restrict__ q, long long q_stride,
                                typename P::T *__restrict__ out,
                                long long out_stride, PagedArgs pa,
                                const __grid_constant__ CUtensorMap kmap,
                                const __grid_constant__ CUtensorMap vmap, int G, int Hkv, float sl2,
                                typename P::Extra extra, int *d_status) {
  using T = typename P::T;
  constexpr int D = P::D;
  using C = DGeo<P, W>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [W][S]
  uint64_t *empty = full + W * C::S;
  uint64_t *cbar = empty + W * C::S;  // all consumer warps
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  const Rings rg{full, empty, reinterpret_cast<int *>(smem + C::OFF_BAD), abort, smem};
  float *macc = reinterpret_cast<float *>(smem + C::OFF_STATE);  // [W][ROWS][D + 4]
  float2 *mml = reinterpret_cast<float2 *>(smem + C::OFF_ML);    // [W][ROWS]
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cs = (int)gridDim.x, rank = (int)cluster_rank();
  const int i = (int)blockIdx.y / Hkv, g = (int)blockIdx.y - i * Hkv;
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int s = 0; s < W * C::S; ++s) {
      mbar_init(&full[s], C::FULL);
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
    uint32_t nf[2] = {0, 0};
    ok = fill_rings<P, W, kPoll>(rg, pa, extra, &kmap, &vmap, warp - W, i, g, Hkv, t_lo, t_hi, keys,
                                 nf, policy_evict_first(), d_status);
    if (lane == 0) {
      if (!ok) {
        *abort = 1;
        record_status(d_status, KVS_ERR_TIMEOUT);
      }
      drain_ring<P, W>(rg, warp - W, nf[0]);
    }
  } else {
    typename P::Rows w;
    UnitInfo f{};
    f.s = s;
    f.ntok = s.n;
    w.start(q, q_stride, 0, rows, G, f, g);
    int reach[2];  // keys that this lane's two rows attend
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) reach[hh] = s.p + min(lane / 4 + 8 * hh, rows - 1) / G + 1;
    bool poison = false;
    ok = consume_ring<P, W, kPoll>(w, rg, warp, rows, t_lo, t_hi, keys, reach, sl2, n, poison);
    if (poison) w.l[0] = w.l[1] = __int_as_float(0x7fc00000);
    put_state<P>(w, macc + warp * C::ROWS * (D + 4), mml + warp * C::ROWS);
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
      join_states<D, W, C::ROWS, P::kScaled>(macc, mml, r, d, acc, mx, ls);
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
        ls = add_sum<P::kScaled>(ls, ml[k].y, ml[k].x - mx, wgt);
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

template <class P, int W>
const ClusterInfo *cluster_info(int dev) {
  using C = DGeo<P, W>;
  static ClusterInfo info[kDMaxDevices];
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (!info[dev].configured) {
    ClusterInfo rec;
    int top = 4;
    for (auto kern : {paged_decode_cluster_kernel<P, W, false>, paged_decode_cluster_kernel<P, W, true>}) {
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
      if (cudaOccupancyMaxActiveClusters(&n, paged_decode_cluster_kernel<P, W, false>, &cfg) !=
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

template <class P, int W>
int launch_clusters(unsigned cs, const void *q, long long q_stride, const PagedArgs &pa, void *out,
                    long long out_stride, int G, int Hkv, float sl2, const CUtensorMap &kmap,
                    const CUtensorMap &vmap, const typename P::Extra &extra, int *d_status,
                    cudaStream_t stream) {
  using T = typename P::T;
  using C = DGeo<P, W>;
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
      &cfg, poll_waits() ? paged_decode_cluster_kernel<P, W, true>
                         : paged_decode_cluster_kernel<P, W, false>,
      static_cast<const T *>(q), q_stride, static_cast<T *>(out), out_stride,
      pa, kmap, vmap, G, Hkv, sl2, extra, d_status);
  if (e != cudaSuccess) {
    cudaGetLastError();  // leave no stale error for the caller's next check
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

// Hkv kv heads; kmap and vmap: boxes of 16 rows of the pages.
template <class P>
int launch_decode(const void *q, long long q_stride, const CUtensorMap &kmap,
                  const CUtensorMap &vmap, const typename P::Extra &extra, int Hkv,
                  const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                  int *d_status, cudaStream_t stream) {
  using T = typename P::T;
  constexpr int D = P::D;
  using C = DGeo<P, P::kRings>;
  static bool configured[kDMaxDevices] = {false};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDMaxDevices)
    return KVS_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      for (auto kern : {paged_decode_kernel<P, false>,
                        paged_decode_kernel<P, true>}) {
        // (with fewer registers at launch the warpgroups' shares would never come together)
        cudaFuncAttributes fa;
        if (C::PW < C::W && (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.numRegs != kLaunchRegs)) {
          cudaGetLastError();
          return KVS_ERR_LAUNCH;
        }
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
  const int grid = sms < kPagedMaxBlocks ? sms : kPagedMaxBlocks;
  const float sl2 = (float)(1.4426950408889634074 / std::sqrt((double)D));
  // the shortest range worth a block: a step of 4 x 1500 keys, 2 kv heads, in
  // float32 took 16.2 us at 48 cost rows, 15.4 at 96, 16.5 at 192, 18.9 at 384
  const int min_column = 3 * 32;
  // Clusters where no block of theirs can have much to do even if every page
  // of the table is in use; else equal ranges, which stay even however the
  // lengths differ.
  const long long units = (long long)pa.M * Hkv;
  const long long unit_bytes = ((long long)pa.max_pages << pa.page_shift) * D * 2 * P::kElem;
  const ClusterInfo *ci = cluster_info<P, 4>(dev);
  if (!ci) return KVS_ERR_LAUNCH;
  int k = 4;  // clusters of 2^k blocks: all resident at once, no block without a tile
  while (k > 0 && (units > ci->active[k - 1] || unit_bytes < (long long)DGeo<P, 4>::STAGE << k)) --k;
  // (a unit of the clusters has all of a sequence's rows)
  const bool one_tile = (long long)pa.max_new * (H / Hkv) <= kDRows;
  if (one_tile && units <= 65535 && unit_bytes <= P::kBlockBytes << k) {
    if (units > sms && unit_bytes <= P::kShortBytes) {
      if (!cluster_info<P, 2>(dev)) return KVS_ERR_LAUNCH;
      return launch_clusters<P, 2>(1, q, q_stride, pa, out, out_stride, H / Hkv, Hkv, sl2, kmap,
                                      vmap, extra, d_status, stream);
    }
    return launch_clusters<P, 4>(1u << k, q, q_stride, pa, out, out_stride, H / Hkv, Hkv, sl2,
                                      kmap, vmap, extra, d_status, stream);
  }
  const cudaError_t e = launch_pdl(
      poll_waits() ? paged_decode_kernel<P, true>
                   : paged_decode_kernel<P, false>,
      dim3(grid), dim3(C::THREADS), C::SMEM, stream, static_cast<const T *>(q), q_stride,
      static_cast<T *>(out), out_stride, pa, kmap, vmap, H / Hkv, Hkv, sl2, min_column,
      static_cast<unsigned char *>(workspace), fresh_tag(), extra, d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}


}  // namespace

}  // namespace kvs
