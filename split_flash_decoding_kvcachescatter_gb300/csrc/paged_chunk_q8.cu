// paged_chunk_q8.cu -- attention of chunks of new tokens over a paged KV cache
// in 8 bits on the 5th-generation tensor cores (tcgen05), q in float16 or
// bfloat16.
//
// Mathematics and split: as paged_chunk.cu; scales as kvs_rows_q8.cuh: stored
// numbers are exact in float16, so both products run in float16.  A tile of 128 keys
// has one scale for K and one for V, the largest of its blocks'; where a block's is
// smaller its numbers are multiplied by the quotient on their way to float16, which
// for powers of two rounds only what is 2^-33 of the tile's largest or less.  The
// tile's scale of K goes into the exponent, and a row's reference is the maximum of
// score + log2(V's scale), so that the weights of V's numbers are 2^13 at most however
// the scales differ; a tile's share of the row sum is its weights' sum over V's scale.
// bfloat16 rows of q are brought to 2^15 by a power of two (exact down to 2^-28 of
// the row's largest element).  Weights are rounded to float16 for the product: they
// keep 11 bits for bfloat16 too.  (A second part of them, as the decode steps have, would
// take 128 columns of tensor memory, of which heads of 128 leave none.)
//
// Block (20 warps, one block an SM):
//   warps 0-3, 4-7  softmax of tile A and of tile B
//   warp 8, 9       issue S_x = Q_x K^T and O_x += P_x V, as in paged_chunk.cu
//   warp 10, 11     walks the units and describes each to the others; copies Q
//   warps 12-15, 16-19  K and V: each thread copies the pieces that it will turn, 32
//                   keys at a time and a tile ahead, and writes them as float16
//                   in the layout that the tensor cores read; the tiles' scales; the
//                   latter warps also turn bfloat16 queries, in place
// TMEM as in paged_chunk.cu.
//
// What bounds it: the turning.  A pair of tiles moves about 320 KB through shared
// memory (pages in and out, float16 in, and what the products read), the pages come
// from L2 with as many bytes on their way as the rings hold, and eight warps convert.
// 4096 rows of 32 query heads on 8 kv heads of 128 behind 4096 keys: 349 us, where
// paged_chunk.cu takes about 255 for pages in 16 bits.
// Measured at that shape: rings of a whole tile and rows that leave without a staging
// area 343 us at the time, 8 KB of staging and three quarters 402; two quarters a step 487; a
// warp that copies for the turning ones 566 to 646; pages read straight into
// registers 701; mma.sync units as the decode steps' 2966.

#include <cmath>
#include <mutex>
#include <type_traits>

#include "kvs_chunk.cuh"
#include "kvs_fp8.cuh"
#include "kvs_rows_q8.cuh"

namespace kvs {

namespace {

constexpr int kCqMmaWarp = 8, kCqPvWarp = 9, kCqUnitWarp = 10, kCqQueryWarp = 11, kCqTurnWarp = 12;
constexpr int kCqThreads = 20 * 32;
// registers a thread: at launch, and by warpgroup; the shares' sum is the launch's
constexpr int kCqRegs = 96;
constexpr int kCqRegsSoftmax = 168, kCqRegsIssue = 48, kCqRegsTurn = 48;
static_assert(2 * kCqRegsSoftmax + kCqRegsIssue + 2 * kCqRegsTurn == 5 * kCqRegs, "what the launch has");
// as paged_chunk.cu's; at 128, 256, 384, 640, 1024 cost rows: 1700 tokens of nine sequences 118, 109,
// 102, 103, 107 us, 1400 of sixteen 92, 82, 77, 78, 83, 4096 over 8192 keys 350, 348, 344, 344, 348
constexpr int kCqFix = 384;
constexpr int kCqMinRange = 768;
constexpr float kCqLift = 5.f;

// The scales of a key tile: K's times log2(e) / sqrt(D), log2 of V's and 1 / V's.
struct CqScales {
  float score, lg, inv, pad;
};

template <int D>
struct CqGeo {
  static constexpr int NB = D / 64;               // 128-byte column blocks of a row
  static constexpr int BLK = 128 * 128;           // bytes of a block of 128 rows
  static constexpr int TILE = NB * BLK;           // one tile of Q, K or V in float16
  static constexpr int KS = 2, VS = 2;            // stages (the turning warps count on two)
  static constexpr int QK = kCN / 4;              // keys of a quarter, as they come from the pages
  static constexpr int QUARTER = QK * D;          // its bytes
  static constexpr int RQ = 4;                    // quarters in a ring: a tile
  static constexpr int SR = 8;                    // tiles whose scales are kept
  static constexpr int OFF_Q = 0;                 // Q_A, Q_B
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + KS * TILE;
  static constexpr int OFF_RAW = OFF_V + VS * TILE;
  // exponents of the rows' factors (biased), by unit parity: uint8 [2][2][128]
  static constexpr int OFF_QFAC = OFF_RAW + 2 * RQ * QUARTER;
  static constexpr int OFF_SCALE = OFF_QFAC + 2 * 2 * 128;  // CqScales [SR]
  static constexpr int OFF_BAR = OFF_SCALE + SR * (int)sizeof(CqScales);
  // q, qraw, qfree, kfull[KS], kfree[KS], vfull[VS], vfree[VS], sfull[2], sread,
  // pfull[2], pvdone[2], wg[2], final[2], ufull[kCUnits], ufree[kCUnits], sgone[4], sbar[SR],
  // qf[2]
  static constexpr int NBAR = 3 + 2 * KS + 2 * VS + 2 + 1 + 6 + 2 + 2 * kCUnits + 4 + SR + 2;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int OFF_MISC = OFF_TMEM + 8;   // abort, last[2], pad
  static constexpr int OFF_UNIT = OFF_MISC + 16;  // CUnit [kCUnits]
  static constexpr int NEED = OFF_UNIT + kCUnits * (int)sizeof(CUnit);
  // (all 512 TMEM columns are this block's: no second one an SM)
  static constexpr int SMEM = NEED > 116 * 1024 ? NEED : 116 * 1024;
  static_assert(SMEM <= 227 * 1024, "one block per SM must fit");
};

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct CqCache {
  const unsigned char *k_pages, *v_pages;
  const float *k_scales, *v_scales;
};

// Two e4m3 numbers times `by` (float16 twice) as float16.
__device__ __forceinline__ uint32_t turned(uint32_t w, uint32_t by) {
  const uint32_t f = from_e4m3x2(w);
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&f), *reinterpret_cast<const __half2 *>(&by));
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <typename T, int D, bool kPoll>
__global__ void __launch_bounds__(kCqThreads, 1)
    paged_chunk_q8_kernel(T *__restrict__ out, long long out_stride, PagedArgs pa,
                          const __grid_constant__ CUtensorMap qmap, CqCache cache, int G, int Hkv,
                          float sl2, unsigned char *ws, unsigned host_tag, int *d_status) {
  using C = CqGeo<D>;
  constexpr int KS = C::KS, VS = C::VS, SR = C::SR;
  constexpr bool kTurnQ = !std::is_same<T, __half>::value;  // q has to become float16
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *bar_q = bars;            // Q of the unit is there in float16
  uint64_t *bar_qraw = bar_q + 1;    // Q of the unit landed
  uint64_t *qfree = bar_qraw + 1;    // the unit's S products done (commit)
  uint64_t *kfull = qfree + 1;       // [KS] an arrival a turning warp
  uint64_t *kfree = kfull + KS;      // [KS] the S products of a stage done (commit)
  uint64_t *vfull = kfree + KS;      // [VS]
  uint64_t *vfree = vfull + VS;      // [VS] the P V products of a stage done (commit)
  uint64_t *sfull = vfree + VS;      // [2] S of tile x ready (commit)
  uint64_t *sread = sfull + 2;       // S is in registers (an arrival of each of the tile's warps)
  uint64_t *pfull = sread + 1;       // [2] P_x written, O_x rescaled (an arrival a warp)
  uint64_t *pvdone = pfull + 2;      // [2] P V_x done (commit)
  uint64_t *wgbar = pvdone + 2;      // [2] the warps of a warpgroup
  uint64_t *final = wgbar + 2;       // [2] every product S, every P V of the block done (commit)
  uint64_t *ufull = final + 2;       // [kCUnits] a unit is described
  uint64_t *ufree = ufull + kCUnits; // [kCUnits] the 19 other warps are done with it
  uint64_t *sgone = ufree + kCUnits; // [4] S product k of the block issued, at k % 4
  uint64_t *sbar = sgone + 4;        // [SR] scales of key tile k, at k % SR (K's and V's)
  uint64_t *qf = sbar + SR;          // [2] factors of unit n's rows, at n % 2 (an arrival a turning warp)
  CUnit *units = reinterpret_cast<CUnit *>(smem + C::OFF_UNIT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  volatile int *s_last = abort + 1;  // [2]
  unsigned char *qfac = smem + C::OFF_QFAC;
  CqScales *scales = reinterpret_cast<CqScales *>(smem + C::OFF_SCALE);
  unsigned *epoch = reinterpret_cast<unsigned *>(ws);
  unsigned long long *counters = reinterpret_cast<unsigned long long *>(ws + 256);
  float *slots = reinterpret_cast<float *>(ws + 256 + (size_t)kPagedMaxBlocks * 16);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const int TT = kCM / G;  // tokens of a tile
  constexpr uint32_t kTileStep = C::TILE >> 4;  // one tile further on, in a descriptor
  const Line ln{Hkv, 2 * TT, kCqFix, kCN, kCqMinRange};

  if (threadIdx.x == 0) {
    prefetch_map(&qmap);
    for (int j = 0; j < C::NBAR; ++j) {  // each once
      uint64_t *bar = bars + j;
      // an arrival a warp of the softmax's four or the four that turn
      const bool of_four = bar == sread || bar == pfull || bar == pfull + 1 || bar == wgbar ||
                           bar == wgbar + 1 || (kTurnQ && bar == bar_q) ||
                           (bar >= kfull && bar < kfull + KS) || (bar >= vfull && bar < vfull + VS) ||
                           bar >= qf;
      const bool of_k_and_v = bar >= sbar && bar < sbar + SR;
      mbar_init(bar, of_four ? 4 : of_k_and_v ? 2 : bar >= ufree && bar < ufree + kCUnits ? 19 : 1);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, kCTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  allow_dependent_launch();
  const uint32_t tmem = *tmem_slot;
  auto tile_of = [&](const CUnit &f, int x) {
    CTile t;
    t.tok0 = f.tok0 + x * TT;
    t.ntok = min(TT, f.ntok - x * TT);
    t.nt = t.ntok > 0 ? (f.p + t.tok0 + t.ntok + kCN - 1) / kCN : 0;
    t.lo = min(f.t_lo, t.nt);
    t.hi = min(f.t_hi, t.nt);
    return t;
  };
  // The block's n-th unit, once it is described; false when a wait ran out.
  auto unit = [&](int n, CUnit &f) -> bool {
    if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&ufull[n % kCUnits], (uint32_t)(n / kCUnits) & 1u, abort)))
      return false;
    f = units[n % kCUnits];
    return true;
  };
  auto unit_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ufree[n % kCUnits]);
  };

  if (warp < 8) {
    // ======================= softmax of tile x ===============================
    more_registers<kCqRegsSoftmax>();
    const int x = warp >> 2;
    const int t = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + lane_base;
    const uint32_t tm_p = tmem + lane_base + kCN + x * (kCN / 2);
    const uint32_t tm_o = tmem + lane_base + 2 * kCN + x * D;
    int sb = 0;   // S_x products of the earlier units
    int kt0 = 0;  // key tiles of the earlier units
    uint32_t wphase = 0;
    bool failed = false;
    auto wg_barrier = [&]() -> bool {  // the warpgroup's four warps, bounded
      __syncwarp();
      if (lane == 0) mbar_arrive(&wgbar[x]);
      const bool got = __all_sync(0xffffffffu, mbar_wait<kPoll>(&wgbar[x], wphase, abort));
      wphase ^= 1u;
      return got;
    };
    // bad sequences: status, and NaN rows where the rows are known
    for (int i = b; i < pa.M; i += gridDim.x) {
      const PagedSeq q = paged_seq(pa, i);
      if (q.err != KVS_OK) {
        if (threadIdx.x == 0) record_status(d_status, q.err);
        for (int r = 0; r < q.n; ++r)
          for (int e = threadIdx.x; e < Hkv * G * D; e += 256)
            out[(long long)(q.row0 + r) * out_stride + e] = from_f32<T>(__int_as_float(0x7fc00000));
      }
    }
    const unsigned tag = launch_tag(host_tag, __ldcg(epoch));
    for (int nq = 0; !failed; ++nq) {
      CUnit f;
      if (!unit(nq, f)) failed = true;
      if (failed || f.t_lo == f.t_hi) break;
      const CTile tl = tile_of(f, x);
      const int rows = tl.ntok * G;
      const bool live = t < rows;
      const int tok = live ? t / G : tl.ntok - 1;
      const int last = f.p + tl.tok0 + tok;  // the row's last key
      const int first_last = f.p + tl.tok0;  // the tile's first row's
      float m = neg_inf_f(), l = 0.f, fac = 1.f, lgmax = 0.f;
      for (int n = tl.lo; n < tl.hi; ++n) {
        const uint32_t ph = (uint32_t)(sb + n - tl.lo) & 1u;
        const int kt = kt0 + n - f.t_lo;
        if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&sbar[kt % SR], (uint32_t)(kt / SR) & 1u, abort) &&
                                         mbar_wait<kPoll>(&sfull[x], ph, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (kTurnQ && n == tl.lo) {
          if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&qf[nq & 1], (uint32_t)(nq >> 1) & 1u, abort))) {
            failed = true;
            break;
          }
          fac = __uint_as_float((unsigned)qfac[(nq & 1) * 256 + x * 128 + t] << 23);
        }
        const CqScales &sc = scales[kt % SR];
        const float f = fac * sc.score, lg0 = sc.lg;  // (f > 0)
        // (2^-60 of the largest scale so far at the least: kvs_rows_q8.cuh)
        lgmax = fmaxf(lgmax, lg0);
        const float lg = fmaxf(lg0, lgmax - 60.f), inv = lg > lg0 ? ex2(-lg) : sc.inv;
        float r[kCN];
        tmem_ld64(tm_s, *reinterpret_cast<float(*)[64]>(&r[0]));
        tmem_ld64(tm_s + 64, *reinterpret_cast<float(*)[64]>(&r[64]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sread);  // the other tile's product may have the columns
        const int key0 = n * kCN;
        if (key0 + kCN - 1 > first_last) {
          const int lim = last - key0;  // keys 0..lim of the tile are attended
#pragma unroll
          for (int v = 0; v < kCN; ++v) r[v] = v <= lim ? r[v] : neg_inf_f();
        }
        float mx[4] = {r[0], r[1], r[2], r[3]};  // four chains (max is exact in any order)
#pragma unroll
        for (int v = 4; v < kCN; v += 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], r[v + k]);
        }
        const float cm = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), f, lg - kCqLift);
        // the reference moves only when the row's grows by more than 2^kCRescale
        // (rows that do not exist hold anything: they never ask for a rescale)
        const float m_ref = cm > m + kCRescale ? cm : m;
        const float ah = (m == neg_inf_f() || !live) ? 1.f : ex2(0.5f * (m - m_ref)), alpha = ah * ah;
        l = l * ah * ah;  // (in two steps: kvs_rows_q8.cuh)
        // P_x and O_x are free once the product before has read and written them
        if (n > tl.lo) {
          if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&pvdone[x], ph ^ 1u, abort))) {
            failed = true;
            break;
          }
          tc_fence_after();
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float o[16];
              uint32_t w[16];
              tmem_ld16(tm_o + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int v = 0; v < 16; ++v) w[v] = __float_as_uint(o[v] * alpha);
              tmem_st16u(tm_o + c * 16, w);
            }
          }
        }
        const float mb = (m_ref == neg_inf_f()) ? 0.f : m_ref;
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 f2 = make_float2(f, f), up2 = make_float2(lg - mb, lg - mb);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t w[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const float2 x2 = __ffma2_rn(make_float2(r[32 * ch + 2 * v], r[32 * ch + 2 * v + 1]), f2, up2);
            const float p0 = ex2(x2.x), p1 = ex2(x2.y);
            ls[v & 1] = __fadd2_rn(ls[v & 1], make_float2(p0, p1));
            w[v] = pack_pair<__half>(p0, p1);
          }
          tmem_st16u(tm_p + ch * 16, w);
        }
        l = fmaf((ls[0].x + ls[1].x) + (ls[0].y + ls[1].y), inv, l);
        m = m_ref;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[x]);
      }
      if (failed) break;
      sb += tl.hi - tl.lo;
      kt0 += f.t_hi - f.t_lo;
      if (tl.lo < tl.hi) {
        // the tile's last product is done: O_x is final
        if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&pvdone[x], (uint32_t)(sb - 1) & 1u, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
        // (the unit is read again there: in registers it would crowd out the row)
        if (!finish_tile<T, D, false, true>(out, out_stride, &units[nq % kCUnits], tl, x, t, lane, live, tok, G, b,
                               tm_o, m, l, nullptr, slots, counters, tag, epoch, d_status, s_last,
                               wg_barrier)) {
          failed = true;
          break;
        }
      }
      unit_done(nq);
    }
    if (failed && lane == 0) give_up(abort, d_status, epoch);
  } else if (warp < kCqTurnWarp) {
    fewer_registers<kCqRegsIssue>();
    if (warp == kCqUnitWarp) {
      // ======================= units ===========================================
      int nq = 0;  // units described
      bool ok = true;
      const Cuts cut = equal_cuts(warp_line_total(pa, ln, lane), ln, gridDim.x);
      bool more = cut.R > 0 && b < cut.NS;
      const long long x0 = more ? cut.start(b) : 0, x1 = more ? cut.start(b + 1) : 0;
      Unit u{pa.M, 0, 0, 0};
      if (more) u = warp_unit_at(pa, ln, x0, lane);
      // Describes a unit, once the one before in the same place is done with.  (Nothing
      // else is waited for: the warps that turn K and V look two tiles ahead, which may
      // be two units.)
      auto describe = [&](int n, const CUnit &f) {
        if (n >= kCUnits &&
            !__all_sync(0xffffffffu, mbar_wait<kPoll>(&ufree[n % kCUnits], (uint32_t)(n / kCUnits - 1) & 1u, abort)))
          return false;
        if (lane == 0) {
          units[n % kCUnits] = f;
          mbar_arrive(&ufull[n % kCUnits]);
        }
        __syncwarp();
        return true;
      };
      while (more && ok) {
        const UnitInfo f = unit_info(pa, u, ln, x0, x1);
        if (f.t_lo < f.t_hi) {
          CUnit d{f.s.p, f.s.row0, f.tok0, f.ntok, f.t_lo, f.t_hi, u.g, 0, u.i, f.s.p + f.s.n, b, {b, b}};
          if (f.t_hi - f.t_lo < f.nt) {
            d.b1 = cut.at(f.k0);
            for (int x = 0; x < 2; ++x) {
              const int nt = tile_of(d, x).nt;
              d.b2[x] = nt > 0 ? cut.at(f.k0 + (long long)(nt - 1) * kCN) : d.b1;
            }
          }
          if (!(ok = describe(nq++, d))) break;
        }
        more = next_unit(pa, u, f, ln) && u.base < x1;
      }
      if (ok) ok = describe(nq, CUnit{});
      if (!ok && lane == 0) give_up(abort, d_status, epoch);
      __syncwarp();
    } else if (warp == kCqQueryWarp) {
      // ======================= Q ===============================================
      uint64_t *qbar = kTurnQ ? bar_qraw : bar_q;
      int nq = 0;  // units whose rows are copied
      bool ok = true;
      for (;; ++nq) {
        CUnit f;
        if (!(ok = unit(nq, f)) || f.t_lo == f.t_hi) break;
        if (nq > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(qfree, (uint32_t)(nq - 1) & 1u, abort))))
          break;
        if (lane == 0) {
          const int tiles = f.ntok > TT ? 2 : 1;
          mbar_arrive_expect_tx(qbar, (uint32_t)(tiles * C::NB * TT * G * 128));
          for (int x = 0; x < tiles; ++x)
            for (int cb = 0; cb < C::NB; ++cb)
              tma_q(smem + C::OFF_Q + x * C::TILE + cb * C::BLK, &qmap, f.g * G,
                    f.row0 + f.tok0 + x * TT, cb, qbar);
        }
        unit_done(nq);
      }
      if (lane == 0) {
        if (!ok) give_up(abort, d_status, epoch);
        // every copy issued lands before the block can exit
        if (nq > 0) mbar_wait_drain(qbar, (uint32_t)(nq - 1) & 1u);
      }
      __syncwarp();
    } else if (warp == kCqMmaWarp) {
      // ======================= products S ======================================
      // (order and waits: paged_chunk.cu)
      const uint32_t lq = (uint32_t)desc_sw128(smem + C::OFF_Q, 16, 1024);
      const uint32_t lk = lq + ((C::OFF_K - C::OFF_Q) >> 4);
      const uint32_t tm = warp_uniform(tmem);
      constexpr uint32_t kIdS = idesc16<__half>(kCM, kCN, false);
      int gt = 0;       // K tiles of the earlier units
      uint32_t ns = 0;  // S products issued
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t phase) {
        return ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(bar, phase & 1u, abort)) != 0;
      };
      for (int nq = 0; ok; ++nq) {
        CUnit f;
        if (!(ok = unit(nq, f)) || f.t_lo == f.t_hi) break;
        const CTile ta = tile_of(f, 0), tb = tile_of(f, 1);
        const int n_x[2] = {ta.hi - ta.lo, tb.hi - tb.lo};  // products of each tile
        const int n_all = f.t_hi - f.t_lo;                  // K tiles of the unit
        if (!wait(bar_q, nq)) break;
        for (int i = 0; i < n_all && ok; ++i, ++gt) {
          if (!wait(&kfull[gt % KS], gt / KS)) break;
          const uint32_t bk = warp_uniform(lk + (uint32_t)(gt % KS) * kTileStep);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (i >= n_x[x]) continue;
            if (ns > 0 && !wait(sread, ns - 1u)) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t at = (uint32_t)(ks >> 2) * (C::BLK >> 4) + (ks & 3) * 2;
              mma_f16_warp(tm, lq + (x ? kTileStep : 0u) + at, bk + at, kDescHi, kIdS, ks > 0 ? 1u : 0u);
            }
            mma_commit_warp(&sfull[x]);
            if (lane == 0) mbar_arrive(&sgone[ns & 3]);
            ++ns;
          }
          if (!ok) break;
          mma_commit_warp(&kfree[gt % KS]);
          if (i + 1 == n_all) mma_commit_warp(qfree);
        }
        if (!ok) break;
        unit_done(nq);
      }
      if (!ok && lane == 0) give_up(abort, d_status, epoch);
      // every product issued finishes before the block frees the tensor memory
      mma_commit_warp(&final[0]);
      mbar_wait_drain(&final[0], 0u);
      __syncwarp();
    } else if (warp == kCqPvWarp) {
      // ======================= products P V ====================================
      const uint32_t lv = (uint32_t)desc_sw128(smem + C::OFF_V, C::BLK, 1024);
      const uint32_t tm = warp_uniform(tmem);
      constexpr uint32_t kIdO = idesc16<__half>(kCM, D, true);
      int gt = 0;             // V tiles of the earlier units
      uint32_t s0 = 0;        // S products of the key tiles before
      int pdone[2] = {0, 0};  // P V_x products of the earlier units
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t phase) {
        return ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(bar, phase & 1u, abort)) != 0;
      };
      for (int nq = 0; ok; ++nq) {
        CUnit f;
        if (!(ok = unit(nq, f)) || f.t_lo == f.t_hi) break;
        const CTile ta = tile_of(f, 0), tb = tile_of(f, 1);
        const int n_x[2] = {ta.hi - ta.lo, tb.hi - tb.lo};
        const int n_all = f.t_hi - f.t_lo;
        for (int j = 0; j < n_all && ok; ++j, ++gt) {
          if (!wait(&vfull[gt % VS], gt / VS)) break;
          const uint32_t bv = warp_uniform(lv + (uint32_t)(gt % VS) * kTileStep);
          const uint32_t acc = warp_uniform(j > 0 ? 1u : 0u);  // O_x (+)= P_x V
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (j >= n_x[x]) continue;
            // O_x += P_x V goes behind the tile's next S (paged_chunk.cu)
            if (j + 1 < n_x[x]) {
              const uint32_t k = s0 + (j < n_x[0]) + (j < n_x[1]) + (x && j + 1 < n_x[0] ? 1 : 0);
              if (!wait(&sgone[k & 3], k >> 2)) break;
            }
            if (!wait(&pfull[x], pdone[x] + j)) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kCN / 16; ++ks)
              mma_f16_ts_warp(tm + 2 * kCN + x * D, tm + kCN + x * (kCN / 2) + ks * 8, bv + 128 * ks,
                              kDescHi, kIdO, ks > 0 ? 1u : acc);
            mma_commit_warp(&pvdone[x]);
          }
          if (!ok) break;
          mma_commit_warp(&vfree[gt % VS]);
          s0 += (j < n_x[0]) + (j < n_x[1]);
        }
        if (!ok) break;
        pdone[0] += n_x[0];
        pdone[1] += n_x[1];
        unit_done(nq);
      }
      if (!ok && lane == 0) give_up(abort, d_status, epoch);
      mma_commit_warp(&final[1]);
      mbar_wait_drain(&final[1], 0u);
      __syncwarp();
    }
  } else {
    // ======================= K and V to float16 ================================
    fewer_registers<kCqRegsTurn>();
    constexpr int NV = C::QUARTER / 16 / 128;  // 16-byte pieces of a quarter, a thread
    static_assert(NV == D / 64, "pieces of a row pair, or of a row");
    const int t = threadIdx.x & 127;
    const bool is_v = warp >= kCqTurnWarp + 4;
    uint64_t *full = is_v ? vfull : kfull, *free = is_v ? vfree : kfree;
    const unsigned char *pages = is_v ? cache.v_pages : cache.k_pages;
    const float *page_scales = is_v ? cache.v_scales : cache.k_scales;
    // This thread's pieces of a quarter.  D = 64: piece t % 4 of row t / 4.  D = 128: of
    // rows r and r ^ 1, r = 2 (t / 8) + s with s = t / 4 % 2, pieces t % 4 + 4 s: eight
    // lanes then read 128 bytes that share no bank, and write to different pieces.  All
    // rows of a warp lie in group `half` of the quarter's two groups of 16.
    const int sub = D == 128 ? (t >> 2) & 1 : 0, half = t >> 6;
    const int row0 = D == 128 ? 2 * (t >> 3) + sub : t >> 2, c = (t & 3) + 4 * sub;
    const int to0 = sub * C::BLK + row0 * 128 + (((2 * c) ^ row0) & 7) * 16;  // the lower half's place
    unsigned char *raw = smem + C::OFF_RAW + (is_v ? C::RQ * C::QUARTER : 0) + row0 * D + c * 16;
    constexpr int kPair = D;  // (row r ^ 1: this far on, or back)
    const int pair = row0 & 1 ? -kPair : kPair;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t phase) {
      return ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(bar, phase & 1u, abort)) != 0;
    };
    // A key tile: this lane's group of 16 rows is number lane % 8 of it.
    struct Tile {
      int row;    // first row of the group in the pages (before resolve(): its page)
      int left;   // keys from the tile's first on
      int unit;   // number of the unit, negative: ~number, the unit's first tile
      float scale;
    };
    // The cursor: tile n of unit uq, which ends at tile t_hi (the rest is read where it is
    // needed: these threads have few registers).
    int uq = -1, n = 0, t_hi = 0;
    // The next key tile of the block, its pages asked for; false after the last one.
    auto next = [&](Tile &a) -> bool {
      const bool first = uq < 0 || n + 1 >= t_hi;
      if (first) {
        if (uq >= 0) unit_done(uq);
        ++uq;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(&ufull[uq % kCUnits], (uint32_t)(uq / kCUnits) & 1u, abort))))
          return false;
        n = units[uq % kCUnits].t_lo;
        t_hi = units[uq % kCUnits].t_hi;
        if (n == t_hi) return false;
      } else {
        ++n;
      }
      const CUnit &f = units[uq % kCUnits];
      a.unit = first ? ~uq : uq;
      a.left = f.L - n * kCN;
      const int key = n * kCN + 16 * (lane & 7);
      a.row = key < f.L ? __ldca(pa.page_table + (size_t)f.seq * pa.max_pages + (key >> pa.page_shift)) : 0;
      return true;
    };
    // Its rows, once the pages are known (next() has not gone on); the scales asked for.
    auto resolve = [&](Tile &a) {
      const int key = n * kCN + 16 * (lane & 7);
      if ((unsigned)a.row >= (unsigned)pa.num_pages) {
        record_status(d_status, KVS_ERR_PAGE);
        *const_cast<volatile int *>(&units[uq % kCUnits].bad) = 1;
        a.row = 0;
      }
      a.row = ((a.row * Hkv + units[uq % kCUnits].g) << pa.page_shift) + (key & ((1 << pa.page_shift) - 1));
      a.scale = 16 * (lane & 7) < a.left ? __ldcg(page_scales + (a.row >> 4)) : 0.f;
    };
    // Quarter q of tile a into the ring, rows behind the last key as zeros.
    auto source = [&](const Tile &a, int q) {
      const int row = __shfl_sync(0xffffffffu, a.row, 2 * q + half) + (row0 & 15);
      return pages + (size_t)row * D + c * 16;
    };
    auto copy = [&](const Tile &a, int q, const unsigned char *from) {
      unsigned char *to = raw + q * C::QUARTER;
      if (a.left >= kCN) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to + k * pair)), "l"(from + k * pair)
                       : "memory");
      } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int live = q * C::QK + (row0 ^ k) < a.left ? 16 : 0;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to + k * pair)),
                       "l"(from + k * pair), "r"(live)
                       : "memory");
        }
      }
    };
    auto commit = [&]() { asm volatile("cp.async.commit_group;" ::: "memory"); };
    Tile a{}, b2{}, b3{};  // a tile under way, the next one (resolved a tile ahead) and the one after (asked for)
    bool have = next(a);
    if (have) resolve(a);
    for (int q = 0; q < 4; ++q) {
      if (have) copy(a, q, source(a, q));
      commit();
    }
    bool more = have && next(b2);
    int done = 0;  // tiles written
    while (have && ok) {
      // the tile's scale, the largest of its blocks', and what each is of that
      float most = a.scale;
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      most = fmaxf(most, kLeastScale);  // 2^-60
      float inv = __uint_as_float((254u << 23) - __float_as_uint(most));
      if (__float_as_uint(most) & 0x7fffffu) inv = 1.f / most;  // (no power of two)
      const __half2 by_h = __float2half2_rn(a.scale * inv);
      const uint32_t by = *reinterpret_cast<const uint32_t *>(&by_h);
      if ((warp & 3) == 0 && lane == 0) {
        CqScales &sc = scales[done % SR];
        if (is_v)
          value_scale(most, sc.lg, sc.inv);
        else
          sc.score = most * sl2;
        mbar_arrive(&sbar[done % SR]);
      }
      if (more) resolve(b2);
      const bool third = more && next(b3);
      if (!ok) break;
      if (kTurnQ && is_v && a.unit < 0) {
        // rows of q to float16 in place: a thread a row
        const int nq = ~a.unit;
        if (!wait(bar_qraw, (uint32_t)nq)) break;
        const int tiles = units[nq % kCUnits].ntok > TT ? 2 : 1;
#pragma unroll 1
        for (int x = 0; x < tiles; ++x) {
          unsigned char *row = smem + C::OFF_Q + x * C::TILE + t * 128;
          auto piece = [&](int j) {
            return reinterpret_cast<uint4 *>(row + (j >> 3) * C::BLK + (((j & 7) ^ (t & 7)) * 16));
          };
          uint32_t top = 0;  // |elements| as integers: bfloat16 orders them
#pragma unroll 2
          for (int j = 0; j < D / 8; ++j) {
            const uint4 w = *piece(j);
            top = __vmaxu2(__vmaxu2(top, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu)),
                           __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
          }
          // largest < 2^(ex + 1)
          const int ex = max((int)(max(top & 0xffffu, top >> 16) >> 7) - 127, -60);
          const float up = __uint_as_float((unsigned)(14 - ex + 127) << 23);
#pragma unroll 2
          for (int j = 0; j < D / 8; ++j) {
            const uint4 w = *piece(j);
            auto half2_of = [&](uint32_t e) {
              return pack_pair<__half>(__uint_as_float(e << 16) * up, __uint_as_float(e & 0xffff0000u) * up);
            };
            *piece(j) = make_uint4(half2_of(w.x), half2_of(w.y), half2_of(w.z), half2_of(w.w));
          }
          qfac[(nq & 1) * 256 + x * 128 + t] = (unsigned char)(ex - 14 + 127);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_q);
          mbar_arrive(&qf[nq & 1]);
        }
      }
      const int st = done & 1;
      if (done >= 2 && !wait(&free[st], (uint32_t)(done / 2 - 1))) break;
      unsigned char *tile = smem + (is_v ? C::OFF_V : C::OFF_K) + st * C::TILE + to0;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        asm volatile("cp.async.wait_group 3;" ::: "memory");  // this thread's pieces of the quarter
        uint4 v[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] = *reinterpret_cast<const uint4 *>(raw + q * C::QUARTER + k * pair);
        const unsigned char *from = source(b2, q);
        const uint32_t m2 = __shfl_sync(0xffffffffu, by, 2 * q + half);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          // (row r ^ 1: the other half's place, a row on or back)
          unsigned char *at = tile + q * C::QK * 128 + (k ? (row0 & 1 ? -128 : 128) : 0);
          const int x = reinterpret_cast<uintptr_t>(at) & 16 ? -16 : 16;
          *reinterpret_cast<uint4 *>(k ? at + x : at) =
              make_uint4(turned(v[k].x, m2), turned(v[k].x >> 16, m2), turned(v[k].y, m2), turned(v[k].y >> 16, m2));
          *reinterpret_cast<uint4 *>(k ? at : at + x) =
              make_uint4(turned(v[k].z, m2), turned(v[k].z >> 16, m2), turned(v[k].w, m2), turned(v[k].w >> 16, m2));
        }
        // the next tile's takes its place (here: what was read has arrived in registers)
        if (more) copy(b2, q, from);
        commit();
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
      ++done;
      a = b2;
      b2 = b3;
      have = more;
      more = third;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) give_up(abort, d_status, epoch);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kCTmemCols);
}

template <typename T, int D>
int launch_chunk(const void *q, long long q_stride, const kvs_paged_cache_q8 &cache, int dtype,
                 const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                 int *d_status, cudaStream_t stream) {
  using C = CqGeo<D>;
  static bool configured[kCMaxDevices] = {false};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kCMaxDevices) return KVS_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      for (auto kern : {paged_chunk_q8_kernel<T, D, false>, paged_chunk_q8_kernel<T, D, true>}) {
        // (with fewer at launch the warpgroups' shares would never come together)
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.numRegs != kCqRegs) {
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
  const int Hkv = cache.num_kv_heads, G = H / Hkv;
  CUtensorMap qmap;
  const int rc = make_q_map(&qmap, q, pa.num_rows, q_stride, H, D, dtype, kCM / G, G);
  if (rc != KVS_OK) return rc;
  const CqCache cc{static_cast<const unsigned char *>(cache.k_pages),
                   static_cast<const unsigned char *>(cache.v_pages), cache.k_scales, cache.v_scales};
  const int grid = sms < kPagedMaxBlocks ? sms : kPagedMaxBlocks;
  const float sl2 = (float)(1.4426950408889634074 / std::sqrt((double)D));
  const cudaError_t e = launch_pdl(
      poll_waits() ? paged_chunk_q8_kernel<T, D, true> : paged_chunk_q8_kernel<T, D, false>, dim3(grid),
      dim3(kCqThreads), C::SMEM, stream, static_cast<T *>(out), out_stride, pa, qmap, cc, G, Hkv, sl2,
      static_cast<unsigned char *>(workspace), fresh_tag(), d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

}  // namespace

int set_wait_limit_chunk_q8(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

int launch_paged_chunk_q8(const void *q, long long q_stride, const kvs_paged_cache_q8 &cache,
                          int dtype, const PagedArgs &pa, void *out, long long out_stride, int H,
                          void *workspace, int *d_status, cudaStream_t stream) {
#define KVS_CHUNK(T)                                                                            \
  return cache.head_dim == 64                                                                   \
             ? launch_chunk<T, 64>(q, q_stride, cache, dtype, pa, out, out_stride, H, workspace, \
                                   d_status, stream)                                            \
             : launch_chunk<T, 128>(q, q_stride, cache, dtype, pa, out, out_stride, H,          \
                                    workspace, d_status, stream)
  if (dtype == KVS_F16) KVS_CHUNK(__half);
  if (dtype == KVS_BF16) KVS_CHUNK(__nv_bfloat16);
#undef KVS_CHUNK
  return KVS_ERR_UNSUPPORTED;
}

}  // namespace kvs
