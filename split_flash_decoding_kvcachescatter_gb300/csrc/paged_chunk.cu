// paged_chunk.cu -- attention of chunks of new tokens over a paged KV cache
// on the 5th-generation tensor cores (tcgen05), float16 and bfloat16.
//
// Mathematics and split: as paged_attention.cu (flash attention over a key
// axis cut into equal cost columns, pieces of a unit merged by the block
// that completes it).  A unit is two tiles A and B of TT = 128 / G whole
// tokens with the G query heads of their kv head, so that both share every
// K and V tile of 128 keys: per key tile a block reads 64 KB (D = 128) for
// four products of 128 x 128 x 128, 2048 tensor-core cycles.
//
// Block (11 warps, one block an SM):
//   warps 0-3, 4-7  softmax of tile A and of tile B: thread t owns row t,
//                   which is TMEM lane t
//   warp 8          issues S_x = Q_x K^T (operands in shared memory, K-major)
//   warp 9          issues O_x += P_x V (P from TMEM; V as the copies leave
//                   it: head elements contiguous, which is the MN-major
//                   operand, so nothing is transposed)
//   warp 10         walks the units and describes each to the others; copies:
//                   Q by tensor maps over (head element, head of the group,
//                   row), K and V page by page, two stages each
// TMEM columns: S [0, 128), used by both tiles in turn; P_A [128, 192) and
// P_B [192, 256) in 16 bits; O_A, O_B behind.
//
// The softmax takes its whole row of S into registers at once and frees S
// for the other tile's product, which then runs under the exponentials; P
// has columns of its own, so a product S never waits for a product P V.
//
// What it took (4096 tokens over 8192, H 32 / 8, D 128, bfloat16; the four
// products of a pair of tiles take 2150 cycles): one warp whose lane 0 issued
// everything 403 us -- beside eight busy softmax warps each product took 143
// cycles to issue instead of 67; issued by an elected lane of a converged
// warp 365 us -- now its polling of six barriers, 140 cycles a look, set the
// pace; with two issuing warps that wait in a fixed order 312 us;
// 281 us by what blocks do at the ends of units (below); 259 us with P V
// held back until the tile's next S is in the pipe -- the two products of one
// pipe took turns before, which doubled the time until S was there, and S is
// what the softmax waits for.  Slower: P laid over S with a first half of P V
// issued early 477 us, S and P V by one warp in the order in which they get
// ready 313 us (it stalls in the pipe while the other could be looked at),
// issuing warps that spin 304 us (they take the softmax's issue slots), a warp
// of its own for V 270 to 296 us (but 16-key pages then 169 us instead of 200
// at 3200 tokens over 3200: their copies of 2 KB take long to issue).  Now 251 to
// 289 us by the clocks that the power limit leaves, at 168 registers a thread;
// 104 to 112 bytes a thread spill.
//
// The softmax keeps a reference maximum that moves only when a row's maximum
// grows by more than 2^8, so P and O are rarely rescaled; the weights are
// rounded to the type for the product, their sum is taken in float32 before.
// (A second 16-bit part of P would need 128 more TMEM columns and twice the
// products P V.)  In float16 the reference is 2^5 below the maximum, so that P
// reaches 2^13 and loses what is below 2^-30 of the largest weight; with no such
// lift 131,072 keys of 2^-26 each, 2^-9 of the sum, were lost.  (2^3 of room are
// left for the reference's own rounding, 2^2 where scores reach 2^25.)

#include <cmath>
#include <mutex>
#include <type_traits>

#include "kvs_paged.cuh"
#include "kvs_tags.cuh"
#include "kvs_tcgen05.cuh"
#include "kvs_tma.cuh"

namespace kvs {

namespace {

constexpr int kCM = 128;                 // rows of a tile (MMA M)
constexpr int kCN = 128;                 // keys of a tile
constexpr int kCMmaWarp = 8, kCPvWarp = 9, kCCopyWarp = 10;
constexpr int kCThreads = 11 * 32;
// A unit's fixed price and the shortest range worth a block, in cost rows (keys
// of a unit): prompts of 2048 tokens, H 32 / 8, took 61 us at a price of 128
// (and a unit's start and end 1.5 us dearer than now), 49 at 128, 44.7 at 384,
// 45.7 at 512; 512 tokens 26.6 us at a shortest range of 256, 23.0 at 768;
// 20 tokens 31 us at 1024, 11 at 768 or less.
constexpr int kCFix = 384;
constexpr int kCMinRange = 768;
constexpr float kCRescale = 8.f;
template <typename T>
constexpr float kCLift = std::is_same<T, __half>::value ? 5.f : 0.f;
constexpr uint32_t kCTmemCols = 512;
constexpr int kCMaxDevices = 64;

// What the copy warp tells the others of a unit of this block.
struct CUnit {
  int p, row0, tok0, ntok;  // position, first row of the sequence; tokens of the unit
  int t_lo, t_hi;           // key tiles of this block; t_lo == t_hi: no further unit
  int g;                    // kv head
  int bad;                  // a page of it is bad
  int seq, L;               // the sequence and its keys
  int b1, b2[2];            // blocks of its first key tile and of the last ones of tiles A and B
};
constexpr int kCUnits = 4;  // the copy warp is at most so many units ahead

template <int D>
struct CGeo {
  static constexpr int NB = D / 64;               // 128-byte column blocks of a row
  static constexpr int BLK = 128 * 128;           // bytes of a block of 128 rows
  static constexpr int TILE = NB * BLK;           // one tile of Q, K or V
  static constexpr int KS = 2, VS = 2;            // stages
  static constexpr int OFF_Q = 0;                 // Q_A, Q_B
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + KS * TILE;
  static constexpr int OFF_STAGE = OFF_V + VS * TILE;  // 4 KB a softmax warp: rows on their way out
  static constexpr int OFF_BAR = OFF_STAGE + 8 * 4096;
  // q, qfree, kfull[KS], kfree[KS], vfull[VS], vfree[VS], sfull[2],
  // sread, pfull[2], pvdone[2], wg[2], final[2], ufull[kCUnits], ufree[kCUnits], sgone[4]
  static constexpr int NBAR = 2 + 2 * KS + 2 * VS + 2 + 1 + 6 + 2 + 2 * kCUnits + 4;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int OFF_MISC = OFF_TMEM + 8;   // abort, last[2], pad
  static constexpr int OFF_UNIT = OFF_MISC + 16;  // CUnit [kCUnits]
  static constexpr int NEED = OFF_UNIT + kCUnits * (int)sizeof(CUnit);
  // all 512 TMEM columns are this block's: more than half of the SM's shared
  // memory keeps a second block away
  static constexpr int SMEM = NEED > 116 * 1024 ? NEED : 116 * 1024;
  static_assert(SMEM <= 227 * 1024, "one block per SM must fit");
};

// Shared-memory descriptor, 128-byte swizzle (tile bases 1024-byte aligned).
// K-major: stride byte offset between 8-row groups; MN-major: leading byte
// offset between 64-element blocks, stride byte offset between groups of 8 k.
__device__ __forceinline__ uint64_t desc_sw128(const void *p, uint32_t lbo, uint32_t sbo) {
  return smem_desc(p, lbo, sbo) | ((uint64_t)2 << 61);
}

// kind::f16 with FP32 accumulation: A and B both FP16 or both BF16.
template <typename T>
constexpr uint32_t idesc16(int M, int N, bool b_mn_major) {
  const uint32_t bf = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return idesc_f16_f32(M, N) | bf << 7 | bf << 10 | (b_mn_major ? 1u << 16 : 0u);
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

// Box of 64 elements x R rows of one column block (coordinates element, row,
// block) and the Q box (element, head, row, block).
__device__ __forceinline__ void tma_block(void *dst, const CUtensorMap *map, int row, int blk,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(0), "r"(row), "r"(blk), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_q(void *dst, const CUtensorMap *map, int head, int row, int blk,
                                      uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(0), "r"(head), "r"(row), "r"(blk), "r"(smem_addr(bar))
      : "memory");
}

// Upper half of every descriptor here (desc_sw128 with a stride byte offset of
// 1024) and one tile further on in the lower half's 16-byte pieces.
constexpr uint32_t kDescHi = 1024u >> 4 | 1u << 14 | 2u << 29;

// 64 columns of a warp's 32 rows on their way out: a thread puts its own row's
// into shared memory (16-byte pieces swizzled by the row, so that no access
// conflicts), then eight threads a row write them.  Straight from the thread
// that owns the row each store would touch 32 rows (2060 cycles for a tile of
// 128 x 128, against 700).
template <typename T>
__device__ __forceinline__ void put_row32(unsigned char *stg, int lane, int half,
                                          const float (&o)[32], float inv) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    *reinterpret_cast<uint4 *>(stg + lane * 128 + (((4 * half + v) ^ (lane & 7)) * 16)) =
        make_uint4(pack_pair<T>(o[8 * v] * inv, o[8 * v + 1] * inv),
                   pack_pair<T>(o[8 * v + 2] * inv, o[8 * v + 3] * inv),
                   pack_pair<T>(o[8 * v + 4] * inv, o[8 * v + 5] * inv),
                   pack_pair<T>(o[8 * v + 6] * inv, o[8 * v + 7] * inv));
}
// at: where this lane's row starts in out, negative for a row that does not exist
template <typename T>
__device__ __forceinline__ void write_rows64(const unsigned char *stg, int lane, T *out,
                                             long long at, int col) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + lane / 8;
    const long long to = __shfl_sync(0xffffffffu, at, r);
    const uint4 v = *reinterpret_cast<const uint4 *>(stg + r * 128 + (((lane ^ r) & 7) * 16));
    if (to >= 0) *reinterpret_cast<uint4 *>(out + to + col + (lane & 7) * 8) = v;
  }
  __syncwarp();
}

// The pieces of a unit's tile: those of ranges b1 .. b2, the first in its
// slot 1, the others in their slots 0; a piece has each row's (m, l), then
// its accumulators, four columns of all 128 rows after the other (thread t
// writes and reads row t, so a warp moves 512 contiguous bytes).  A row's pieces always join in this way, whichever block
// does it: the largest m first, then weighted sums in range order.
struct Pieces {
  const float *slots;  // of this tile
  size_t stride;       // floats between a block's slots
  int b1, b2;
  __device__ float2 *ml(int c, int row) const {
    float *p = const_cast<float *>(slots) + (2 * (size_t)c + (c == b1 ? 1 : 0)) * stride;
    return reinterpret_cast<float2 *>(p) + row;
  }
  __device__ float4 *acc(int c, int row, int d) const {  // columns d .. d + 3
    float *p = const_cast<float *>(slots) + (2 * (size_t)c + (c == b1 ? 1 : 0)) * stride;
    return reinterpret_cast<float4 *>(p + 2 * kCM) + (d / 4) * kCM + row;
  }
};
// Weight of a piece with maximum m beside the overall maximum mx.
__device__ __forceinline__ float piece_weight(float m, float mx) {
  return ex2(m - (mx == neg_inf_f() ? 0.f : mx));
}

// The two tiles of a unit: tokens, key tiles that each attends, and those of
// this block's column.
struct CTile {
  int tok0, ntok, nt, lo, hi;
};

template <typename T, int D, bool kPoll>
__global__ void __launch_bounds__(kCThreads, 1)
    paged_chunk_kernel(T *__restrict__ out, long long out_stride, PagedArgs pa,
                       const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, int G, int Hkv, int box_shift,
                       float sl2, unsigned char *ws, unsigned host_tag, int *d_status) {
  using C = CGeo<D>;
  constexpr int KS = C::KS, VS = C::VS;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *bar_q = bars;            // Q of the unit landed
  uint64_t *qfree = bar_q + 1;       // the unit's S products done (commit)
  uint64_t *kfull = qfree + 1;       // [KS]
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
  uint64_t *ufree = ufull + kCUnits; // [kCUnits] the ten other warps are done with it
  uint64_t *sgone = ufree + kCUnits;  // [4] S product k of the block issued, at k % 4
  CUnit *units = reinterpret_cast<CUnit *>(smem + C::OFF_UNIT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  volatile int *s_last = abort + 1;  // [2]
  unsigned *epoch = reinterpret_cast<unsigned *>(ws);
  unsigned long long *counters = reinterpret_cast<unsigned long long *>(ws + 256);
  float *slots = reinterpret_cast<float *>(ws + 256 + (size_t)kPagedMaxBlocks * 16);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const int TT = kCM / G;  // tokens of a tile
  constexpr uint32_t kTileStep = C::TILE >> 4;  // one tile further on, in a descriptor
  const Line ln{Hkv, 2 * TT, kCFix, kCN, kCMinRange};

  if (threadIdx.x == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int j = 0; j < C::NBAR; ++j) {  // each once
      uint64_t *bar = bars + j;
      const bool of_warpgroup = bar == sread || bar == pfull || bar == pfull + 1 || bar == wgbar ||
                                bar == wgbar + 1;
      // (an arrival a warp: one a thread took some 200 cycles)
      mbar_init(bar, of_warpgroup ? 4 : bar >= ufree && bar < ufree + kCUnits ? 10 : 1);
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

  const int R = 1 << box_shift;          // rows of a copy
  const int pieces = kCN >> box_shift;   // copies of a tile's column block
  const int piece = lane & (pieces - 1), blk = lane / pieces;  // a copying lane's part of a tile
  // The row of the cache where this lane's part of key tile n starts; live:
  // parts that hold keys; mine: this lane has one.
  struct Part {
    int row, live;
    bool mine, bad;
  };
  auto part_of = [&](int seq, int L, int g, int n) {
    Part c;
    const int key = n * kCN + piece * R;
    c.live = min(pieces, (L - n * kCN + R - 1) / R);
    c.mine = blk < C::NB && piece < c.live;
    int page = c.mine ? __ldca(pa.page_table + (size_t)seq * pa.max_pages + (key >> pa.page_shift)) : 0;
    c.bad = (unsigned)page >= (unsigned)pa.num_pages;
    if (c.bad) page = 0;
    c.row = ((page * Hkv + g) << pa.page_shift) + (key & ((1 << pa.page_shift) - 1));
    return c;
  };
  const uint32_t part_bytes = (uint32_t)(C::NB * R) * 128;  // of all column blocks
  const int part_at = blk * C::BLK + piece * R * 128;

  if (warp == kCCopyWarp) {
    // ======================= units and copies ================================
    int nk = 0, nv = 0, nq = 0;  // K and V tiles issued, units described
    bool ok = true;
    const Cuts cut = equal_cuts(warp_line_total(pa, ln, lane), ln, gridDim.x);
    bool more = cut.R > 0 && b < cut.NS;
    const long long x0 = more ? cut.start(b) : 0, x1 = more ? cut.start(b + 1) : 0;
    Unit u{pa.M, 0, 0, 0};
    if (more) u = warp_unit_at(pa, ln, x0, lane);
    // Describes a unit, once the one before in the same place is done with.
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
        if (!(ok = describe(nq, d))) break;
        if (nq > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(qfree, (uint32_t)(nq - 1) & 1u, abort))))
          break;
        if (lane == 0) {
          const int tiles = f.ntok > TT ? 2 : 1;
          mbar_arrive_expect_tx(bar_q, (uint32_t)(tiles * C::NB * TT * G * 128));
          for (int x = 0; x < tiles; ++x)
            for (int cb = 0; cb < C::NB; ++cb)
              tma_q(smem + C::OFF_Q + x * C::TILE + cb * C::BLK, &qmap, u.g * G,
                    f.s.row0 + f.tok0 + x * TT, cb, bar_q);
        }
        ++nq;
        __syncwarp();
        // in the order in which their places get free: K one tile ahead of V
        Part cv, ck = part_of(u.i, d.L, u.g, f.t_lo);
        for (int n = f.t_lo; n <= f.t_hi && ok; ++n) {
          if (n < f.t_hi) {
            if (ck.bad) {
              record_status(d_status, KVS_ERR_PAGE);
              *const_cast<volatile int *>(&units[(nq - 1) % kCUnits].bad) = 1;
            }
            const int ks = nk % KS;
            if (nk >= KS && !(ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(&kfree[ks], (uint32_t)((nk - KS) / KS) & 1u, abort))))
              break;
            if (lane == 0) mbar_arrive_expect_tx(&kfull[ks], ck.live * part_bytes);
            __syncwarp();
            if (ck.mine) tma_block(smem + C::OFF_K + ks * C::TILE + part_at, &kmap, ck.row, blk, &kfull[ks]);
            ++nk;
          }
          if (n > f.t_lo) {
            const int vs = nv % VS;
            if (nv >= VS && !(ok = __all_sync(0xffffffffu, mbar_wait<kPoll>(&vfree[vs], (uint32_t)((nv - VS) / VS) & 1u, abort))))
              break;
            if (lane == 0) mbar_arrive_expect_tx(&vfull[vs], cv.live * part_bytes);
            __syncwarp();
            if (cv.mine) tma_block(smem + C::OFF_V + vs * C::TILE + part_at, &vmap, cv.row, blk, &vfull[vs]);
            ++nv;
          }
          cv = ck;
          if (n + 1 < f.t_hi) ck = part_of(u.i, d.L, u.g, n + 1);
        }
      }
      more = ok && next_unit(pa, u, f, ln) && u.base < x1;
    }
    if (ok) ok = describe(nq, CUnit{});
    if (lane == 0) {
      if (!ok) give_up(abort, d_status, epoch);
      // every copy issued lands before the block can exit
      if (nq > 0) mbar_wait_drain(bar_q, (uint32_t)(nq - 1) & 1u);
      for (int j = (nk > KS ? nk - KS : 0); j < nk; ++j)
        mbar_wait_drain(&kfull[j % KS], (uint32_t)(j / KS) & 1u);
      for (int j = (nv > VS ? nv - VS : 0); j < nv; ++j)
        mbar_wait_drain(&vfull[j % VS], (uint32_t)(j / VS) & 1u);
    }
    __syncwarp();
  } else if (warp == kCMmaWarp) {
    // ======================= products S ======================================
    // The whole warp runs the loop, converged; an elected lane issues.  Order:
    // S_A(0), S_B(0), S_A(1), ... into the same columns, each once the one
    // before has been read.
    const uint32_t lq = (uint32_t)desc_sw128(smem + C::OFF_Q, 16, 1024);
    const uint32_t lk = lq + ((C::OFF_K - C::OFF_Q) >> 4);
    const uint32_t tm = warp_uniform(tmem);
    constexpr uint32_t kIdS = idesc16<T>(kCM, kCN, false);
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
  } else if (warp == kCPvWarp) {
    // ======================= products P V ====================================
    const uint32_t lv = (uint32_t)desc_sw128(smem + C::OFF_V, C::BLK, 1024);
    const uint32_t tm = warp_uniform(tmem);
    constexpr uint32_t kIdO = idesc16<T>(kCM, D, true);
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
        const int left = f.L - (f.t_lo + j) * kCN;
        if (left < kCN) {
          // rows past the last key hold anything (their weights are zero, but
          // 0 x NaN is not)
          unsigned char *v = smem + C::OFF_V + (gt % VS) * C::TILE;
          for (int e = lane; e < (kCN - left) * 8 * C::NB; e += 32) {
            const int r = left + (e >> 3) / C::NB, bb = (e >> 3) % C::NB;
            *reinterpret_cast<uint4 *>(v + bb * C::BLK + r * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
          __syncwarp();
        }
        const uint32_t bv = warp_uniform(lv + (uint32_t)(gt % VS) * kTileStep);
        const uint32_t acc = warp_uniform(j > 0 ? 1u : 0u);  // O_x (+)= P_x V
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (j >= n_x[x]) continue;
          // O_x += P_x V goes behind the tile's next S.  (sgone is at most two
          // products past the one waited for: the softmax needs this P V
          // before it can read the S after that.)
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
  } else if (warp < 8) {
    // ======================= softmax of tile x ===============================
    const int x = warp >> 2;
    const int t = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + lane_base;
    const uint32_t tm_p = tmem + lane_base + kCN + x * (kCN / 2);
    const uint32_t tm_o = tmem + lane_base + 2 * kCN + x * D;
    const float nan = __int_as_float(0x7fc00000);
    unsigned char *stg = smem + C::OFF_STAGE + warp * 4096;
    int sb = 0;  // S_x products of the earlier units
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
            out[(long long)(q.row0 + r) * out_stride + e] = from_f32<T>(nan);
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
      float m = neg_inf_f(), l = 0.f;
      for (int n = tl.lo; n < tl.hi; ++n) {
        const uint32_t ph = (uint32_t)(sb + n - tl.lo) & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&sfull[x], ph, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
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
        const float cm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2 - kCLift<T>;
        // the reference maximum moves only when the row's grows by more
        // than 2^kCRescale: below that P stays in range and nothing needs
        // rescaling
        const float m_ref = cm > m + kCRescale ? cm : m;
        // (rows that do not exist hold anything: they never ask for a rescale)
        const float alpha = (m == neg_inf_f() || !live) ? 1.f : ex2(m - m_ref);
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
        const float2 sl2x2 = make_float2(sl2, sl2), nmb2 = make_float2(-mb, -mb);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t w[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const float2 x2 = __ffma2_rn(make_float2(r[32 * ch + 2 * v], r[32 * ch + 2 * v + 1]),
                                         sl2x2, nmb2);
            const float p0 = ex2(x2.x), p1 = ex2(x2.y);
            ls[v & 1] = __fadd2_rn(ls[v & 1], make_float2(p0, p1));
            w[v] = pack_pair<T>(p0, p1);
          }
          tmem_st16u(tm_p + ch * 16, w);
        }
        l = l * alpha + ((ls[0].x + ls[1].x) + (ls[0].y + ls[1].y));
        m = m_ref;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[x]);
      }
      if (failed) break;
      sb += tl.hi - tl.lo;
      if (tl.lo < tl.hi) {
        // the tile's last product is done: O_x is final
        if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&pvdone[x], (uint32_t)(sb - 1) & 1u, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
        // (read again: in registers they would crowd out the row)
        const volatile CUnit *ud = &units[nq % kCUnits];
        if (ud->bad) l = nan;
        const bool whole = tl.hi - tl.lo == tl.nt;
        const long long row0 = ud->row0 + tl.tok0;
        const long long at =
            live ? (row0 + tok) * out_stride + (long long)(ud->g * G + (t - tok * G)) * D : -1;
        if (whole) {
          const float inv = 1.f / l;
#pragma unroll 1
          for (int ch = 0; ch < D / 64; ++ch) {
            float o[2][32];
            tmem_ld32(tm_o + ch * 64, o[0]);
            tmem_ld32(tm_o + ch * 64 + 32, o[1]);
            tmem_wait_ld();
            put_row32<T>(stg, lane, 0, o[0], inv);
            put_row32<T>(stg, lane, 1, o[1], inv);
            write_rows64(stg, lane, out, at, ch * 64);
          }
        } else {
          // the blocks of tile x's first and last key tile, and their partials
          const Pieces pc{slots + x * paged_slot_floats(kCM, D), 2 * paged_slot_floats(kCM, D),
                          ud->b1, ud->b2[x]};
          unsigned long long *ctr = counters + 2 * pc.b1 + x;
          const unsigned add = (unsigned)(tl.hi - tl.lo);
          // Usually the other pieces were finished long ago: then this block
          // joins them with the accumulator it still holds in TMEM.
          if (t == 0) {
            const unsigned long long v = ld_acquire_u64(ctr);
            s_last[x] = (unsigned)(v >> 32) == tag && (unsigned)v + add == (unsigned)tl.nt;
          }
          if (!wg_barrier()) {
            failed = true;
            break;
          }
          if (s_last[x]) {
            __threadfence();
            if (t == 0) *ctr = 0ull;  // (no other block will look; a replayed graph uses the tag again)
            if (pc.b2 == pc.b1 + 1) {  // two pieces, the usual unit: all loads first
              const int oc = b == pc.b1 ? pc.b2 : pc.b1;
              const float2 om = __ldcg(pc.ml(oc, t));
#pragma unroll 1
              for (int ch = 0; ch < D / 64; ++ch) {
                float4 q[16];
#pragma unroll
                for (int v = 0; v < 16; ++v) q[v] = __ldcg(pc.acc(oc, t, ch * 64 + 4 * v));
                const float mx = fmaxf(m, om.x);
                const float wo = piece_weight(om.x, mx), ww = piece_weight(m, mx);
                const float ls = b == pc.b1 ? fmaf(wo, om.y, ww * l) : fmaf(ww, l, wo * om.y);
                const float inv = 1.f / ls;
#pragma unroll
                for (int hc = 0; hc < 2; ++hc) {
                  float o[32];
                  tmem_ld32(tm_o + ch * 64 + hc * 32, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int v = 0; v < 32; ++v) {
                    const float4 qq = q[8 * hc + v / 4];
                    const float other = v % 4 == 0 ? qq.x : v % 4 == 1 ? qq.y : v % 4 == 2 ? qq.z : qq.w;
                    o[v] = b == pc.b1 ? fmaf(wo, other, ww * o[v]) : fmaf(ww, o[v], wo * other);
                  }
                  put_row32<T>(stg, lane, hc, o, inv);
                }
                write_rows64(stg, lane, out, at, ch * 64);
              }
            } else {
            float mx = m;
            for (int c = pc.b1; c <= pc.b2; ++c)
              if (c != b) mx = fmaxf(mx, __ldcg(pc.ml(c, t)).x);
            float ls = 0.f;
            for (int c = pc.b1; c <= pc.b2; ++c) {
              const float2 ml = c == b ? make_float2(m, l) : __ldcg(pc.ml(c, t));
              ls = fmaf(piece_weight(ml.x, mx), ml.y, ls);
            }
            const float inv = 1.f / ls;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              float o[32], acc[32];
              tmem_ld32(tm_o + ch * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int v = 0; v < 32; ++v) acc[v] = 0.f;
              for (int c = pc.b1; c <= pc.b2; ++c) {
                if (c == b) {
                  const float w = piece_weight(m, mx);
#pragma unroll
                  for (int v = 0; v < 32; ++v) acc[v] = fmaf(w, o[v], acc[v]);
                } else {
                  float4 q[8];
#pragma unroll
                  for (int v = 0; v < 8; ++v) q[v] = __ldcg(pc.acc(c, t, ch * 32 + 4 * v));
                  const float w = piece_weight(__ldcg(pc.ml(c, t)).x, mx);
#pragma unroll
                  for (int v = 0; v < 8; ++v) {
                    acc[4 * v] = fmaf(w, q[v].x, acc[4 * v]);
                    acc[4 * v + 1] = fmaf(w, q[v].y, acc[4 * v + 1]);
                    acc[4 * v + 2] = fmaf(w, q[v].z, acc[4 * v + 2]);
                    acc[4 * v + 3] = fmaf(w, q[v].w, acc[4 * v + 3]);
                  }
                }
              }
              put_row32<T>(stg, lane, ch & 1, acc, inv);
              if (ch & 1) write_rows64(stg, lane, out, at, (ch - 1) * 32);
            }
            }
          } else {
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              float o[32];
              tmem_ld32(tm_o + ch * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int v = 0; v < 8; ++v)
                __stcg(pc.acc(b, t, ch * 32 + 4 * v),
                       make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]));
            }
            __stcg(pc.ml(b, t), make_float2(m, l));
            __threadfence();  // the partial is visible GPU-wide before it counts
            if (!wg_barrier()) {
              failed = true;
              break;
            }
            if (t == 0) {
              const unsigned before = tagged_add(ctr, add, tag, d_status, epoch);
              const bool fin = before != 0xffffffffu && before + add == (unsigned)tl.nt;
              if (fin) *ctr = 0ull;
              s_last[x] = fin;
            }
            if (!wg_barrier()) {
              failed = true;
              break;
            }
            if (s_last[x]) {
              // (the others finished in the meantime: all pieces from memory)
              __threadfence();
              float mx = neg_inf_f(), ls = 0.f;
              for (int c = pc.b1; c <= pc.b2; ++c) mx = fmaxf(mx, __ldcg(pc.ml(c, t)).x);
              for (int c = pc.b1; c <= pc.b2; ++c) {
                const float2 ml = __ldcg(pc.ml(c, t));
                ls = fmaf(piece_weight(ml.x, mx), ml.y, ls);
              }
              const float inv = 1.f / ls;
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ++ch) {
                float acc[32];
#pragma unroll
                for (int v = 0; v < 32; ++v) acc[v] = 0.f;
                for (int c = pc.b1; c <= pc.b2; ++c) {
                  const float w = piece_weight(__ldcg(pc.ml(c, t)).x, mx);
#pragma unroll
                  for (int v = 0; v < 8; ++v) {
                    const float4 q = __ldcg(pc.acc(c, t, ch * 32 + 4 * v));
                    acc[4 * v] = fmaf(w, q.x, acc[4 * v]);
                    acc[4 * v + 1] = fmaf(w, q.y, acc[4 * v + 1]);
                    acc[4 * v + 2] = fmaf(w, q.z, acc[4 * v + 2]);
                    acc[4 * v + 3] = fmaf(w, q.w, acc[4 * v + 3]);
                  }
                }
                put_row32<T>(stg, lane, ch & 1, acc, inv);
              if (ch & 1) write_rows64(stg, lane, out, at, (ch - 1) * 32);
              }
            }
          }
        }
      }
      unit_done(nq);
    }
    if (failed && lane == 0) give_up(abort, d_status, epoch);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kCTmemCols);
}

template <typename T, int D>
int launch_chunk(const void *q, long long q_stride, const kvs_paged_cache &cache,
                 const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                 int *d_status, cudaStream_t stream) {
  using C = CGeo<D>;
  static bool configured[kCMaxDevices] = {false};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kCMaxDevices) return KVS_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      for (auto kern : {paged_chunk_kernel<T, D, false>, paged_chunk_kernel<T, D, true>}) {
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
  CUtensorMap qmap, kmap, vmap;
  const uint64_t rows = (uint64_t)cache.num_pages * Hkv * cache.page_size;
  const int box_shift = pa.page_shift < 7 ? pa.page_shift : 7;
  int rc = make_row_map(&kmap, cache.k_pages, rows, D, cache.dtype, 1 << box_shift, 1);
  if (rc == KVS_OK) rc = make_row_map(&vmap, cache.v_pages, rows, D, cache.dtype, 1 << box_shift, 1);
  if (rc == KVS_OK)
    rc = make_q_map(&qmap, q, pa.num_rows, q_stride, H, D, cache.dtype, kCM / G, G);
  if (rc != KVS_OK) return rc;
  const int grid = sms < kPagedMaxBlocks ? sms : kPagedMaxBlocks;
  const float sl2 = (float)(1.4426950408889634074 / std::sqrt((double)D));
  const cudaError_t e = launch_pdl(
      poll_waits() ? paged_chunk_kernel<T, D, true> : paged_chunk_kernel<T, D, false>, dim3(grid),
      dim3(kCThreads), C::SMEM, stream, static_cast<T *>(out), out_stride, pa, qmap, kmap, vmap, G,
      Hkv, box_shift, sl2, static_cast<unsigned char *>(workspace), fresh_tag(), d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

}  // namespace

int set_wait_limit_chunk(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

// Workspace: 256 bytes (epoch), two counters a block (tiles A and B), then
// per block two units' partials (begun earlier, not finished), each two tiles.
size_t paged_chunk_workspace_bytes(int D) {
  return 256 + (size_t)kPagedMaxBlocks * 16 +
         4 * (size_t)kPagedMaxBlocks * paged_slot_floats(kCM, D) * 4;
}

int launch_paged_chunk(const void *q, long long q_stride, const kvs_paged_cache &cache,
                       const PagedArgs &pa, void *out, long long out_stride, int H,
                       void *workspace, int *d_status, cudaStream_t stream) {
#define KVS_CHUNK(T)                                                                            \
  return cache.head_dim == 64                                                                   \
             ? launch_chunk<T, 64>(q, q_stride, cache, pa, out, out_stride, H, workspace,       \
                                   d_status, stream)                                            \
             : launch_chunk<T, 128>(q, q_stride, cache, pa, out, out_stride, H, workspace,      \
                                    d_status, stream)
  if (cache.dtype == KVS_F16) KVS_CHUNK(__half);
  if (cache.dtype == KVS_BF16) KVS_CHUNK(__nv_bfloat16);
#undef KVS_CHUNK
  return KVS_ERR_UNSUPPORTED;
}

}  // namespace kvs
