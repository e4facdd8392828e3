// kvs_rows.cuh -- attention of chunks of new tokens in float32 over a paged KV
// cache, on mma.sync: the kernel and its launch, for the plain pages of
// paged_attention.cu and the 8-bit ones of paged_rows_q8.cu.  Mathematics,
// units and ranges as in paged_attention.cu.
//
// Block: one producer warp and 7 consumer warps of 16 rows (eight warps, so
// that a thread may have 255 registers), which share a ring of stages (K and
// V of one tile, swizzled 128-byte column blocks, moved by tensor-map copies
// of 16 rows, each looked up in the page table).
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

constexpr int kRWarps = 7;            // consumer warps
constexpr int kRRows = 16 * kRWarps;  // rows of a unit
constexpr int kRThreads = (kRWarps + 1) * 32;
constexpr int kRMaxDevices = 64;

// What the kernel needs to know of the pages is its policy P: the head size D, the bytes
// kElem of an element, the warp's rows (WarpRows or a class like it), whether 16 keys share
// a scale (kScaled), the cost rows kFix that stand for a unit's fixed price, and what a
// launch passes beside the tensor maps (Extra).
template <class P>
struct RGeo {
  static constexpr int D = P::D;
  static constexpr int KT = P::Rows::KT;             // keys of a tile
  static constexpr int GB = 16 * D * P::kElem;       // bytes of a 16-row copy
  static constexpr int TILE = KT / 16 * GB;          // K (or V) of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int SCALES = P::kScaled ? 2 * KT / 16 * 4 : 0;  // bytes of a stage's scales
  static constexpr int S = 8;                        // stages of the ring
  // arrivals that fill a stage: the one that expects the copies, and with scales
  // each lane's, made when its part of them has landed
  static constexpr int FULL = P::kScaled ? 33 : 1;
  static constexpr int OFF_SCALE = S * STAGE;        // float [S][2][KT / 16]
  static constexpr int OFF_BAR = OFF_SCALE + S * SCALES;
  static constexpr int OFF_BAD = OFF_BAR + (2 * S + 1) * 8;  // int [S]
  static constexpr int OFF_MISC = OFF_BAD + S * 4;           // abort, last
  // one block an SM (a second one would find no registers)
  static constexpr int SMEM = OFF_MISC + 8;
  static_assert(SMEM <= 227 * 1024, "one block per SM must fit");
};

// Workspace: 256 bytes (epoch), a counter per block, then per block two
// partial slots (0: a unit begun in an earlier range, 1: one begun here and
// not finished) as the threads hold them: a float4 (m, l, m, l) of every
// thread's two rows, then the threads' accumulators, a float4 of all threads
// after the other.
__host__ __device__ constexpr size_t rows_slot_floats(int D) {
  return (size_t)kRWarps * 32 * 4 * (1 + D / 8);
}
inline size_t rows_workspace_bytes(int D) {
  return 256 + (size_t)kPagedMaxBlocks * 8 +
         2 * (size_t)kPagedMaxBlocks * rows_slot_floats(D) * 4;
}

// A thread's rows joined over a unit's pieces (ranges b1 .. b2, the first in
// its slot 1, the others in their slots 0): the largest m first, then weighted
// sums in range order, whichever block joins.  Piece `own` is in registers
// (w), the others come from the workspace; own = -1: all of them.  Leaves
// the joined accumulators in w.o and the row sums in w.l.
template <class P>
__device__ __forceinline__ void join_pieces(typename P::Rows &w, const float *slots, int b1,
                                            int b2, int own) {
  constexpr int D = P::D, kThreads = kRWarps * 32;
  auto slot = [&](int c) {
    return reinterpret_cast<const float4 *>(slots + (2 * (size_t)c + (c == b1 ? 1 : 0)) *
                                                        rows_slot_floats(D)) + threadIdx.x;
  };
  const float4 mine = make_float4(w.m[0], w.l[0], w.m[1], w.l[1]);
  float mx[2] = {neg_inf_f(), neg_inf_f()};
  for (int c = b1; c <= b2; ++c) {
    const float4 ml = c == own ? mine : __ldcg(slot(c));
    mx[0] = fmaxf(mx[0], ml.x);
    mx[1] = fmaxf(mx[1], ml.z);
  }
  const float mz[2] = {mx[0] == neg_inf_f() ? 0.f : mx[0], mx[1] == neg_inf_f() ? 0.f : mx[1]};
  float acc[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  float ls[2] = {0.f, 0.f};
  for (int c = b1; c <= b2; ++c) {
    float4 v[D / 8];
    const float4 ml = c == own ? mine : __ldcg(slot(c));
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
      v[j] = c == own ? make_float4(w.o[j][0], w.o[j][1], w.o[j][2], w.o[j][3])
                      : __ldcg(slot(c) + (j + 1) * kThreads);
    const float wt[2] = {ex2f(ml.x - mz[0]), ex2f(ml.z - mz[1])};
    ls[0] = add_sum<P::kScaled>(ls[0], ml.y, ml.x - mz[0], wt[0]);  // (a NaN sum stays one also under a zero weight)
    ls[1] = add_sum<P::kScaled>(ls[1], ml.w, ml.z - mz[1], wt[1]);
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      acc[j][0] = fmaf(wt[0], v[j].x, acc[j][0]);
      acc[j][1] = fmaf(wt[0], v[j].y, acc[j][1]);
      acc[j][2] = fmaf(wt[1], v[j].z, acc[j][2]);
      acc[j][3] = fmaf(wt[1], v[j].w, acc[j][3]);
    }
  }
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) w.o[j][e] = acc[j][e];
  w.l[0] = ls[0];
  w.l[1] = ls[1];
}

template <class P, bool kPoll>
__global__ void __launch_bounds__(kRThreads, 1)
    paged_rows_kernel(const float *__restrict__ q, long long q_stride, float *__restrict__ out,
                      long long out_stride, PagedArgs pa, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, int G, int Hkv, float sl2,
                      unsigned char *ws, unsigned host_tag, typename P::Extra extra, int *d_status) {
  constexpr int D = P::D;
  using C = RGeo<P>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [S]
  uint64_t *empty = full + C::S;
  uint64_t *cbar = empty + C::S;  // all consumer warps
  int *bad = reinterpret_cast<int *>(smem + C::OFF_BAD);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  volatile int *s_last = abort + 1;
  unsigned *epoch = reinterpret_cast<unsigned *>(ws);
  unsigned long long *counters = reinterpret_cast<unsigned long long *>(ws + 256);
  float *slots = reinterpret_cast<float *>(ws + 256 + (size_t)kPagedMaxBlocks * 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const Line ln{Hkv, kRRows / G, P::kFix, C::KT, C::KT + P::kFix};
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], C::FULL);
      mbar_init(&empty[s], kRWarps);
    }
    mbar_init(cbar, kRWarps);
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
      const float nan = __int_as_float(0x7fc00000);
      for (int r = 0; r < s.n; ++r)
        for (int e = threadIdx.x; e < Hkv * G * D; e += kRThreads)
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

  if (warp == kRWarps) {
    // ======================= producer =======================================
    const uint64_t policy = policy_evict_normal();  // row tiles share rows through L2
    uint32_t n = 0;  // tiles put in the ring
    bool ok = true;
    constexpr int NP = C::KT / 16;  // 16-row pieces of a tile
    constexpr int AHEAD = 32 / NP;  // tiles whose pages one look-up finds
    const int piece = lane % NP;    // lanes 0..NP-1: K pieces, NP..2NP-1: V pieces
    do {
      const UnitInfo f = unit_info(pa, u, ln, x0, x1);
      const int32_t *table = pa.page_table + (size_t)u.i * pa.max_pages;
      int page = 0, k = 0;  // lane: the page of piece `piece` of tile k + lane / NP
      for (int t = f.t_lo; t < f.t_hi; ++t, ++n, ++k) {
        if (k % AHEAD == 0) {
          const int r0 = (t + lane / NP) * C::KT + 16 * piece;
          page = r0 < f.keys ? __ldca(table + (r0 >> pa.page_shift)) : 0;
        }
        const int pg = __shfl_sync(0xffffffffu, page, (k % AHEAD) * NP + piece);
        const int npieces = min(NP, (f.keys - t * C::KT + 15) / 16);
        const bool mine = lane < 2 * NP && piece < npieces;
        const bool wrong = mine && (unsigned)pg >= (unsigned)pa.num_pages;
        const unsigned any_bad = __ballot_sync(0xffffffffu, wrong);
        const int st = (int)(n % C::S);
        if (!__all_sync(0xffffffffu,
                        mbar_wait<kPoll>(&empty[st], ((n / C::S) & 1u) ^ 1u, abort))) {
          ok = false;
          break;
        }
        [[maybe_unused]] float *scales = reinterpret_cast<float *>(smem + C::OFF_SCALE + st * C::SCALES);
        if constexpr (P::kScaled) {  // (groups behind the last key: any scale that is a number)
          if (lane < 2 * NP && !mine) scales[lane] = 1.f;
          __syncwarp();
        }
        if (lane == 0) {
          bad[st] = any_bad != 0u;
          if (any_bad) record_status(d_status, KVS_ERR_PAGE);
          mbar_arrive_expect_tx(&full[st], 2u * (uint32_t)npieces * C::GB);
        }
        __syncwarp();
        if (mine) {
          const int r0 = t * C::KT + 16 * piece;
          const int row = ((wrong ? 0 : pg) * Hkv + u.g) * (1 << pa.page_shift) +
                          (r0 & ((1 << pa.page_shift) - 1));
          unsigned char *dst = smem + st * C::STAGE + (lane >= NP ? C::TILE : 0) + piece * C::GB;
          tma_rows(dst, lane >= NP ? &vmap : &kmap, P::map_row(row), &full[st], policy);
          if constexpr (P::kScaled)
            copy_async4(&scales[lane], (lane >= NP ? extra.v_scales : extra.k_scales) + (row >> 4));
        }
        if constexpr (P::kScaled) arrive_when_copied(&full[st]);
      }
      if (!ok) break;
      if (!next_unit(pa, u, f, ln)) break;
    } while (u.base < x1);
    if (lane == 0) {
      if (!ok) give_up(abort, d_status, epoch);
      // every copy lands before the block exits
      for (uint32_t j = n > (uint32_t)C::S ? n - C::S : 0u; j < n; ++j)
        mbar_wait_drain(&full[j % C::S], (j / C::S) & 1u);
    }
    return;
  }

  // ========================= consumers ======================================
  uint32_t n = 0, cphase = 0;
  auto consumers_barrier = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(cbar);
    const bool got = __all_sync(0xffffffffu, mbar_wait<kPoll>(cbar, cphase, abort));
    if (!got) {
      if (lane == 0) give_up(abort, d_status, epoch);
      return false;
    }
    cphase ^= 1u;
    return true;
  };
  typename P::Rows w;
  do {
    const UnitInfo f = unit_info(pa, u, ln, x0, x1);
    if (f.t_lo < f.t_hi) {
      const int rows = f.ntok * G;
      const bool any_rows = 16 * warp < rows;  // (a warp past the rows only keeps the ring going)
      w.start(q, q_stride, warp, rows, G, f, u.g);
      int reach[2];  // keys that this lane's two rows attend
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        reach[hh] = f.s.p + f.tok0 + min(16 * warp + lane / 4 + 8 * hh, rows - 1) / G + 1;
      const int warp_reach = f.s.p + f.tok0 + min(16 * warp + 15, rows - 1) / G + 1;
      bool poison = false;
      for (int t = f.t_lo; t < f.t_hi; ++t, ++n) {
        const int st = (int)(n % C::S);
        if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&full[st], (n / C::S) & 1u, abort))) {
          if (lane == 0) give_up(abort, d_status, epoch);
          return;
        }
        poison |= bad[st] != 0;
        unsigned char *sk = smem + st * C::STAGE;
        const int left = f.keys - t * C::KT;  // keys of the tile that exist
        if (left < C::KT) {
          // rows past the last key hold anything: V's become zero (their
          // weights are zero, but 0 x NaN is not); it is the unit's last
          // tile, and all warps meet here
          if (warp == 0) {
            P::clear_rows(sk + C::TILE, left);
            fence_proxy_async_shared();
          }
          if (!consumers_barrier()) return;
        }
        if (any_rows && t * C::KT < warp_reach) {
          const int lim[2] = {reach[0] - t * C::KT, reach[1] - t * C::KT};
          if constexpr (P::kScaled)
            w.tile(smem_addr(sk), smem_addr(sk + C::TILE),
                   reinterpret_cast<const float *>(smem + C::OFF_SCALE + st * C::SCALES), sl2, lim);
          else
            w.tile(smem_addr(sk), smem_addr(sk + C::TILE), sl2, lim);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
      w.finish();
      if (poison) w.l[0] = w.l[1] = __int_as_float(0x7fc00000);
      float *orow = out + (long long)(f.s.row0 + f.tok0) * out_stride + (long long)u.g * G * D;
      bool write = f.t_hi - f.t_lo == f.nt;  // the whole unit is here, or joined here
      if (!write) {
        // the ranges of the unit's first and last tile; every range between has some
        const int b1 = cut.at(f.k0);
        const int b2 = cut.at(f.k0 + (long long)(f.nt - 1) * C::KT);
        unsigned long long *ctr = counters + b1;
        const unsigned add = (unsigned)(f.t_hi - f.t_lo);
        // usually the other pieces were finished long ago: then this block
        // joins them with the accumulators it still holds
        if (threadIdx.x == 0) {
          const unsigned long long v = ld_acquire_u64(ctr);
          *s_last = (unsigned)(v >> 32) == tag && (unsigned)v + add == (unsigned)f.nt;
        }
        if (!consumers_barrier()) return;
        write = *s_last != 0;
        if (write) {
          __threadfence();
          if (threadIdx.x == 0) *ctr = 0ull;  // (a replayed graph uses the tag again)
          join_pieces<P>(w, slots, b1, b2, b);
        } else {
          float4 *sl = reinterpret_cast<float4 *>(slots + (2 * (size_t)b + (f.t_lo == 0 ? 1 : 0)) *
                                                              rows_slot_floats(D)) + threadIdx.x;
          __stcg(sl, make_float4(w.m[0], w.l[0], w.m[1], w.l[1]));
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            __stcg(sl + (j + 1) * kRWarps * 32, make_float4(w.o[j][0], w.o[j][1], w.o[j][2], w.o[j][3]));
          __threadfence();  // the partial is visible GPU-wide before it counts
          if (!consumers_barrier()) return;
          if (threadIdx.x == 0) {
            const unsigned before = tagged_add(ctr, add, tag, d_status, epoch);
            const bool last = before != 0xffffffffu && before + add == (unsigned)f.nt;
            if (last) *ctr = 0ull;
            *s_last = last;
          }
          if (!consumers_barrier()) return;
          write = *s_last != 0;
          if (write) {
            __threadfence();
            join_pieces<P>(w, slots, b1, b2, -1);
          }
        }
        if (!consumers_barrier()) return;  // (s_last has been read)
      }
      if (write && any_rows) {
        const float inv[2] = {1.f / w.l[0], 1.f / w.l[1]};
        w.each([&](int hh, int d, const float(&v)[4]) {
          const int r = 16 * warp + lane / 4 + 8 * hh;
          if (r >= rows) return;
          const int tok = r / G;
          *reinterpret_cast<float4 *>(orow + (long long)tok * out_stride + (r - tok * G) * D + d) =
              make_float4(v[0] * inv[hh], v[1] * inv[hh], v[2] * inv[hh], v[3] * inv[hh]);
        });
      }
    }
    if (!next_unit(pa, u, f, ln)) break;
  } while (u.base < x1);
}

// Hkv kv heads; kmap and vmap: boxes of 16 rows of the pages.
template <class P>
int launch_rows(const void *q, long long q_stride, const CUtensorMap &kmap, const CUtensorMap &vmap,
                const typename P::Extra &extra, int Hkv, const PagedArgs &pa, void *out,
                long long out_stride, int H, void *workspace, int *d_status, cudaStream_t stream) {
  using C = RGeo<P>;
  static bool configured[kRMaxDevices] = {false};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kRMaxDevices) return KVS_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      for (auto kern : {paged_rows_kernel<P, false>, paged_rows_kernel<P, true>}) {
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
  const float sl2 = (float)(1.4426950408889634074 / std::sqrt((double)P::D));
  const cudaError_t e = launch_pdl(
      poll_waits() ? paged_rows_kernel<P, true> : paged_rows_kernel<P, false>, dim3(grid),
      dim3(kRThreads), C::SMEM, stream, static_cast<const float *>(q), q_stride,
      static_cast<float *>(out), out_stride, pa, kmap, vmap, H / Hkv, Hkv, sl2,
      static_cast<unsigned char *>(workspace), fresh_tag(), extra, d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

}  // namespace

}  // namespace kvs
