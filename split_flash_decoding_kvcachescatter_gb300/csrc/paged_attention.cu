// paged_attention.cu -- attention of a ragged batch's new tokens over a paged
// KV cache: the choice of kernel, and the kernel for chunks in float32.
//
// Mathematics: flash attention over a split key axis.  For a row (token,
// query head) and a set of keys, (m, l, acc) = (max s_j, sum 2^(s_j - m),
// sum 2^(s_j - m) v_j), s_j = log2(e) q.k_j / sqrt(D); sets merge by
// rescaling to the larger m, and the row's output is acc / l.
//
// Work unit of all kernels: (sequence, row tile, kv head).  A row tile
// is TT = RT / G whole tokens with the G query heads of the group: RT rows
// share every K and V row.  Units follow each other on one line of "cost
// rows" (a fixed price, then one per key a unit attends); the line is cut
// into ranges, whatever the lengths are: a block runs the key tiles that
// start in its range.  A unit inside one range is written directly; the
// pieces of a unit that spans ranges go to the workspace, and the block that
// completes the unit merges them in order (the tagged counters of
// kvs_tags.cuh; no block waits for another).  Everything is derived on the
// device from the positions and offsets, so a captured graph follows them.
//
// Kernels: rows that a unit's 16 can hold (max_new G <= 16: a decode step)
// paged_decode.cu; more rows in 16 bits paged_chunk.cu (tcgen05); more rows
// in float32 the one here, on mma.sync: float32 as three TF32 products of a
// high and a low part (hi hi + hi lo + lo hi), off by 2^-21 of it at most (lo lo 2^-22,
// a lost bit of each lo 2^-23).
//
// Block: one producer warp and 7 consumer warps of 16 rows (eight warps, so
// that a thread may have 255 registers), which share a ring of stages (K and
// V of one tile, swizzled 128-byte column blocks, moved by tensor-map copies
// of 16 rows, each looked up in the page table).
//
// Measured: 1001 new tokens of three sequences over up to 2048, H 14 / 2, D 64:
// 57 to 74 us by the positions (65 us at 3.7 GFLOP, whose three TF32 products
// would take 36 us at the 303 TFLOP/s that mma.sync reaches here; splitting the
// operands and the softmax take the rest).  At positions where it took 82 us:
// 101 with the pieces of split units joined from memory by one group of threads;
// dearer units in the split 84 us (128 cost rows) and 92 (256); 11 warps of fewer
// registers 84.  1001 tokens over up to 1900, H 40 / 8, D 128: 483 us
// (22.6 GFLOP; 223 us).

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
constexpr int kRFix = 64;             // cost rows that stand for a unit's fixed price
constexpr int kRMaxDevices = 64;

template <int D_>
struct RGeo {
  static constexpr int D = D_;
  static constexpr int KT = WarpRows<float, D>::KT;  // keys of a tile
  static constexpr int GB = 16 * D * 4;              // bytes of a 16-row copy
  static constexpr int BLK = 2048;                   // one of its column blocks
  static constexpr int TILE = KT / 16 * GB;          // K (or V) of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int S = 8;                        // stages of the ring
  static constexpr int OFF_BAR = S * STAGE;
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
template <int D>
__device__ __forceinline__ void join_pieces(WarpRows<float, D> &w, const float *slots, int b1,
                                            int b2, int own) {
  constexpr int kThreads = kRWarps * 32;
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
    ls[0] = fmaf(wt[0], ml.y, ls[0]);  // (a NaN sum stays one also under a zero weight)
    ls[1] = fmaf(wt[1], ml.w, ls[1]);
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

template <int D, bool kPoll>
__global__ void __launch_bounds__(kRThreads, 1)
    paged_rows_kernel(const float *__restrict__ q, long long q_stride, float *__restrict__ out,
                      long long out_stride, PagedArgs pa, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, int G, int Hkv, float sl2,
                      unsigned char *ws, unsigned host_tag, int *d_status) {
  using C = RGeo<D>;
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
  const Line ln{Hkv, kRRows / G, kRFix, C::KT, C::KT + kRFix};
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 1);
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
          tma_rows(dst, lane >= NP ? &vmap : &kmap, row, &full[st], policy);
        }
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
  WarpRows<float, D> w;
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
            for (int e = lane; e < (C::KT - left) * (D / 4); e += 32) {
              const int row = left + e % (C::KT - left), pc = e / (C::KT - left);
              *reinterpret_cast<uint4 *>(sk + C::TILE + (row >> 4) * C::GB + (pc >> 3) * C::BLK +
                                         (row & 15) * 128 + (pc & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_shared();
          }
          if (!consumers_barrier()) return;
        }
        if (any_rows && t * C::KT < warp_reach) {
          const int lim[2] = {reach[0] - t * C::KT, reach[1] - t * C::KT};
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
          join_pieces<D>(w, slots, b1, b2, b);
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
            join_pieces<D>(w, slots, b1, b2, -1);
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

template <int D>
int launch_rows(const void *q, long long q_stride, const kvs_paged_cache &cache,
                const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                int *d_status, cudaStream_t stream) {
  using C = RGeo<D>;
  static bool configured[kRMaxDevices] = {false};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kRMaxDevices) return KVS_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      for (auto kern : {paged_rows_kernel<D, false>, paged_rows_kernel<D, true>}) {
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
  int rc = make_row_map(&kmap, cache.k_pages, rows, D, cache.dtype, 16, D / 32);
  if (rc == KVS_OK) rc = make_row_map(&vmap, cache.v_pages, rows, D, cache.dtype, 16, D / 32);
  if (rc != KVS_OK) return rc;
  const int Hkv = cache.num_kv_heads;
  const int grid = sms < kPagedMaxBlocks ? sms : kPagedMaxBlocks;
  const float sl2 = (float)(1.4426950408889634074 / std::sqrt((double)D));
  const cudaError_t e = launch_pdl(
      poll_waits() ? paged_rows_kernel<D, true> : paged_rows_kernel<D, false>, dim3(grid),
      dim3(kRThreads), C::SMEM, stream, static_cast<const float *>(q), q_stride,
      static_cast<float *>(out), out_stride, pa, kmap, vmap, H / Hkv, Hkv, sl2,
      static_cast<unsigned char *>(workspace), fresh_tag(), d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

// A decode step: every sequence's rows with the G heads of a group fit the 16
// rows of a paged_decode unit.
bool is_decode(long long max_new, int G) { return max_new * G <= 16; }

}  // namespace

int set_wait_limit_paged(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

size_t paged_attention_workspace_bytes(int H, int Hkv, int D, int max_new) {
  if (is_decode(max_new, H / Hkv)) return paged_decode_workspace_bytes(D);
  return std::max(rows_workspace_bytes(D), paged_chunk_workspace_bytes(D));
}

int launch_paged_attention(const void *q, long long q_stride, const kvs_paged_cache &cache,
                           const PagedArgs &pa, void *out, long long out_stride, int H,
                           void *workspace, int *d_status, cudaStream_t stream) {
  if (is_decode(pa.max_new, H / cache.num_kv_heads))
    return launch_paged_decode(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status,
                               stream);
  if (cache.dtype != KVS_F32)
    return launch_paged_chunk(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status,
                              stream);
  if (cache.head_dim == 64)
    return launch_rows<64>(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status, stream);
  return launch_rows<128>(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status, stream);
}

}  // namespace kvs
