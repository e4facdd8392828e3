// kvs_chunk.cuh -- what the tcgen05 kernels for chunks of new tokens over a
// paged cache share (paged_chunk.cu has the mathematics, the split and the block's
// layout): units, descriptors, a tile's way out and the joining of its pieces.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <type_traits>

#include "kvs_paged.cuh"
#include "kvs_tags.cuh"
#include "kvs_tcgen05.cuh"
#include "kvs_tma.cuh"

namespace kvs {

namespace {

constexpr int kCM = 128;                 // rows of a tile (MMA M)
constexpr int kCN = 128;                 // keys of a tile
constexpr float kCRescale = 8.f;         // a row's reference moves when its maximum grows by more than 2^this
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

// The way out in steps of 32 columns: through 4 KB of shared memory a warp, as above
// (kStaged), or, where that is taken, by each thread into its own row.
template <typename T, bool kStaged>
__device__ __forceinline__ void put_columns(unsigned char *stg, int lane, T *out, long long at,
                                            int c32, const float (&o)[32], float inv) {
  if constexpr (kStaged) {
    put_row32<T>(stg, lane, c32 & 1, o, inv);
    if (c32 & 1) write_rows64(stg, lane, out, at, (c32 - 1) * 32);
  } else if (at >= 0) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *reinterpret_cast<uint4 *>(out + at + c32 * 32 + 8 * v) =
          make_uint4(pack_pair<T>(o[8 * v] * inv, o[8 * v + 1] * inv),
                     pack_pair<T>(o[8 * v + 2] * inv, o[8 * v + 3] * inv),
                     pack_pair<T>(o[8 * v + 4] * inv, o[8 * v + 5] * inv),
                     pack_pair<T>(o[8 * v + 6] * inv, o[8 * v + 7] * inv));
  }
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
// ls + the share of its sum l.
template <bool kFar>
__device__ __forceinline__ float add_piece(float ls, float l, float m, float mx) {
  return add_sum<kFar>(ls, l, m - (mx == neg_inf_f() ? 0.f : mx), kFar ? 0.f : piece_weight(m, mx));
}

// The two tiles of a unit: tokens, key tiles that each attends, and those of
// this block's column.
struct CTile {
  int tok0, ntok, nt, lo, hi;
};

// Tile x of a block's unit, all of whose products are done: its rows to out, or,
// where other blocks have key tiles of it, its piece to the workspace, or to out
// joined with theirs by the block that completes it.  By the tile's four warps
// (thread t has row t: live, token tok of the tile, running maximum m and sum l,
// accumulators at tm_o); false when a wait ran out.
// kFar (8-bit pages): sums as add_sum's (kvs_paged.cuh), and units of more than two pieces join
// from memory alone: each 100 instructions here cost that kernel's loops time, which fill
// the instruction cache (4096 tokens over 8192 382 us with the two ways, 349 with one).
template <typename T, int D, bool kStaged, bool kFar, class Barrier>
__device__ __forceinline__ bool finish_tile(T *out, long long out_stride, const volatile CUnit *ud,
                                            const CTile &tl, int x, int t, int lane, bool live,
                                            int tok, int G, int b, uint32_t tm_o, float m, float l,
                                            unsigned char *stg, float *slots,
                                            unsigned long long *counters, unsigned tag,
                                            unsigned *epoch, int *d_status, volatile int *s_last,
                                            Barrier wg_barrier) {
  const float nan = __int_as_float(0x7fc00000);
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
      put_columns<T, kStaged>(stg, lane, out, at, 2 * ch, o[0], inv);
      put_columns<T, kStaged>(stg, lane, out, at, 2 * ch + 1, o[1], inv);
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
      s_last[x] = (unsigned)(v >> 32) == tag && (unsigned)v + add == (unsigned)tl.nt &&
                  (!kFar || pc.b2 == pc.b1 + 1);
    }
    if (!wg_barrier()) return false;
    if (s_last[x]) {
      __threadfence();
      if (t == 0) *ctr = 0ull;  // (no other block will look; a replayed graph uses the tag again)
      if (kFar || pc.b2 == pc.b1 + 1) {  // two pieces, the usual unit: all loads first
        const int oc = b == pc.b1 ? pc.b2 : pc.b1;
        const float2 om = __ldcg(pc.ml(oc, t));
#pragma unroll 1
        for (int ch = 0; ch < D / 64; ++ch) {
          float4 q[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) q[v] = __ldcg(pc.acc(oc, t, ch * 64 + 4 * v));
          const float mx = fmaxf(m, om.x);
          const float wo = piece_weight(om.x, mx), ww = piece_weight(m, mx);
          const float ls = b == pc.b1 ? add_piece<kFar>(add_piece<kFar>(0.f, l, m, mx), om.y, om.x, mx)
                                      : add_piece<kFar>(add_piece<kFar>(0.f, om.y, om.x, mx), l, m, mx);
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
            put_columns<T, kStaged>(stg, lane, out, at, 2 * ch + hc, o, inv);
          }
        }
      } else {
      float mx = m;
      for (int c = pc.b1; c <= pc.b2; ++c)
        if (c != b) mx = fmaxf(mx, __ldcg(pc.ml(c, t)).x);
      float ls = 0.f;
      for (int c = pc.b1; c <= pc.b2; ++c) {
        const float2 ml = c == b ? make_float2(m, l) : __ldcg(pc.ml(c, t));
        ls = add_piece<kFar>(ls, ml.y, ml.x, mx);
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
        put_columns<T, kStaged>(stg, lane, out, at, ch, acc, inv);
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
      if (!wg_barrier()) return false;
      if (t == 0) {
        const unsigned before = tagged_add(ctr, add, tag, d_status, epoch);
        const bool fin = before != 0xffffffffu && before + add == (unsigned)tl.nt;
        if (fin) *ctr = 0ull;
        s_last[x] = fin;
      }
      if (!wg_barrier()) return false;
      if (s_last[x]) {
        // (the others finished in the meantime: all pieces from memory)
        __threadfence();
        float mx = neg_inf_f(), ls = 0.f;
        for (int c = pc.b1; c <= pc.b2; ++c) mx = fmaxf(mx, __ldcg(pc.ml(c, t)).x);
        for (int c = pc.b1; c <= pc.b2; ++c) {
          const float2 ml = __ldcg(pc.ml(c, t));
          ls = add_piece<kFar>(ls, ml.y, ml.x, mx);
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
          put_columns<T, kStaged>(stg, lane, out, at, ch, acc, inv);
        }
      }
    }
  }
  return true;
}

}  // namespace

}  // namespace kvs
