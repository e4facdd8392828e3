// paged_attention.cu -- attention of a ragged batch's new tokens over a paged
// KV cache: prompts, chunks of prompts and decode steps in one call.
//
// Mathematics: flash attention over a split key axis.  For a row (token,
// query head) and a set of keys, (m, l, acc) = (max s_j, sum 2^(s_j - m),
// sum 2^(s_j - m) v_j), s_j = log2(e) q.k_j / sqrt(D); sets merge by
// rescaling to the larger m, and the row's output is acc / l.
//
// Work unit: (sequence, row tile, kv head).  A row tile is TT = RT / G whole
// tokens with the G query heads of the group: RT rows share every K and V
// row.  Units follow each other on one line of "cost rows" (a fixed price,
// then one per key a unit attends); the line is cut into equal columns, one
// a block, whatever the lengths are: a block runs the 16- or 32-key tiles
// that start in its column.  A unit inside one column is written directly;
// the pieces of a unit that spans columns go to the workspace, and the block
// that completes the unit merges them in column order (the tagged counters
// of kvs_tags.cuh; no block waits for another).  Everything is derived on the device from
// the positions and offsets, so a captured graph follows them.
//
// Block: WK * WR consumer warps and a producer warp for each of WK key
// groups.  A key group has a ring of stages (a stage: K and V of one tile, swizzled 128-byte
// column blocks moved by tensor-map copies of 16 rows, each looked up in the
// page table); the WR warps of a group take 16 rows each.  Small row tiles
// (RT = 16, a decode step) run WK = 4, WR = 1 -- the keys are split over the
// warps, whose states merge in shared memory; larger ones WK = 1, WR = 7 (eight warps in all,
// so that a thread may have 255 registers).
//
// Products run on mma.sync (16 rows: an M = 128 tcgen05 tile would be seven
// eighths padding): m16n8k16 for the 16-bit types; float32 as three TF32
// products of a high and a low part (hi hi + hi lo + lo hi), 2^-21 a
// product.  A 32-key tile of a decode step costs a warp about 900 cycles for
// 16 KB where HBM delivers 23 bytes a cycle an SM, so four warps keep ahead.

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "kvs_paged.cuh"
#include "kvs_tags.cuh"
#include "kvs_tma.cuh"

namespace kvs {

namespace {

constexpr int kUnitCost = 64;         // cost rows that stand for a unit's fixed price
constexpr int kPagedMaxDevices = 64;

template <typename T, int D_, int WK_, int WR_>
struct PagedGeo {
  static constexpr int D = D_, WK = WK_, WR = WR_;
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int NW = WK * WR;         // consumer warps
  static constexpr int RT = 16 * WR;         // rows of a unit
  static constexpr int KT = F32 && D == 128 ? 16 : 32;  // keys of a tile
  static constexpr int GB = 16 * D * (int)sizeof(T);  // bytes of a 16-row copy
  static constexpr int BLK = 2048;           // one of its column blocks
  static constexpr int TILE = KT / 16 * GB;  // K (or V) of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int MERGE = WK > 1 ? NW * 16 * (D + 4) * 4 : 0;  // warp states
  static constexpr int BUDGET = 227 * 1024 - 2048 - MERGE;
  static constexpr int S0 = BUDGET / (WK * STAGE);
  static constexpr int S = S0 > 8 ? 8 : S0;  // stages of a ring
  static constexpr int OFF_MERGE = WK * S * STAGE;
  static constexpr int OFF_ML = OFF_MERGE + MERGE;        // float2 [NW][16]
  static constexpr int OFF_BAR = OFF_ML + (WK > 1 ? NW * 16 * 8 : 0);
  static constexpr int OFF_BAD = OFF_BAR + (2 * WK * S + 1) * 8;  // int [WK][S]
  static constexpr int OFF_MISC = OFF_BAD + WK * S * 4;           // abort, last, tag, pad
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr int THREADS = (NW + WK) * 32;  // a producer warp a ring
  static_assert(WK == 1 || WR == 1, "keys or rows over the warps");
  static_assert(S >= 2, "two stages at least");
  static_assert(SMEM <= 227 * 1024, "one block per SM must fit");
};

// Workspace: 256 bytes (epoch), a counter per block, then per block two
// partial slots (0: a unit begun in an earlier column, 1: one begun here and
// not finished), each RT float2 (m, l) and RT x D floats.
inline size_t paged_ws_bytes(int RT, int D) {
  return 256 + (size_t)kPagedMaxBlocks * 8 + 2 * (size_t)kPagedMaxBlocks * paged_slot_floats(RT, D) * 4;
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- fragments --------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi has TF32's 11 significant bits (truncated), lo the other 13
// of which TF32 keeps 11: 2^-21 of x is lost.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

// Key (of 8) that column n of a score fragment stands for.  16-bit types:
// n.  float32: 0 5 2 7 4 1 6 3, which makes the shared-memory reads of both
// K (8 rows by n, 4 pieces) and V (rows of columns 2q, and of 2q + 1)
// free of bank conflicts under the 128-byte swizzle.
template <bool F32>
__device__ __forceinline__ int key_of_col(int n) {
  return F32 ? ((n & 1) ? (n ^ 4) : n) : n;
}

// One warp's 16 rows: query fragments, running state, one tile at a time.
// Fragment coordinates: row r = lane / 4 (+ 8), q = lane % 4.
template <typename T, int D>
struct WarpRows {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int KT = F32 && D == 128 ? 16 : 32;
  // float32 with D = 128: q stays in L1 (its fragments would take 64 of the
  // 255 registers)
  static constexpr bool QL1 = F32 && D == 128;
  static constexpr int NQ = QL1 ? 1 : F32 ? D / 2 : D / 4;

  uint32_t qf[NQ];
  const T *qrow[2];  // QL1: this lane's two rows of q, nullptr where there is none
  float o[D / 8][4];
  float m[2], l[2];
  int lane;

  // Four columns (from 16 c + 4 q) of this lane's row half hh (float32).
  __device__ __forceinline__ float4 q_piece(int hh, int c) const {
    return qrow[hh] ? __ldca(reinterpret_cast<const float4 *>(qrow[hh] + 16 * c))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }

  // Rows 16 w .. of the unit: row x is token x / G of the tile, head x % G.
  __device__ __forceinline__ void start(const T *q, long long q_stride, int w, int rows, int G,
                                        const UnitInfo &f, int g) {
    lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      m[hh] = neg_inf_f();
      l[hh] = 0.f;
      const int x = 16 * w + lane / 4 + 8 * hh;
      const bool live = x < rows;
      const int tok = live ? x / G : 0;
      const T *src = q + (long long)(f.s.row0 + f.tok0 + tok) * q_stride +
                     (long long)(g * G + (live ? x - tok * G : 0)) * D;
      if constexpr (F32) {
        qrow[hh] = live ? src + 4 * (lane & 3) : nullptr;
        if constexpr (!QL1) {  // registers [column group of 16][row half][4]
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const float4 v = q_piece(hh, c);
            qf[(c * 2 + hh) * 4 + 0] = __float_as_uint(v.x);
            qf[(c * 2 + hh) * 4 + 1] = __float_as_uint(v.y);
            qf[(c * 2 + hh) * 4 + 2] = __float_as_uint(v.z);
            qf[(c * 2 + hh) * 4 + 3] = __float_as_uint(v.w);
          }
        }
      } else {
        // registers [k step of 16][a0 a1 a2 a3]: a0, a1 rows, a2, a3 k + 8
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
          for (int kh = 0; kh < 2; ++kh)
            qf[ks * 4 + kh * 2 + hh] =
                live ? __ldcg(reinterpret_cast<const unsigned *>(src + 16 * ks + 8 * kh + 2 * (lane & 3)))
                     : 0u;
        }
      }
    }
  }

  // One tile at (K at sk, V at sv).  lim[hh]: keys of the tile that row half
  // hh attends (>= KT: all of them).
  __device__ __forceinline__ void tile(uint32_t sk, uint32_t sv, float sl2, const int (&lim)[2]) {
    constexpr int NT = KT / 8;
    [[maybe_unused]] constexpr int kGroup = 16 * D * (int)sizeof(T);  // bytes of 16 keys
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
    if constexpr (F32) {
      float small[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) small[j][e] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {  // 16 columns: block c / 2, half c % 2
        uint32_t ah[2][4], al[2][4];      // two k steps of 8: a0: row, even; a1: row + 8; a2, a3: odd
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float4 v;
          if constexpr (QL1) {
            v = q_piece(hh, c);
          } else {
            const uint32_t *r = &qf[(c * 2 + hh) * 4];
            v = make_float4(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]),
                            __uint_as_float(r[3]));
          }
          split_tf32(v.x, ah[0][hh], al[0][hh]);
          split_tf32(v.y, ah[0][2 + hh], al[0][2 + hh]);
          split_tf32(v.z, ah[1][hh], al[1][hh]);
          split_tf32(v.w, ah[1][2 + hh], al[1][2 + hh]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          // (the small products gather apart: the tensor cores truncate each
          // sum, so a long chain of additions would lose its last bits)
          const int row = 8 * j + key_of_col<true>(lane >> 2);
          const int pc = ((lane & 3) + 4 * (c & 1)) ^ (row & 7);
          const float4 kv =
              lds_f4(sk + (j >> 1) * kGroup + (c >> 1) * 2048 + (row & 15) * 128 + pc * 16);
          uint32_t bh[4], bl[4];
          split_tf32(kv.x, bh[0], bl[0]);
          split_tf32(kv.y, bh[1], bl[1]);
          split_tf32(kv.z, bh[2], bl[2]);
          split_tf32(kv.w, bh[3], bl[3]);
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            mma_tf32(small[j], al[e2], bh[2 * e2], bh[2 * e2 + 1]);
            mma_tf32(small[j], ah[e2], bl[2 * e2], bl[2 * e2 + 1]);
            mma_tf32(s[j], ah[e2], bh[2 * e2], bh[2 * e2 + 1]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] += small[j][e];
    } else {
      const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t a[4] = {qf[ks * 4], qf[ks * 4 + 1], qf[ks * 4 + 2], qf[ks * 4 + 3]};
        const int pc = ((2 * ks + ((lane >> 3) & 1)) & 7) ^ (row & 7);
#pragma unroll
        for (int gg = 0; gg < KT / 16; ++gg) {
          uint32_t b[4];
          ldsm4(sk + gg * kGroup + (ks >> 2) * 2048 + row * 128 + pc * 16, b);
          mma16<T>(s[2 * gg], a, b[0], b[1]);
          mma16<T>(s[2 * gg + 1], a, b[2], b[3]);
        }
      }
    }
    // ---- mask, running maximum, weights ----
    if (__any_sync(0xffffffffu, min(lim[0], lim[1]) < KT)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * j + key_of_col<F32>(2 * (lane & 3) + (e & 1)) >= lim[e >> 1])
            s[j][e] = neg_inf_f();
    }
    float alpha[2], mb[2];
    bool moved = false;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float x = neg_inf_f();
#pragma unroll
      for (int j = 0; j < NT; ++j) x = fmaxf(x, fmaxf(s[j][2 * hh], s[j][2 * hh + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      const float mn = fmaxf(m[hh], x * sl2);
      mb[hh] = mn == neg_inf_f() ? 0.f : mn;  // (no key so far: every weight is 2^-inf = 0)
      alpha[hh] = ex2f(m[hh] - mb[hh]);
      moved |= mn != m[hh];
      m[hh] = mn;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = ex2f(fmaf(s[j][e], sl2, -mb[e >> 1]));
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) t += s[j][2 * hh] + s[j][2 * hh + 1];
      l[hh] = l[hh] * alpha[hh] + t;  // this lane's columns; summed over the lanes at the end
    }
    if (!F32 && __any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= alpha[e >> 1];
    }
    // ---- weights times V ----
    if constexpr (F32) {
      // a tile's products gather in registers of their own and join the
      // accumulator by one rounded addition a tile (the tensor cores truncate
      // each sum: over thousands of keys that would add up)
      uint32_t ph[NT][4], plo[NT][4];  // a0: row, key 2q; a1: row + 8; a2, a3: column 2q + 1's key
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        split_tf32(s[j][0], ph[j][0], plo[j][0]);
        split_tf32(s[j][2], ph[j][1], plo[j][1]);
        split_tf32(s[j][1], ph[j][2], plo[j][2]);
        split_tf32(s[j][3], ph[j][3], plo[j][3]);
      }
      const int n = lane >> 2;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        float t[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) t[e][k] = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r0 = 8 * j + key_of_col<true>(2 * (lane & 3));
          const int r1 = 8 * j + key_of_col<true>(2 * (lane & 3) + 1);
          const float4 v0 = lds_f4(sv + (j >> 1) * kGroup + b * 2048 + (r0 & 15) * 128 + (n ^ (r0 & 7)) * 16);
          const float4 v1 = lds_f4(sv + (j >> 1) * kGroup + b * 2048 + (r1 & 15) * 128 + (n ^ (r1 & 7)) * 16);
          const float e0[4] = {v0.x, v0.y, v0.z, v0.w}, e1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h0, l0, h1, l1;
            split_tf32(e0[e], h0, l0);
            split_tf32(e1[e], h1, l1);
            mma_tf32(t[e], plo[j], h0, h1);
            mma_tf32(t[e], ph[j], l0, l1);
            mma_tf32(t[e], ph[j], h0, h1);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[b * 4 + e][k] = fmaf(o[b * 4 + e][k], alpha[k >> 1], t[e][k]);
      }
    } else {
      const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
      for (int gg = 0; gg < KT / 16; ++gg) {
        const uint32_t a[4] = {pack2<T>(s[2 * gg][0], s[2 * gg][1]),
                               pack2<T>(s[2 * gg][2], s[2 * gg][3]),
                               pack2<T>(s[2 * gg + 1][0], s[2 * gg + 1][1]),
                               pack2<T>(s[2 * gg + 1][2], s[2 * gg + 1][3])};
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
          const int pc = ((c + (lane >> 4)) & 7) ^ (row & 7);
          uint32_t b[4];
          ldsm4t(sv + gg * kGroup + (c >> 3) * 2048 + row * 128 + pc * 16, b);
          mma16<T>(o[c], a, b[0], b[1]);
          mma16<T>(o[c + 1], a, b[2], b[3]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish() {  // row sums over the four lanes of a row
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
      l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
    }
  }

  // f(hh, d, values[4]) for the accumulator in pieces of four columns d..d+3
  // (16-bit types: two columns, values[0..1]).
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      if constexpr (F32) {
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float v[4] = {o[b * 4][2 * hh + c], o[b * 4 + 1][2 * hh + c],
                                o[b * 4 + 2][2 * hh + c], o[b * 4 + 3][2 * hh + c]};
            f(hh, 32 * b + 8 * (lane & 3) + 4 * c, v);
          }
      } else {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float v[4] = {o[j][2 * hh], o[j][2 * hh + 1], 0.f, 0.f};
          f(hh, 8 * j + 2 * (lane & 3), v);
        }
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v) {
  if constexpr (std::is_same<T, float>::value) {
    *reinterpret_cast<float4 *>(p) = v;
  } else {
    uint2 u;
    u.x = pack2<T>(v.x, v.y);
    u.y = pack2<T>(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) = u;
  }
}

// ---- the kernel ---------------------------------------------------------------
template <typename T, int D, int WK, int WR, bool kPoll>
__global__ void __launch_bounds__((WK * WR + WK) * 32, 1)
    paged_stream_kernel(const T *__restrict__ q, long long q_stride, T *__restrict__ out,
                        long long out_stride, PagedArgs pa,
                        const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int G, int Hkv, float sl2,
                        int min_column, unsigned char *ws, unsigned host_tag, int *d_status) {
  using C = PagedGeo<T, D, WK, WR>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [WK][S]
  uint64_t *empty = full + WK * C::S;
  uint64_t *cbar = empty + WK * C::S;  // all consumer warps
  int *bad = reinterpret_cast<int *>(smem + C::OFF_BAD);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
  volatile int *s_last = abort + 1;
  unsigned *epoch = reinterpret_cast<unsigned *>(ws);
  unsigned long long *counters = reinterpret_cast<unsigned long long *>(ws + 256);
  float *slots = reinterpret_cast<float *>(ws + 256 + (size_t)kPagedMaxBlocks * 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const Line ln{Hkv, C::RT / G, kUnitCost, C::KT, min_column};
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int s = 0; s < WK * C::S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], WR);
    }
    mbar_init(cbar, C::NW);
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
  const PagedPlan pl = warp_plan(pa, ln, gridDim.x, b, lane);
  if (pl.R == 0 || b >= pl.P) return;
  const long long x0 = column_start(pl.R, pl.P, b), x1 = column_start(pl.R, pl.P, b + 1);
  Unit u = pl.first;

  if (warp >= C::NW) {
    // ======================= producer of ring kw ==============================
    // (one warp for all rings issued a tile in about 1000 cycles: half the
    // rate at which HBM could fill them)
    // a decode step reads a row once; row tiles of a chunk share them through L2
    const uint64_t policy = WR == 1 ? policy_evict_first() : policy_evict_normal();
    const int ring = warp - C::NW;
    uint32_t n = 0;  // tiles put in the ring
    bool ok = true;
    constexpr int NP = C::KT / 16;  // 16-row pieces of a tile
    constexpr int AHEAD = 32 / NP;  // tiles whose pages one look-up finds
    const int piece = lane % NP;    // lanes 0..NP-1: K pieces, NP..2NP-1: V pieces
    do {
      const UnitInfo f = unit_info(pa, u, ln, x0, x1);
      const int32_t *table = pa.page_table + (size_t)u.i * pa.max_pages;
      int page = 0, k = 0;  // lane: the page of piece `piece` of the ring's tile k + lane / NP
      for (int t = f.t_lo + ring; t < f.t_hi; t += WK, ++n, ++k) {
        if (k % AHEAD == 0) {
          const int r0 = (t + WK * (lane / NP)) * C::KT + 16 * piece;
          page = r0 < f.keys ? __ldca(table + (r0 >> pa.page_shift)) : 0;
        }
        const int pg = __shfl_sync(0xffffffffu, page, (k % AHEAD) * NP + piece);
        const int npieces = min(NP, (f.keys - t * C::KT + 15) / 16);
        const bool mine = lane < 2 * NP && piece < npieces;
        const bool wrong = mine && (unsigned)pg >= (unsigned)pa.num_pages;
        const unsigned any_bad = __ballot_sync(0xffffffffu, wrong);
        const int st = ring * C::S + (int)(n % C::S);
        if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&empty[st], ((n / C::S) & 1u) ^ 1u, abort))) {
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
        mbar_wait_drain(&full[ring * C::S + j % C::S], (j / C::S) & 1u);
    }
    return;
  }

  // ========================= consumers ======================================
  const int kw = warp / WR, wr = warp % WR;
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
      const bool any_rows = 16 * wr < rows;  // (a warp past the rows only keeps the ring going)
      w.start(q, q_stride, wr, rows, G, f, u.g);
      // keys that this lane's two rows attend
      int reach[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        reach[hh] = f.s.p + f.tok0 + min(16 * wr + lane / 4 + 8 * hh, rows - 1) / G + 1;
      const int warp_reach = f.s.p + f.tok0 + min(16 * wr + 15, rows - 1) / G + 1;
      bool poison = false;
      for (int t = f.t_lo + kw; t < f.t_hi; t += WK, ++n) {
        const int st = kw * C::S + (int)(n % C::S);
        if (!__all_sync(0xffffffffu, mbar_wait<kPoll>(&full[st], (n / C::S) & 1u, abort))) {
          if (lane == 0) give_up(abort, d_status, epoch);
          return;
        }
        poison |= bad[st] != 0;
        unsigned char *sk = smem + st * C::STAGE;
        const int left = f.keys - t * C::KT;  // keys of the tile that exist
        if (left < C::KT) {
          // rows past the last key hold anything: V's become zero (their
          // weights are zero, but 0 x NaN is not)
          if (wr == 0) {
            for (int e = lane; e < (C::KT - left) * (D * (int)sizeof(T) / 16); e += 32) {
              const int row = left + e % (C::KT - left), pc = e / (C::KT - left);
              *reinterpret_cast<uint4 *>(sk + C::TILE + (row >> 4) * C::GB + (pc >> 3) * C::BLK +
                                         (row & 15) * 128 + (pc & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_shared();
          }
          if (WR > 1) {  // (the last tile of a unit: all WR warps meet here)
            if (!consumers_barrier()) return;
          } else {
            __syncwarp();
          }
        }
        if (any_rows && t * C::KT < warp_reach) {
          const int lim[2] = {reach[0] - t * C::KT, reach[1] - t * C::KT};
          w.tile(smem_addr(sk), smem_addr(sk + C::TILE), sl2, lim);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
      w.finish();
      if (poison) w.l[0] = w.l[1] = nan;
      const bool whole = f.t_hi - f.t_lo == f.nt;
      const int slot = 2 * b + (f.t_lo == 0 ? 1 : 0);
      float *sl = slots + slot * paged_slot_floats(C::RT, D);
      float *sacc = sl + 2 * C::RT;
      T *orow = out + (long long)(f.s.row0 + f.tok0) * out_stride + (long long)u.g * G * D;
      if constexpr (WK > 1) {
        // the key groups' states merge in shared memory
        float *macc = reinterpret_cast<float *>(smem + C::OFF_MERGE);  // [NW][16][D + 4]
        float2 *mml = reinterpret_cast<float2 *>(smem + C::OFF_ML);    // [NW][16]
        float *mine = macc + warp * 16 * (D + 4);
        w.each([&](int hh, int d, const float(&v)[4]) {
          float *p = mine + (lane / 4 + 8 * hh) * (D + 4) + d;
          if constexpr (C::F32)
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
          else
            *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
        });
        if ((lane & 3) == 0) {
          mml[warp * 16 + lane / 4] = make_float2(w.m[0], w.l[0]);
          mml[warp * 16 + lane / 4 + 8] = make_float2(w.m[1], w.l[1]);
        }
        if (!consumers_barrier()) return;
        for (int e = threadIdx.x; e < rows * (D / 4); e += C::NW * 32) {
          const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
          float mx = neg_inf_f();
#pragma unroll
          for (int k = 0; k < WK; ++k) mx = fmaxf(mx, mml[k * 16 + r].x);
          const float mz = mx == neg_inf_f() ? 0.f : mx;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float ls = 0.f;
#pragma unroll
          for (int k = 0; k < WK; ++k) {
            const float2 ml = mml[k * 16 + r];
            const float wgt = ex2f(ml.x - mz);
            const float4 v = *reinterpret_cast<const float4 *>(macc + (k * 16 + r) * (D + 4) + d);
            acc.x = fmaf(wgt, v.x, acc.x);
            acc.y = fmaf(wgt, v.y, acc.y);
            acc.z = fmaf(wgt, v.z, acc.z);
            acc.w = fmaf(wgt, v.w, acc.w);
            // (a NaN sum stays one also under a zero weight)
            ls = fmaf(wgt, ml.y, ls);
          }
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
      } else if (any_rows) {
        const float inv[2] = {1.f / w.l[0], 1.f / w.l[1]};
        w.each([&](int hh, int d, const float(&v)[4]) {
          const int r = 16 * wr + lane / 4 + 8 * hh;
          if (r >= rows) return;
          if (whole) {
            const int tok = r / G;
            T *p = orow + (long long)tok * out_stride + (r - tok * G) * D + d;
            if constexpr (C::F32)
              *reinterpret_cast<float4 *>(p) =
                  make_float4(v[0] * inv[hh], v[1] * inv[hh], v[2] * inv[hh], v[3] * inv[hh]);
            else
              *reinterpret_cast<uint32_t *>(p) = pack2<T>(v[0] * inv[hh], v[1] * inv[hh]);
          } else {
            float *p = sacc + (size_t)r * D + d;
            if constexpr (C::F32)
              __stcg(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
            else
              __stcg(reinterpret_cast<float2 *>(p), make_float2(v[0], v[1]));
          }
        });
        if (!whole && (lane & 3) == 0) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int r = 16 * wr + lane / 4 + 8 * hh;
            if (r < rows) __stcg(reinterpret_cast<float2 *>(sl) + r, make_float2(w.m[hh], w.l[hh]));
          }
        }
      }
      if (!whole) __threadfence();  // the partial is visible GPU-wide before it counts
      if (WK > 1 || !whole) {
        if (!consumers_barrier()) return;  // (also: the merge buffers may be written again)
      }
      if (!whole) {
        // the blocks of the unit's first and last tile; every block between has some
        const int b1 = column_at(f.k0, pl.R, pl.P);
        const int b2 = column_at(f.k0 + (long long)(f.nt - 1) * C::KT, pl.R, pl.P);
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
          for (int e = threadIdx.x; e < rows * (D / 4); e += C::NW * 32) {
            const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
            float4 acc;
            float ls;
            merge_pieces(slots, paged_slot_floats(C::RT, D), 2 * C::RT + r * D + d, r, b1, b2, acc, ls);
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

template <typename T, int D, int WK, int WR>
int launch_stream(const void *q, long long q_stride, const kvs_paged_cache &cache,
                  const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                  int *d_status, cudaStream_t stream) {
  using C = PagedGeo<T, D, WK, WR>;
  static bool configured[kPagedMaxDevices] = {false};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kPagedMaxDevices)
    return KVS_ERR_LAUNCH;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      for (auto kern : {paged_stream_kernel<T, D, WK, WR, false>,
                        paged_stream_kernel<T, D, WK, WR, true>}) {
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
  const int min_column = WK * C::KT + kUnitCost;
  const cudaError_t e = launch_pdl(
      poll_waits() ? paged_stream_kernel<T, D, WK, WR, true>
                   : paged_stream_kernel<T, D, WK, WR, false>,
      dim3(grid), dim3(C::THREADS), C::SMEM, stream, static_cast<const T *>(q), q_stride,
      static_cast<T *>(out), out_stride, pa, kmap, vmap, H / Hkv, Hkv, sl2, min_column,
      static_cast<unsigned char *>(workspace), fresh_tag(), d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

template <typename T, int D>
int dispatch_rows(const void *q, long long q_stride, const kvs_paged_cache &cache,
                  const PagedArgs &pa, void *out, long long out_stride, int H, void *workspace,
                  int *d_status, cudaStream_t stream) {
  if ((long long)pa.max_new * (H / cache.num_kv_heads) <= 16)
    return launch_stream<T, D, 4, 1>(q, q_stride, cache, pa, out, out_stride, H, workspace,
                                     d_status, stream);
  if constexpr (std::is_same<T, float>::value)
    return launch_stream<T, D, 1, 7>(q, q_stride, cache, pa, out, out_stride, H, workspace,
                                     d_status, stream);
  else
    return launch_paged_chunk(q, q_stride, cache, pa, out, out_stride, H, workspace, d_status,
                              stream);
}

}  // namespace

int set_wait_limit_paged(uint64_t ns) {
  if (set_unit_wait_limit(ns) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_LAUNCH;
  }
  return KVS_OK;
}

size_t paged_attention_workspace_bytes(int H, int Hkv, int D, int max_new) {
  if ((long long)max_new * (H / Hkv) <= 16) return paged_ws_bytes(16, D);
  return std::max(paged_ws_bytes(128, D), paged_chunk_workspace_bytes(D));
}

int launch_paged_attention(const void *q, long long q_stride, const kvs_paged_cache &cache,
                           const PagedArgs &pa, void *out, long long out_stride, int H,
                           void *workspace, int *d_status, cudaStream_t stream) {
#define KVS_PAGED(T)                                                                             \
  return cache.head_dim == 64                                                                    \
             ? dispatch_rows<T, 64>(q, q_stride, cache, pa, out, out_stride, H, workspace,       \
                                    d_status, stream)                                            \
             : dispatch_rows<T, 128>(q, q_stride, cache, pa, out, out_stride, H, workspace,      \
                                     d_status, stream)
  if (cache.dtype == KVS_F32) KVS_PAGED(float);
  if (cache.dtype == KVS_F16) KVS_PAGED(__half);
  KVS_PAGED(__nv_bfloat16);
#undef KVS_PAGED
}

}  // namespace kvs
