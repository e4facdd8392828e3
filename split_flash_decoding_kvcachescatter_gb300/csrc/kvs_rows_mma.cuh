// kvs_rows_mma.cuh -- one warp's share of paged attention on mma.sync: 16
// rows (token, query head) against tiles of keys in shared memory, with the
// running softmax state in registers.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <type_traits>

#include "kvs_paged.cuh"

namespace kvs {

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
// x = hi + lo: hi is x rounded to TF32's 11 significant bits, lo the rest, 2^-11
// of x at most; of its 12 bits TF32 keeps 11, so 2^-23 of x is lost.  (hi
// truncated, one addition less a value, loses 2^-21, always toward zero:
// attention over 600 keys was then off by 1.1e-6, now by 6e-7.  Rounding takes
// the last 2^-12 below the largest float to infinity.)
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
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

// (a, b) = hi + lo in 16 bits each: hi is rounded, lo what it leaves, rounded.
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack2<T>(a, b);
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    lo = pack2<T>(a - f.x, b - f.y);
  } else {
    lo = pack2<T>(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
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
// The state's m is the reference of its weights 2^(s - m): the running maximum
// less kLift, so that float16 weights reach 2^10 and lose what is below 2^-35 of
// the largest one (with a lift of 0 they lost what is below 2^-25: 131,072 keys
// of 2^-26 each are 2^-9 of the sum).  All of a row's sums carry the factor, so
// nothing else knows of it.  (2^6 of room are left for m's own rounding, which
// is 2^5 where scores reach 2^26.)
// Fragment coordinates: row r = lane / 4 (+ 8), q = lane % 4.
template <typename T, int D>
struct WarpRows {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int KT = F32 && D == 128 ? 16 : 32;
  // float32 with D = 128: q stays in L1 (its fragments would take 64 of the
  // 255 registers)
  static constexpr bool QL1 = F32 && D == 128;
  static constexpr float kLift = std::is_same<T, __half>::value ? 10.f : 0.f;
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
  // hh attends (>= KT: all of them).  kFew (16-bit types): the unit has 8 rows
  // at most, and those behind them carry the second parts of their weights.
  template <bool kFew = false>
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
      const float mn = fmaxf(m[hh], x * sl2 - kLift);
      mb[hh] = mn == neg_inf_f() ? 0.f : mn;  // (no key so far: every weight is 2^-inf = 0)
      alpha[hh] = ex2f(m[hh] - mb[hh]);
      moved |= mn != m[hh];
      m[hh] = mn;
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      if (kFew && hh == 1) break;
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        s[j][2 * hh] = ex2f(fmaf(s[j][2 * hh], sl2, -mb[hh]));
        s[j][2 * hh + 1] = ex2f(fmaf(s[j][2 * hh + 1], sl2, -mb[hh]));
        t += s[j][2 * hh] + s[j][2 * hh + 1];
      }
      l[hh] = l[hh] * alpha[hh] + t;  // this lane's columns; summed over the lanes at the end
    }
    if (!F32 && __any_sync(0xffffffffu, moved)) {
      if (kFew) alpha[1] = alpha[0];
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
      // Each weight in two 16-bit parts, so that what one rounding would lose
      // (a third of the outputs then differed in their last bit) stays.  Units of
      // 8 rows at most, which is every single token: row r's second part stands
      // where row r + 8 would, and costs no product; finish() adds the two sums.
      // More rows: a second product (it took 2 to 6 % of a step's time; the form
      // for few rows takes none).
      const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
      for (int gg = 0; gg < KT / 16; ++gg) {
        uint32_t a[4], al[4];
        if constexpr (kFew) {
          split2<T>(s[2 * gg][0], s[2 * gg][1], a[0], a[1]);
          split2<T>(s[2 * gg + 1][0], s[2 * gg + 1][1], a[2], a[3]);
        } else {
          split2<T>(s[2 * gg][0], s[2 * gg][1], a[0], al[0]);
          split2<T>(s[2 * gg][2], s[2 * gg][3], a[1], al[1]);
          split2<T>(s[2 * gg + 1][0], s[2 * gg + 1][1], a[2], al[2]);
          split2<T>(s[2 * gg + 1][2], s[2 * gg + 1][3], a[3], al[3]);
        }
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
          const int pc = ((c + (lane >> 4)) & 7) ^ (row & 7);
          uint32_t b[4];
          ldsm4t(sv + gg * kGroup + (c >> 3) * 2048 + row * 128 + pc * 16, b);
          if constexpr (!kFew) {
            mma16<T>(o[c], al, b[0], b[1]);
            mma16<T>(o[c + 1], al, b[2], b[3]);
          }
          mma16<T>(o[c], a, b[0], b[1]);
          mma16<T>(o[c + 1], a, b[2], b[3]);
        }
      }
    }
  }

  template <bool kFew = false>
  __device__ __forceinline__ void finish() {  // row sums over the four lanes of a row
    if constexpr (kFew) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] += o[j][2];
        o[j][1] += o[j][3];
      }
    }
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

}  // namespace kvs
