// kvs_rows_q8.cuh -- one warp's share of attention over an 8-bit paged cache on
// mma.sync: 16 rows (token, query head) against tiles of keys in shared memory,
// with the running softmax state in registers (kvs_rows_mma.cuh for plain pages).
//
// Mathematics.  Key j stands for sk_b e_j and value j for sv_b f_j, with the stored
// numbers e_j, f_j and the scales of j's block b of 16.  Stored numbers are exact in
// float16, so all products run in float16 whatever q's type:
//   score  x_j = (log2(e) / sqrt D) sk_b (q . e_j).  A row of q is brought to at most
//          2^15 by a power of two, which goes into the row's factor; float16 then
//          holds 16-bit rows exactly down to 2^-28 of the row's largest element, and
//          float32 rows as a high and a low part (22 bits).
//   output (sum 2^x_j sv_b f_j) / (sum 2^x_j).  The running reference m is the
//          maximum of x_j + log2 sv_b, and w_j = 2^(x_j + log2 sv_b - m) is the weight
//          of f_j, at most 2^kLift, however the scales differ; the sum l takes
//          w_j / sv_b.  Weights go into the product as a high and a low float16 part.
// Scales of V reach up to 2^100, so a w_j could be below float32's range although w_j / sv_b
// counts in the sum, and m may move by more than that range:
//  - scales under 2^-60 of the largest so far count as that much: what they stand for is
//    nothing beside it.  A w_j below 2^-126 is then less than 2^-76 of the sum: with sv* the
//    scale of the key that made m, l >= 2^kLift / sv*, and w_j / sv_b < 2^-126 2^60 / sv*.
//  - the sum is multiplied by 2^(m - m') in two steps of half the exponent: l is 2^-90 at
//    least, a step 2^-86.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <type_traits>

#include "kvs_fp8.cuh"
#include "kvs_paged.cuh"
#include "kvs_rows_mma.cuh"

namespace kvs {

__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// The least that scales of V count as: 2^-60, so that 1 / scale stays in range, and 2^-60 of
// the largest so far.
constexpr float kLeastScale = 8.673617379884035e-19f;
__device__ __forceinline__ float least_scale(float largest) { return kLeastScale * fmaxf(largest, 1.f); }

// log2 of a scale of V (2^-60 at least), and its reciprocal.
__device__ __forceinline__ void value_scale(float sv, float &lg, float &inv) {
  const unsigned u = __float_as_uint(sv);
  const float mant = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
  lg = (float)((int)(u >> 23) - 127) + (mant == 1.f ? 0.f : __log2f(mant));
  inv = mant == 1.f ? __uint_as_float((254u << 23) - u) : 1.f / sv;
}

// The scales of a cache.
struct ScalesQ8 {
  const float *k_scales, *v_scales;
};

// Pages, and tiles of KT rows, as lines of 128 bytes.
template <int D, int KT>
struct LinesQ8 {
  // the line of 128 bytes that row `row` of the pages begins in
  static __device__ __forceinline__ int map_row(int row) { return D == 128 ? row : row >> 1; }
  // Rows `left` and up of a tile become zero (by one warp).
  static __device__ __forceinline__ void clear_rows(unsigned char *tile, int left) {
    constexpr int PC = D / 16;  // 16-byte pieces of a row
    for (int e = threadIdx.x & 31; e < (KT - left) * PC; e += 32) {
      const int row = left + e / PC, line = D == 128 ? row : row >> 1;
      const int pc = ((D == 128 ? 0 : (row & 1) * 4) + e % PC) ^ (line & 7);
      *reinterpret_cast<uint4 *>(tile + line * 128 + pc * 16) = make_uint4(0, 0, 0, 0);
    }
  }
};

// The tile in shared memory: rows of D bytes in lines of 128, 16-byte pieces
// swizzled by the line (piece c of line r at c ^ (r % 8)).
// Which elements a lane reads is free as long as both operands agree on it, and
// chosen so that it reads 16 bytes at a time without bank conflicts: of a key, lane
// (n, q) takes the D / 4 elements from D / 4 q (k step s: four of them, from 4 s), of
// a value those from D / 8 n (column n of product c: element D / 8 n + c).
// kFewForm: units of 8 rows at most have a form of their own (tile<true>).
template <typename T, int D, bool kFewForm = true>
struct RowsQ8 {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int KT = D == 128 ? 32 : 64;
  static constexpr int kEach = 4;
  static constexpr float kLift = 10.f;  // as WarpRows' in float16
  static constexpr int KS = D / 16;     // k steps of a score
  static constexpr int NB = KT / 16;    // blocks of a tile

  // Registers a0 a1 a2 a3 of each k step: a0, a2 row r, a1, a3 row r + 8.  Units of 8
  // rows at most have row r's low parts in a1, a3 (zero in 16 bits), others in ql.
  uint32_t qf[KS][4];
  uint32_t ql[F32 ? KS : 1][4];
  float fac[2];  // of the rows' scores
  float o[D / 8][4];
  float m[2], l[2];
  float svmax;  // the largest scale of V so far
  int lane;

  __device__ __forceinline__ void start(const T *q, long long q_stride, int w, int rows, int G,
                                        const UnitInfo &f, int g) {
    lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    const bool few = kFewForm && rows <= 8;
    svmax = 0.f;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      m[hh] = neg_inf_f();
      l[hh] = 0.f;
      const int x = 16 * w + lane / 4 + 8 * hh;
      const bool live = x < rows;
      const int tok = live ? x / G : 0;
      const T *src = q + (long long)(f.s.row0 + f.tok0 + tok) * q_stride +
                     (long long)(g * G + (live ? x - tok * G : 0)) * D + (D / 4) * (lane & 3);
      float v[KS][4];
      float most = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        Vec<T, 4> r{};
        if (live) r = vec_load<T, 4>(src + 4 * s);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[s][e] = live ? to_f32(r.e[e]) : 0.f;
          most = fmaxf(most, fabsf(v[s][e]));
        }
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int ex = max((int)(__float_as_uint(most) >> 23) - 127, -100);  // most < 2^(ex + 1)
      const float up = __uint_as_float((unsigned)(14 - ex + 127) << 23);
      fac[hh] = __uint_as_float((unsigned)(ex - 14 + 127) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint32_t h0, l0, h1, l1;
        split2<__half>(v[s][0] * up, v[s][1] * up, h0, l0);
        split2<__half>(v[s][2] * up, v[s][3] * up, h1, l1);
        if (hh == 0 || !few) {
          qf[s][hh] = h0;
          qf[s][2 + hh] = h1;
        }
        if (few && hh == 0) {
          qf[s][1] = F32 ? l0 : 0u;
          qf[s][3] = F32 ? l1 : 0u;
        }
        if (F32) {
          ql[F32 ? s : 0][hh] = l0;
          ql[F32 ? s : 0][2 + hh] = l1;
        }
      }
    }
  }

  // One tile: K at sk, V at sv, the blocks' scales (K's, then V's); sl2 and lim as
  // for WarpRows.  kFew: the unit has 8 rows at most.
  template <bool kFew = false>
  __device__ __forceinline__ void tile(uint32_t sk, uint32_t sv, const float *scales, float sl2,
                                       const int (&lim)[2]) {
    constexpr int NT = KT / 8;
    const int n = lane >> 2, q = lane & 3;
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
      uint32_t w[D / 16];
      if constexpr (D == 128) {
        const uint32_t at = sk + (8 * j + n) * 128;
        const uint4 a = lds_u4(at + ((2 * q) ^ n) * 16), b = lds_u4(at + ((2 * q + 1) ^ n) * 16);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      } else {
        const int line = 4 * j + (n >> 1);
        const uint4 a = lds_u4(sk + line * 128 + ((((n & 1) * 4) + q) ^ (line & 7)) * 16);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      }
      if constexpr (F32 && !kFew) {  // the small products first
#pragma unroll
        for (int k = 0; k < KS; ++k) mma16<__half>(s[j], ql[k], from_e4m3x2(w[k]), from_e4m3x2(w[k] >> 16));
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) mma16<__half>(s[j], qf[k], from_e4m3x2(w[k]), from_e4m3x2(w[k] >> 16));
      if constexpr (F32 && kFew) {
        s[j][0] += s[j][2];
        s[j][1] += s[j][3];
      }
    }
    // ---- scales, mask, running reference, weights ----
    constexpr int HH = kFew ? 1 : 2;
    float lg[NB], inv[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) svmax = fmaxf(svmax, scales[NB + b]);
    const float least = least_scale(svmax);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float ks = scales[b] * sl2;
      value_scale(fmaxf(scales[NB + b], least), lg[b], inv[b]);
#pragma unroll
      for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
        for (int e = 0; e < 2 * HH; ++e) s[j][e] *= fac[e >> 1] * ks;
    }
    if (__any_sync(0xffffffffu, min(lim[0], lim[1]) < KT)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2 * HH; ++e)
          if (8 * j + 2 * q + (e & 1) >= lim[e >> 1]) s[j][e] = neg_inf_f();
    }
    float alpha[2] = {1.f, 1.f};
    bool moved = false;
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
      float x = neg_inf_f();
#pragma unroll
      for (int b = 0; b < NB; ++b)
        x = fmaxf(x, fmaxf(fmaxf(s[2 * b][2 * hh], s[2 * b][2 * hh + 1]),
                           fmaxf(s[2 * b + 1][2 * hh], s[2 * b + 1][2 * hh + 1])) + lg[b]);
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      const float mn = fmaxf(m[hh], x - kLift);
      const float mb = mn == neg_inf_f() ? 0.f : mn;  // (no key so far: every weight is 2^-inf = 0)
      const float ah = ex2f(0.5f * (m[hh] - mb));
      alpha[hh] = ah * ah;
      moved |= mn != m[hh];
      m[hh] = mn;
      l[hh] = l[hh] * ah * ah;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float up = lg[b] - mb;
        float t = 0.f;
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j) {
          s[j][2 * hh] = ex2f(s[j][2 * hh] + up);
          s[j][2 * hh + 1] = ex2f(s[j][2 * hh + 1] + up);
          t += s[j][2 * hh] + s[j][2 * hh + 1];
        }
        l[hh] = fmaf(t, inv[b], l[hh]);  // this lane's columns; summed over the lanes at the end
      }
    }
    if (kFew) alpha[1] = alpha[0];
    if (!F32 && __any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= alpha[e >> 1];
    }
    // ---- weights times V (the two parts of a weight: see WarpRows) ----
    uint32_t a[NB][4];
    uint32_t al[kFew ? 1 : NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (kFew) {
        split2<__half>(s[2 * b][0], s[2 * b][1], a[b][0], a[b][1]);
        split2<__half>(s[2 * b + 1][0], s[2 * b + 1][1], a[b][2], a[b][3]);
      } else {
        split2<__half>(s[2 * b][0], s[2 * b][1], a[b][0], al[b][0]);
        split2<__half>(s[2 * b][2], s[2 * b][3], a[b][1], al[b][1]);
        split2<__half>(s[2 * b + 1][0], s[2 * b + 1][1], a[b][2], al[b][2]);
        split2<__half>(s[2 * b + 1][2], s[2 * b + 1][3], a[b][3], al[b][3]);
      }
    }
    // Words of four columns (element D / 8 n + 4 w of a key), WN at a time.  float32: a
    // tile's products gather in registers of their own and join the accumulator by one
    // rounded addition (the tensor cores truncate each sum: over thousands of keys that
    // would add up), for which only some of the columns find room at once.
    constexpr int WN = D == 128 && !F32 ? 4 : 2;
#pragma unroll
    for (int w0 = 0; w0 < D / 32; w0 += WN) {
      float t[F32 ? 4 * WN : 1][4];
      if constexpr (F32) {
#pragma unroll
        for (int c = 0; c < 4 * WN; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) t[c][e] = 0.f;
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t v[4][WN];  // of keys 2q, 2q + 1, 2q + 8, 2q + 9
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 16 * b + 2 * q + (k & 1) + 8 * (k >> 1);
          if constexpr (D == 128) {
            const uint32_t at = sv + key * 128 + (n ^ (key & 7)) * 16;
            if constexpr (WN == 4) {
              const uint4 x = lds_u4(at);
              v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
            } else {
              const uint2 x = lds_u2(at + 4 * w0);
              v[k][0] = x.x, v[k][1] = x.y;
            }
          } else {
            const int line = key >> 1;
            const uint2 x = lds_u2(sv + line * 128 + ((((key & 1) * 4) + (n >> 1)) ^ (line & 7)) * 16 +
                                   (n & 1) * 8);
            v[k][0] = x.x, v[k][1] = x.y;
          }
        }
#pragma unroll
        for (int w = 0; w < WN; ++w) {
          // bytes of a pair of keys side by side: (column 0, 1), (column 2, 3)
          const uint32_t lo0 = __byte_perm(v[0][w], v[1][w], 0x5140), lo1 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t hi0 = __byte_perm(v[2][w], v[3][w], 0x5140), hi1 = __byte_perm(v[2][w], v[3][w], 0x7362);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t b0 = from_e4m3x2((c & 2 ? lo1 : lo0) >> (16 * (c & 1)));
            const uint32_t b1 = from_e4m3x2((c & 2 ? hi1 : hi0) >> (16 * (c & 1)));
            float(&acc)[4] = F32 ? t[F32 ? 4 * w + c : 0] : o[4 * (w0 + w) + c];
            if constexpr (!kFew) mma16<__half>(acc, al[kFew ? 0 : b], b0, b1);
            mma16<__half>(acc, a[b], b0, b1);
          }
        }
      }
      if constexpr (F32) {
#pragma unroll
        for (int c = 0; c < 4 * WN; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[4 * w0 + c][e] = fmaf(o[4 * w0 + c][e], alpha[e >> 1], t[F32 ? c : 0][e]);
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

  // f(hh, d, values[4]) for the accumulator in pieces of four columns d .. d + 3.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < D / 8; c += 4) {
          const float v[4] = {o[c][2 * hh + e], o[c + 1][2 * hh + e], o[c + 2][2 * hh + e],
                              o[c + 3][2 * hh + e]};
          f(hh, (D / 8) * (2 * (lane & 3) + e) + c, v);
        }
  }
};

}  // namespace kvs
