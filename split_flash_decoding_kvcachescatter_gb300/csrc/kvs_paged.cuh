// kvs_paged.cuh -- the device view of a ragged batch over a paged cache, and
// the element types of the paged-cache and logit kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvs_device.cuh"
#include "kvs_launch.h"
#include "kvsdecode.h"

namespace kvs {

// One sequence of the batch: first position, new tokens and first row of q
// and out; n = 0 when there is nothing to do, err when the sequence is bad
// (n and row0 are then the rows to mark, 0 rows if the offsets are bad).
struct PagedSeq {
  int p, n, row0, err;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs &b, int i) {
  const int a = __ldca(b.row_offsets + i), e = __ldca(b.row_offsets + i + 1);
  const int p = __ldca(b.positions + i);
  PagedSeq s{p, 0, a, KVS_OK};
  if (a < 0 || e < a || e > b.num_rows || e - a > b.max_new) {
    s.err = KVS_ERR_ROWS;
    return s;
  }
  s.n = e - a;
  if (s.n > 0 && (p < 0 || (long long)p + s.n > (long long)b.max_pages << b.page_shift))
    s.err = KVS_ERR_POSITION;
  return s;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N elements of T moved by one load or store (N * sizeof(T) = 2, 4, 8 or 16
// bytes, aligned to that).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T e[N];
};

// Coherent at L2: with programmatic dependent launch the data may have been
// written by the preceding kernel.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> vec_load(const T *p) {
  Vec<T, N> v;
  if constexpr (sizeof(v) == 16) {
    *reinterpret_cast<uint4 *>(&v) = __ldcg(reinterpret_cast<const uint4 *>(p));
  } else if constexpr (sizeof(v) == 8) {
    *reinterpret_cast<uint2 *>(&v) = __ldcg(reinterpret_cast<const uint2 *>(p));
  } else if constexpr (sizeof(v) == 4) {
    *reinterpret_cast<unsigned *>(&v) = __ldcg(reinterpret_cast<const unsigned *>(p));
  } else {
    *reinterpret_cast<unsigned short *>(&v) = __ldcg(reinterpret_cast<const unsigned short *>(p));
  }
  return v;
}

template <typename T, int N>
__device__ __forceinline__ void vec_store(T *p, const Vec<T, N> &v) {
  if constexpr (sizeof(v) == 16) {
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&v);
  } else if constexpr (sizeof(v) == 8) {
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(&v);
  } else if constexpr (sizeof(v) == 4) {
    *reinterpret_cast<unsigned *>(p) = *reinterpret_cast<const unsigned *>(&v);
  } else {
    *reinterpret_cast<unsigned short *>(p) = *reinterpret_cast<const unsigned short *>(&v);
  }
}

// ---- the line of cost rows ------------------------------------------------
// What fixes the line: kv heads, tokens of a row tile, fixed price of a unit,
// keys of a tile, the shortest column worth a block.
struct Line {
  int Hkv, TT, fix, KT, min_column;
};

// Sequence with n tokens from position p, TT tokens a row tile: Rn row tiles;
// unit (rt, g) attends p + min(n, (rt + 1) TT) keys.
struct SeqCost {
  int p, n, Rn, TT, fix;
  __device__ SeqCost(const PagedSeq &s, const Line &ln)
      : p(s.p), n(s.err == KVS_OK ? s.n : 0), Rn(0), TT(ln.TT), fix(ln.fix) {
    Rn = (n + TT - 1) / TT;
  }
  __device__ int keys(int rt) const { return p + min(n, (rt + 1) * TT); }
  // cost rows of one kv head's units before row tile rt (rt < Rn)
  __device__ long long before(int rt) const {
    return (long long)rt * (p + fix) + (long long)TT * ((long long)rt * (rt + 1) / 2);
  }
  __device__ long long head_total() const {
    return n > 0 ? before(Rn - 1) + p + n + fix : 0;
  }
};

// A unit of the line: sequence i, row tile rt, kv head g, first cost row base.
struct Unit {
  int i, rt, g;
  long long base;
};

// a / b for a >= 0, b > 0: a 32-bit division when both fit (the 64-bit one
// is a long instruction sequence, on the path to a block's first copy).
__device__ __forceinline__ long long div_nn(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}

// A line of R cost rows cut into NS equal ranges.
struct Cuts {
  long long R;
  int NS;
  __device__ long long start(int r) const { return div_nn(R * r, NS); }
  // The range that holds cost row x: the last one that starts at or before it.
  __device__ int at(long long x) const {
    const long long c = div_nn(x * NS + NS - 1, R);
    return (int)(c < NS - 1 ? c : NS - 1);
  }
};

// The cost rows of the whole line (warp-cooperative; every lane returns it).
static __device__ long long warp_line_total(const PagedArgs &a, const Line &ln, int lane) {
  long long sum = 0;
  for (int i = lane; i < a.M; i += 32) sum += SeqCost(paged_seq(a, i), ln).head_total();
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * ln.Hkv;
}

// The line in at most `blocks` equal ranges, fewer when short, so that one
// holds work worth a block.
__device__ __forceinline__ Cuts equal_cuts(long long R, const Line &ln, int blocks) {
  Cuts c{R, 1};
  if (R > 0) c.NS = (int)max(1ll, min((long long)blocks, div_nn(R, ln.min_column)));
  return c;
}

// The unit that holds cost row x of the line, x < R (warp-cooperative; every
// lane returns it).
static __device__ Unit warp_unit_at(const PagedArgs &a, const Line &ln, long long x, int lane) {
  Unit u{a.M, 0, 0, 0};
  long long base = 0;
  for (int i0 = 0; i0 < a.M; i0 += 32) {
    const int i = i0 + lane;
    long long mine = 0;
    if (i < a.M) mine = SeqCost(paged_seq(a, i), ln).head_total() * ln.Hkv;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const bool hit = mine > 0 && x >= base + inc - mine && x < base + inc;
    const unsigned ballot = __ballot_sync(0xffffffffu, hit);
    if (ballot) {
      const int src = __ffs(ballot) - 1;
      const long long sb = __shfl_sync(0xffffffffu, base + inc - mine, src);
      u.i = i0 + src;
      const SeqCost c(paged_seq(a, u.i), ln);
      const long long off = x - sb;
      int lo = 0, hi = c.Rn - 1;  // the last row tile that starts at or before off
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c.before(mid) * ln.Hkv <= off) lo = mid;
        else hi = mid - 1;
      }
      const long long tile_base = c.before(lo) * ln.Hkv;
      const long long span = c.keys(lo) + ln.fix;
      u.rt = lo;
      u.g = (int)div_nn(off - tile_base, span);
      u.base = sb + tile_base + u.g * span;
      return u;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return u;
}

// Everything a warp needs to know about a unit.
struct UnitInfo {
  PagedSeq s;
  int keys, nt;     // keys it attends, its tiles
  int t_lo, t_hi;   // tiles of this block
  int tok0, ntok;   // tokens of the row tile (within the sequence)
  long long k0;     // cost row where tile 0 starts
};

// Of nt tiles of KT keys, the first one at cost row k0: how many start before x.
__device__ __forceinline__ int tiles_before(long long x, long long k0, int nt, int KT) {
  const long long d = x - k0;
  return d <= 0 ? 0 : (int)min((long long)nt, (d + KT - 1) / KT);
}

__device__ __forceinline__ UnitInfo unit_info(const PagedArgs &a, const Unit &u, const Line &ln,
                                              long long x0, long long x1) {
  UnitInfo f;
  f.s = paged_seq(a, u.i);
  const SeqCost c(f.s, ln);
  f.keys = c.keys(u.rt);
  f.nt = (f.keys + ln.KT - 1) / ln.KT;
  f.tok0 = u.rt * ln.TT;
  f.ntok = min(ln.TT, c.n - f.tok0);
  f.k0 = u.base + ln.fix;
  f.t_lo = tiles_before(x0, f.k0, f.nt, ln.KT);
  f.t_hi = tiles_before(x1, f.k0, f.nt, ln.KT);
  return f;
}

// The unit after u; false past the last sequence.
__device__ __forceinline__ bool next_unit(const PagedArgs &a, Unit &u, const UnitInfo &f,
                                          const Line &ln) {
  u.base += f.keys + ln.fix;
  if (++u.g < ln.Hkv) return true;
  u.g = 0;
  if ((++u.rt) * ln.TT < f.s.n) return true;
  u.rt = 0;
  for (++u.i; u.i < a.M; ++u.i) {
    const PagedSeq s = paged_seq(a, u.i);
    if (s.err == KVS_OK && s.n > 0) return true;
  }
  return false;
}

// Four accumulator columns of one row, merged over a unit's pieces in column
// order: range b1's piece began the unit (its slot 2 b1 + 1), those of ranges
// b1 + 1 .. b2 continue it (slots 2 b).  A slot of `stride` floats has the
// row's (m, l) at float2 `r` and its accumulators at float `at`.  Pieces are
// taken eight at a time, all loads of a batch before the first is used, so a
// batch costs one L2 round trip.
static __device__ __forceinline__ void merge_pieces(const float *slots, size_t stride, int at,
                                                    int r, int b1, int b2, float4 &acc, float &l) {
  constexpr int kBatch = 8;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
  float m = neg_inf_f();
  for (int c = b1; c <= b2; c += kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (c + j <= b2) {
        const float *ps = slots + (2 * (size_t)(c + j) + (c + j == b1 ? 1 : 0)) * stride;
        ml[j] = __ldcg(reinterpret_cast<const float2 *>(ps) + r);
        v[j] = __ldcg(reinterpret_cast<const float4 *>(ps + at));
      }
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (c + j <= b2) mn = fmaxf(mn, ml[j].x);
    const float mz = mn == neg_inf_f() ? 0.f : mn;
    const float w = exp2f(m - mz);
    acc = make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w);
    l *= w;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (c + j <= b2) {
        const float wj = exp2f(ml[j].x - mz);
        acc.x = fmaf(wj, v[j].x, acc.x);
        acc.y = fmaf(wj, v[j].y, acc.y);
        acc.z = fmaf(wj, v[j].z, acc.z);
        acc.w = fmaf(wj, v[j].w, acc.w);
        l = fmaf(wj, ml[j].y, l);  // (a NaN sum stays one also under a zero weight)
      }
    }
    m = mn;
  }
}

}  // namespace kvs
