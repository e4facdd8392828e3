// kvs_rope.cuh -- what the rotary kernels share: the sequence of a row and the
// exact reduction of an angle (rope_scatter.cu has the mathematics).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kvs_paged.cuh"

namespace kvs {

// The sequence whose rows hold `row`, by one warp (every lane gets index and
// sequence): its index is the number of sequences that end at or before the
// row, M behind the last one.
__device__ __forceinline__ int warp_find_seq(const PagedArgs &b, int row, int lane, PagedSeq &s) {
  if (b.M <= 32) {  // offsets and positions in one round trip
    PagedSeq mine{0, 0, 0, KVS_OK};
    if (lane < b.M) mine = paged_seq(b, lane);
    const bool before = lane < b.M && __ldca(b.row_offsets + lane + 1) <= row;
    const int i = __popc(__ballot_sync(0xffffffffu, before));
    const int src = i & 31;
    s.p = __shfl_sync(0xffffffffu, mine.p, src);
    s.n = __shfl_sync(0xffffffffu, mine.n, src);
    s.row0 = __shfl_sync(0xffffffffu, mine.row0, src);
    s.err = __shfl_sync(0xffffffffu, mine.err, src);
    return i;
  }
  int n = 0;
  for (int i = lane; i < b.M; i += 32) n += __ldca(b.row_offsets + i + 1) <= row;
  n = __reduce_add_sync(0xffffffffu, n);
  if (n < b.M) s = paged_seq(b, n);
  return n;
}

// Where pair j's (cos, sin) sits in shared memory: one gap for eight pairs,
// so that the eight lanes of a head that read pairs 8 apart hit 16 banks.
__device__ __forceinline__ constexpr int cs_at(int j) { return j + (j >> 3); }

// Turns a position, in units of 2^-64 turns: |w| / 2 pi modulo 1.  w = f 2^e
// with a 24-bit integer f and e < 0 (|w| < 2^24), and 1 / 2 pi to 128 bits,
// so the integer product f / 2 pi is exact to 2^-64 before the shift by -e.
__device__ __forceinline__ unsigned long long turns_of(float w) {
  constexpr unsigned long long kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;
  const unsigned u = __float_as_uint(w);
  const unsigned ex = (u >> 23) & 255u;
  const unsigned long long f = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int e = 150 - (int)(ex ? ex : 1u);  // w = f 2^-e
  // f (hi + lo 2^-64), a number of 64 + 24 bits
  const unsigned long long low = f * kHi, carry = __umul64hi(f, kLo);
  const unsigned long long sum = low + carry;
  const unsigned long long high = __umul64hi(f, kHi) + (sum < low ? 1ull : 0ull);
  unsigned long long t;
  if (e >= 128)
    t = 0ull;
  else if (e >= 64)
    t = high >> (e - 64);
  else if (e > 0)
    t = (sum >> e) | (high << (64 - e));
  else
    t = sum << -e;  // (beyond the documented range: whole turns drop out)
  return (u >> 31) ? 0ull - t : t;
}

}  // namespace kvs
