// kvs_tags.cuh -- completion counters that need no initialisation: each
// carries the tag of the call that last used it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kvs_device.cuh"

namespace kvs {

// Counters tagged with the call that last used them: the value is
// (tag << 32 | count).  A value left by another call (another tag, or
// whatever the workspace held) counts as zero: the first adder of this call
// replaces it with (tag, amount).  Each returns the count before the add.
// Bounded: after 2^20 failed attempts they record KVS_ERR_TIMEOUT and return
// 0xffffffff.  `v` is what an atomicAdd(ctr, amount) returned.
static __device__ unsigned resolve_tagged_add(unsigned long long *ctr, unsigned long long v,
                                              unsigned amount, unsigned tag, int *d_status,
                                              unsigned *epoch) {
  for (int attempt = 0; attempt < (1 << 20); ++attempt) {
    if ((unsigned)(v >> 32) == tag) return (unsigned)v;
    const unsigned long long cur = v + amount;
    const unsigned long long mine = ((unsigned long long)tag << 32) | amount;
    const unsigned long long prev = atomicCAS(ctr, cur, mine);
    if (prev == cur) return 0u;
    if ((unsigned)(prev >> 32) == tag)
      v = atomicAdd(ctr, (unsigned long long)amount);
    else
      v = prev - amount;
  }
  record_status(d_status, KVS_ERR_TIMEOUT);
  atomicAdd(epoch, 1u);
  return 0xffffffffu;
}

static __device__ __forceinline__ unsigned tagged_add(unsigned long long *ctr, unsigned amount,
                                                      unsigned tag, int *d_status,
                                                      unsigned *epoch) {
  return resolve_tagged_add(ctr, atomicAdd(ctr, (unsigned long long)amount), amount, tag,
                            d_status, epoch);
}

// The tag this launch's counters carry: the host's per-launch tag combined
// with the workspace epoch.  Every block of a launch reads the same epoch
// (nothing changes it unless a block gives up), so every block computes the
// same tag.  A launch that gives up changes the epoch, so the counts it
// leaves can never be taken for a later launch's own, not even by a replayed
// graph, whose host tag is frozen at capture.  Never 0: a reset counter
// holds tag 0.
__device__ __forceinline__ unsigned launch_tag(unsigned host_tag, unsigned epoch) {
  const unsigned t = host_tag ^ (epoch * 0x9E3779B1u);
  return t != 0u ? t : 0x5BD1E995u;
}

__device__ __forceinline__ unsigned long long ld_acquire_u64(const unsigned long long *p) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}

// A block gives up the call: stop every role of the block, report it, and
// move the workspace epoch on (see launch_tag).
__device__ __forceinline__ void give_up(volatile int *abort, int *d_status, unsigned *epoch) {
  *abort = 1;
  record_status(d_status, KVS_ERR_TIMEOUT);
  atomicAdd(epoch, 1u);
}

}  // namespace kvs
