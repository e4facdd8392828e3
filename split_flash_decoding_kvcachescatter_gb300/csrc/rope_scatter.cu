// rope_scatter.cu -- rotary positions on a ragged batch's new queries and
// keys, and the new K and V rows written into a paged cache, in one launch.
//
// Mathematics: pair j of a head at position P turns by t = P w_j.  t matters
// modulo a full turn only, so the kernel makes w_j / 2 pi a 64-bit binary
// fraction of a turn (in integers) and multiplies it by P in wrapping 64-bit
// integers: the reduction is exact, where a float32 product P w_j would be
// off by 2^-24 P w_j radians (0.008 at position 131072).  The top 32 bits of
// the fraction go to sincospi.
//
// Bound: bytes (each row of q, k, v read once and written once).  A block
// takes one token, or a slice of its heads when tokens are few: it puts the
// token's rot_dim / 2 (cos, sin) pairs in shared memory once for all heads,
// then each thread moves up to kRopeItems pair vectors at a time (two 16-byte
// loads each with the half layout), all loads issued before the first is used.
//
// Measured: 8192 tokens, H 32 / 8, D 128, bfloat16 (201 MB read and written)
// 36.9 us, 5.4 TB/s, 80 % of the measured copy peak; a decode step of 32
// tokens 2.7 us; 1531 tokens, H 14 / 2, D 64, float32, 16 elements rotated in
// pairs 5.4 us.  (Ten blocks an SM leave 48 registers a thread: the half layout
// at its widest spills 68 bytes, in float32 100.)  Threads x vectors, for the first: 128 x 3 36.9, 192 x 2 36.5,
// 96 x 4 37.8, 64 x 6 41, 384 x 1 48 us.

#include "kvs_paged.cuh"
#include "kvs_rope.cuh"

namespace kvs {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeItems = 3;

struct RopeArgs {
  const void *q, *k, *v;
  void *q_out, *k_pages, *v_pages;
  long long q_stride, k_stride, v_stride, q_out_stride;
  const float *inv_freq;
  int H, Hkv, D, rot;
  float scale;
};

// grid (num_rows, slices).  VE: elements of a vector; IL: interleaved pairs.
// A thread's first vectors are loaded before anything is known of the row's
// sequence, so that the look-ups (offsets, position, page) run in the shadow
// of the copy.
template <typename T, int VE, bool IL>
__global__ void __launch_bounds__(kRopeThreads, 10)
    rope_scatter_kernel(RopeArgs a, PagedArgs b, int *d_status) {
  __shared__ float2 cs[cs_at(64)];
  const int tid = threadIdx.x;
  const int row = blockIdx.x;
  const int half = a.rot / 2;
  // vectors of a rotated head: pair vectors first, then those copied
  const int npair = IL ? a.rot / VE : half / VE;
  const int per_head = npair + (a.D - a.rot) / VE;
  const float inv_per_head = 1.f / (float)per_head;
  const int nrot = (a.H + a.Hkv) * per_head;
  const int total = nrot + a.Hkv * (a.D / VE);
  const T *q = static_cast<const T *>(a.q) + (long long)row * a.q_stride;
  const T *k = static_cast<const T *>(a.k) + (long long)row * a.k_stride;
  const T *v = static_cast<const T *>(a.v) + (long long)row * a.v_stride;
  const int step = kRopeThreads * gridDim.y;
  Vec<T, VE> x[kRopeItems], y[kRopeItems];
  // item it: vector w of head h (q's heads, k's, then v's with every vector copied)
  auto where = [&](int it, int &h, int &w, int &first) {  // first: its element in the head
    if (it < nrot) {
      h = (int)(((float)it + 0.5f) * inv_per_head);  // it / per_head (it < 2^20)
      w = it - h * per_head;
      first = w < npair ? w * VE : a.rot + (w - npair) * VE;
    } else {
      const int e = (it - nrot) * VE;
      h = e / a.D;
      first = e - h * a.D;
      h += a.H + a.Hkv;
      w = npair;
    }
  };
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kRopeItems; ++u) {
      const int it = base + u * step;
      if (it >= total) break;
      int h, w, first;
      where(it, h, w, first);
      const T *src = (h < a.H               ? q + h * a.D
                      : h < a.H + a.Hkv     ? k + (h - a.H) * a.D
                                            : v + (h - a.H - a.Hkv) * a.D) +
                     first;
      x[u] = vec_load<T, VE>(src);
      if (!IL && w < npair) y[u] = vec_load<T, VE>(src + half);
    }
  };
  int base = blockIdx.y * kRopeThreads + tid;
  grid_dependency_wait();
  load(base);
  allow_dependent_launch();
  if (blockIdx.y == 0)  // the status of every sequence, spread over the blocks (past 2^31 threads)
    for (long long i = (long long)row * kRopeThreads + tid; i < b.M;
         i += (long long)gridDim.x * kRopeThreads) {
      const int err = paged_seq(b, (int)i).err;
      if (err != KVS_OK) record_status(d_status, err);
    }
  PagedSeq s{0, 0, 0, KVS_OK};
  const int i = warp_find_seq(b, row, tid & 31, s);
  if (i >= b.M) return;  // a row behind the last sequence
  if (s.err == KVS_ERR_ROWS || row < s.row0 || row >= s.row0 + s.n) return;
  const bool bad_pos = s.err != KVS_OK;
  const int pos = s.p + (row - s.row0);
  int page = -1;
  if (!bad_pos) {
    page = __ldca(b.page_table + (size_t)i * b.max_pages + (pos >> b.page_shift));
    if ((unsigned)page >= (unsigned)b.num_pages) {
      if (tid == 0) record_status(d_status, KVS_ERR_PAGE);
      page = -1;
    }
  }
  if (tid < half) {  // (half <= 64 < kRopeThreads)
    const unsigned long long turn = turns_of(a.inv_freq[tid]) * (unsigned long long)(unsigned)pos;
    // the angle over pi, in [-1, 1): the fraction's top 32 bits, signed, times 2^-31
    const float t = (float)(int)(unsigned)(turn >> 32) * 4.656612873077393e-10f;
    float sn, c;
    sincospif(t, &sn, &c);
    cs[cs_at(tid)] = make_float2(c * a.scale, sn * a.scale);
  }
  __syncthreads();
  T *qo = static_cast<T *>(a.q_out) + (long long)row * a.q_out_stride;
  // kv head g's row in the page: elements g * head_step further
  const size_t head_step = (size_t)a.D << b.page_shift;
  const size_t page_at = (size_t)(page < 0 ? 0 : page) * a.Hkv * head_step +
                         (size_t)(pos & ((1 << b.page_shift) - 1)) * a.D;
  T *kp = static_cast<T *>(a.k_pages) + page_at;
  T *vp = static_cast<T *>(a.v_pages) + page_at;
  for (;;) {
#pragma unroll
    for (int u = 0; u < kRopeItems; ++u) {
      const int it = base + u * step;
      if (it >= total) break;
      int h, w, first;
      where(it, h, w, first);
      if (page < 0 && h >= a.H) continue;  // nowhere to write
      T *dst = (h < a.H             ? qo + h * a.D
                : h < a.H + a.Hkv   ? kp + (h - a.H) * head_step
                                    : vp + (h - a.H - a.Hkv) * head_step) +
               first;
      if (bad_pos) {  // (page is -1, so this is q_out)
        const T nan = from_f32<T>(__int_as_float(0x7fc00000));
#pragma unroll
        for (int e = 0; e < VE; ++e) x[u].e[e] = y[u].e[e] = nan;
      } else if (w < npair) {
        if (IL) {
#pragma unroll
          for (int e = 0; e + 1 < VE; e += 2) {
            const float2 t = cs[cs_at(w * (VE / 2) + e / 2)];
            const float p = to_f32(x[u].e[e]), r = to_f32(x[u].e[e + 1]);
            x[u].e[e] = from_f32<T>(p * t.x - r * t.y);
            x[u].e[e + 1] = from_f32<T>(r * t.x + p * t.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float2 t = cs[cs_at(w * VE + e)];
            const float p = to_f32(x[u].e[e]), r = to_f32(y[u].e[e]);
            x[u].e[e] = from_f32<T>(p * t.x - r * t.y);
            y[u].e[e] = from_f32<T>(r * t.x + p * t.y);
          }
        }
      }
      vec_store<T, VE>(dst, x[u]);
      if (!IL && w < npair) vec_store<T, VE>(dst + half, y[u]);
    }
    base += kRopeItems * step;
    if (base >= total) break;
    load(base);
  }
}

template <typename T, int VE, bool IL>
int launch_rope(const RopeArgs &a, const PagedArgs &b, int *d_status, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return KVS_ERR_LAUNCH;
  const int total = (a.H + a.Hkv) * ((IL ? a.rot / VE : a.rot / 2 / VE) + (a.D - a.rot) / VE) +
                    a.Hkv * (a.D / VE);
  // Few tokens: a token's vectors are split over blocks until every SM has
  // one block or a thread has one vector left.
  const int most = (total + kRopeThreads - 1) / kRopeThreads;
  const int want = (2 * sms + b.num_rows - 1) / b.num_rows;
  const int slices = want < 1 ? 1 : want < most ? want : most;
  const cudaError_t e =
      launch_pdl(rope_scatter_kernel<T, VE, IL>, dim3((unsigned)b.num_rows, (unsigned)slices),
                 dim3(kRopeThreads), 0, stream, a, b, d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

// The widest vector (16 bytes at most) that the head splits into: it must
// divide the rotated half (half layout) or the rotated part (interleaved).
template <typename T>
int dispatch_rope(const RopeArgs &a, const PagedArgs &b, int interleaved, int *d_status,
                  cudaStream_t stream) {
  constexpr int kMost = 16 / sizeof(T);
  const int n = interleaved ? a.rot : a.rot / 2;
  if (n % kMost == 0)
    return interleaved ? launch_rope<T, kMost, true>(a, b, d_status, stream)
                       : launch_rope<T, kMost, false>(a, b, d_status, stream);
  if (kMost == 8 && n % 4 == 0)
    return interleaved ? launch_rope<T, 4, true>(a, b, d_status, stream)
                       : launch_rope<T, 4, false>(a, b, d_status, stream);
  if (n % 2 == 0)
    return interleaved ? launch_rope<T, 2, true>(a, b, d_status, stream)
                       : launch_rope<T, 2, false>(a, b, d_status, stream);
  return launch_rope<T, 1, false>(a, b, d_status, stream);  // (interleaved: rot is even)
}

}  // namespace

int launch_rope_scatter(const void *q, long long q_stride, const void *k, long long k_stride,
                        const void *v, long long v_stride, void *q_out, long long q_out_stride,
                        void *k_pages, void *v_pages, const PagedArgs &b, const float *inv_freq,
                        int H, int Hkv, int D, int dtype, int rot, int interleaved, float scale,
                        int *d_status, cudaStream_t stream) {
  const RopeArgs a{q,        k,        v,   q_out, k_pages, v_pages, q_stride, k_stride,
                   v_stride, q_out_stride, inv_freq, H,     Hkv,     D,       rot,      scale};
  if (dtype == KVS_F32) return dispatch_rope<float>(a, b, interleaved, d_status, stream);
  if (dtype == KVS_F16) return dispatch_rope<__half>(a, b, interleaved, d_status, stream);
  return dispatch_rope<__nv_bfloat16>(a, b, interleaved, d_status, stream);
}

}  // namespace kvs
