// rope_scatter_q8.cu -- rotary positions on a ragged batch's new queries and
// keys, and the new K and V rows written into a paged cache in 8 bits, in one
// launch.
//
// Mathematics: the rotation as in rope_scatter.cu.  A block of 16 positions of a
// kv head shares a scale, the least power of two 2^k (k >= -60) that keeps every
// row written to it within 448 2^k; its rows are rounded to e4m3 after division by
// it, which is exact.  Where a block holds older rows its scale can only grow, and
// its older numbers are then divided by the growth and rounded again (exact down
// to 2^-6, the end of e4m3's normal range).
//
// A thread block takes the 16-position blocks whose first new row lies in its
// rows of the batch, and a slice of the heads: it makes the (cos, sin) of the
// block's tokens in shared memory once, then a warp takes a head at a time: one
// pass over the new rows for the largest element, one that rounds and writes them
// (the rows come from L2 then).
//
// Bound: bytes (each row of q, k, v read once, q and the 8-bit rows written once).

#include "kvs_fp8.cuh"
#include "kvs_paged.cuh"
#include "kvs_rope.cuh"

namespace kvs {

namespace {

constexpr int kRqThreads = 256;

struct RopeQ8Args {
  const void *q, *k, *v;
  void *q_out;
  uint8_t *k_pages, *v_pages;
  float *k_scales, *v_scales;
  long long q_stride, k_stride, v_stride, q_out_stride;
  const float *inv_freq;
  int H, Hkv, D, rot, group;  // group: rows of the batch that a thread block looks at
  float scale;
};

// VE numbers to e4m3 at p (aligned to VE bytes).
template <int VE>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[VE], float inv) {
  if constexpr (VE == 8) {
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                   to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
  } else if constexpr (VE == 4) {
    *reinterpret_cast<unsigned *>(p) = to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
  } else if constexpr (VE == 2) {
    *reinterpret_cast<unsigned short *>(p) = (unsigned short)to_e4m3x2(f[0] * inv, f[1] * inv);
  } else {
    *p = (uint8_t)to_e4m3x2(f[0] * inv, 0.f);
  }
}

// VE: elements of a vector; IL: interleaved pairs.
template <typename T, int VE, bool IL>
__global__ void __launch_bounds__(kRqThreads)
    rope_scatter_q8_kernel(RopeQ8Args a, PagedArgs b, int *d_status) {
  __shared__ float2 cs[kScaleBlock][cs_at(64)];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = a.rot / 2;
  // vectors of a rotated head: pair vectors first, then those copied
  const int npair = IL ? a.rot / VE : half / VE;
  const int per_head = npair + (a.D - a.rot) / VE;
  const float inv_per_head = 1.f / (float)per_head, inv_half = 1.f / (float)max(half, 1);
  const int first_row = (int)min((long long)blockIdx.x * a.group, (long long)b.num_rows);
  const int end_row = (int)min((long long)first_row + a.group, (long long)b.num_rows);
  grid_dependency_wait();
  allow_dependent_launch();
  if (blockIdx.y == 0)  // the status of every sequence, spread over the blocks
    for (long long i = (long long)blockIdx.x * kRqThreads + tid; i < b.M;
         i += (long long)gridDim.x * kRqThreads) {
      const int err = paged_seq(b, (int)i).err;
      if (err != KVS_OK) record_status(d_status, err);
    }
  for (int row = first_row; row < end_row;) {  // (the same for every thread)
    PagedSeq s{0, 0, 0, KVS_OK};
    const int i = warp_find_seq(b, row, lane, s);
    if (i >= b.M) return;  // rows behind the last sequence
    if (s.err == KVS_ERR_ROWS || row < s.row0 || row >= s.row0 + s.n) {
      ++row;
      continue;
    }
    const int t0 = row - s.row0;
    const bool bad_pos = s.err != KVS_OK;
    if (bad_pos) {  // its rows are NaN
      const T nan = from_f32<T>(__int_as_float(0x7fc00000));
      T *qo = static_cast<T *>(a.q_out) + (long long)row * a.q_out_stride;
      if (blockIdx.y == 0)
        for (int e = tid; e < a.H * a.D; e += kRqThreads) qo[e] = nan;
      ++row;
      continue;
    }
    const int pos = s.p + t0, in = pos & (kScaleBlock - 1);
    if (t0 > 0 && in != 0) {  // an earlier row begins this block
      row += min(kScaleBlock - in, s.n - t0);
      continue;
    }
    const int ntok = min(kScaleBlock - in, s.n - t0);
    const int page = __ldca(b.page_table + (size_t)i * b.max_pages + (pos >> b.page_shift));
    const bool bad_page = (unsigned)page >= (unsigned)b.num_pages;
    if (bad_page && tid == 0) record_status(d_status, KVS_ERR_PAGE);
    __syncthreads();  // the table of the block before has been read
    for (int e = tid; e < ntok * half; e += kRqThreads) {
      const int tok = (int)(((float)e + 0.5f) * inv_half), j = e - tok * half;
      const unsigned long long turn =
          turns_of(a.inv_freq[j]) * (unsigned long long)(unsigned)(pos + tok);
      // the angle over pi, in [-1, 1): the fraction's top 32 bits, signed, times 2^-31
      const float t = (float)(int)(unsigned)(turn >> 32) * 4.656612873077393e-10f;
      float sn, c;
      sincospif(t, &sn, &c);
      cs[tok][cs_at(j)] = make_float2(c * a.scale, sn * a.scale);
    }
    __syncthreads();
    // f(token, element of the head, its vector, the second one of a half-layout pair or
    // nullptr) for every vector of a head's new rows
    auto each = [&](const T *src, long long stride, bool turn, auto f) {
      const int total = ntok * (turn ? per_head : a.D / VE);
      for (int it = lane; it < total; it += 32) {
        int tok, w, first;
        if (turn) {
          tok = (int)(((float)it + 0.5f) * inv_per_head);
          w = it - tok * per_head;
          first = w < npair ? w * VE : a.rot + (w - npair) * VE;
        } else {
          tok = it / (a.D / VE);
          first = (it - tok * (a.D / VE)) * VE;
          w = npair;
        }
        const T *at = src + tok * stride + first;
        const Vec<T, VE> x = vec_load<T, VE>(at);
        float fx[VE], fy[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) fx[e] = to_f32(x.e[e]);
        const bool pair = !IL && w < npair;
        if (w < npair) {
          if constexpr (IL) {
#pragma unroll
            for (int e = 0; e + 1 < VE; e += 2) {
              const float2 t = cs[tok][cs_at(w * (VE / 2) + e / 2)];
              const float p = fx[e], r = fx[e + 1];
              fx[e] = p * t.x - r * t.y;
              fx[e + 1] = r * t.x + p * t.y;
            }
          } else {
            const Vec<T, VE> y = vec_load<T, VE>(at + half);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              const float2 t = cs[tok][cs_at(w * VE + e)];
              const float p = fx[e], r = to_f32(y.e[e]);
              fx[e] = p * t.x - r * t.y;
              fy[e] = r * t.x + p * t.y;
            }
          }
        }
        f(tok, first, fx, fy, pair);
      }
    };
    const size_t head_step = (size_t)a.D << b.page_shift;  // elements of a kv head's page
    const int nb_shift = b.page_shift - 4;                 // blocks of a page
    const int slot = pos & ((1 << b.page_shift) - 1);
    const int items = a.H + 2 * a.Hkv;
    for (int h = blockIdx.y * (kRqThreads / 32) + warp; h < items; h += gridDim.y * (kRqThreads / 32)) {
      if (h < a.H) {
        T *qo = static_cast<T *>(a.q_out) + (long long)row * a.q_out_stride + h * a.D;
        each(static_cast<const T *>(a.q) + (long long)row * a.q_stride + h * a.D, a.q_stride, true,
             [&](int tok, int first, const float(&fx)[VE], const float(&fy)[VE], bool pair) {
               T *to = qo + tok * a.q_out_stride + first;
               Vec<T, VE> x;
#pragma unroll
               for (int e = 0; e < VE; ++e) x.e[e] = from_f32<T>(fx[e]);
               vec_store<T, VE>(to, x);
               if (pair) {
#pragma unroll
                 for (int e = 0; e < VE; ++e) x.e[e] = from_f32<T>(fy[e]);
                 vec_store<T, VE>(to + half, x);
               }
             });
        continue;
      }
      if (bad_page) continue;  // nowhere to write
      const bool is_k = h < a.H + a.Hkv;
      const int g = h - a.H - (is_k ? 0 : a.Hkv);
      const T *src = is_k ? static_cast<const T *>(a.k) + (long long)row * a.k_stride + g * a.D
                          : static_cast<const T *>(a.v) + (long long)row * a.v_stride + g * a.D;
      const long long stride = is_k ? a.k_stride : a.v_stride;
      const size_t head = (size_t)page * a.Hkv + g;
      float *scale_at = (is_k ? a.k_scales : a.v_scales) + (head << nb_shift) + (slot >> 4);
      uint8_t *block = (is_k ? a.k_pages : a.v_pages) + head * head_step + (size_t)(slot - in) * a.D;
      const float old = in > 0 ? __ldcg(scale_at) : 0.f;
      float most = 0.f;
      each(src, stride, is_k, [&](int, int, const float(&fx)[VE], const float(&fy)[VE], bool pair) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          most = fmaxf(most, fabsf(fx[e]));
          if (pair) most = fmaxf(most, fabsf(fy[e]));
        }
      });
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      float scale = scale_for(most);
      if (in > 0 && old >= scale) {
        scale = old;
      } else {
        if (in > 0) {  // older rows under a scale that has grown
          const float ratio = old / scale;
          unsigned *w = reinterpret_cast<unsigned *>(block);
          for (int e = lane; e < in * a.D / 4; e += 32) {
            const unsigned x = __ldcg(w + e);
            const uint32_t u0 = from_e4m3x2(x), u1 = from_e4m3x2(x >> 16);
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&u0));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&u1));
            w[e] = to_e4m3x4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio);
          }
        }
        if (lane == 0) *scale_at = scale;
      }
      const float inv = 1.f / scale;
      uint8_t *to = block + in * a.D;
      each(src, stride, is_k,
           [&](int tok, int first, const float(&fx)[VE], const float(&fy)[VE], bool pair) {
             store_e4m3<VE>(to + tok * a.D + first, fx, inv);
             if (pair) store_e4m3<VE>(to + tok * a.D + first + half, fy, inv);
           });
    }
    row += ntok;
  }
}

template <typename T, int VE, bool IL>
int launch_rope(RopeQ8Args a, const PagedArgs &b, int *d_status, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return KVS_ERR_LAUNCH;
  // Few rows: a thread block a row (those that do not begin a block of 16 leave at
  // once); else 16 rows, which begin one block of a prompt.
  a.group = b.num_rows <= 4 * sms ? 1 : kScaleBlock;
  const int groups = (b.num_rows + a.group - 1) / a.group;
  const int most = (a.H + 2 * a.Hkv + kRqThreads / 32 - 1) / (kRqThreads / 32);
  const int want = (8 * sms + groups - 1) / groups;
  const int slices = want < 1 ? 1 : want < most ? want : most;
  const cudaError_t e =
      launch_pdl(rope_scatter_q8_kernel<T, VE, IL>, dim3((unsigned)groups, (unsigned)slices),
                 dim3(kRqThreads), 0, stream, a, b, d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

// The widest vector (16 bytes at most) that the head splits into (rope_scatter.cu).
template <typename T>
int dispatch_rope(const RopeQ8Args &a, const PagedArgs &b, int interleaved, int *d_status,
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

int launch_rope_scatter_q8(const void *q, long long q_stride, const void *k, long long k_stride,
                           const void *v, long long v_stride, void *q_out, long long q_out_stride,
                           const kvs_paged_cache_q8 &cache, int dtype, const PagedArgs &b,
                           const float *inv_freq, int H, int rot, int interleaved, float scale,
                           int *d_status, cudaStream_t stream) {
  const RopeQ8Args a{q, k, v, q_out, static_cast<uint8_t *>(cache.k_pages),
                     static_cast<uint8_t *>(cache.v_pages), cache.k_scales, cache.v_scales,
                     q_stride, k_stride, v_stride, q_out_stride, inv_freq, H, cache.num_kv_heads,
                     cache.head_dim, rot, 1, scale};
  if (dtype == KVS_F32) return dispatch_rope<float>(a, b, interleaved, d_status, stream);
  if (dtype == KVS_F16) return dispatch_rope<__half>(a, b, interleaved, d_status, stream);
  return dispatch_rope<__nv_bfloat16>(a, b, interleaved, d_status, stream);
}

}  // namespace kvs
