// rope_scatter_q8.cu -- rotary positions on a ragged batch's new queries and
// keys, and the new K and V rows written into a paged cache in 8 bits, in one
// launch.
//
// Mathematics: the rotation as in rope_scatter.cu.  A block of 16 positions of a
// kv head shares a scale, the least power of two 2^k (-60 <= k <= 100) that keeps every
// finite element written to it within 448 2^k; its rows are rounded to e4m3 after division by
// it, which is exact.  Where a block holds older rows its scale can only grow, and
// its older numbers are then divided by the growth and rounded again (exact down
// to 2^-6, the end of e4m3's normal range).
//
// Bound: bytes (each row of q, k, v read once, q and the 8-bit rows written once).  Two
// kernels.  The usual one, for heads of whole 16-byte vectors that turn whole or in
// interleaved pairs, has two kinds of thread blocks in one launch.  K or V: the 16-position
// blocks whose first new row lies in the thread block's rows of the batch, two warps a kv
// head, eight rows each, which hold the turned rows in registers between the look for the
// largest element and the rounding.  q: a token or two.  Both issue their loads before
// the look-ups (sequence, page, old scale) that decide where the results go.
// The other kernel, for any head: a warp a head of a 16-position block at a time, the rows
// of K and V read twice.
// Measured (32 query heads on 8 kv heads of 128, bfloat16): 8192 rows of prompts 41 us, 66% of
// what a copy of the same bytes takes; by the other kernel 82 (with 64 or 32 of 128 turned, too); 16 rows a warp 64, eight of them
// with q's angles made by every warp 72 to 78.  A decode step of 32 tokens: 3.2 us, a launch
// and four dependent reads.

#include <type_traits>

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

// Older numbers of a block, `words` words of four, under a scale that has grown: times
// `ratio`, rounded again.  By threads `first`, first + step, ...
__device__ __forceinline__ void requantise(unsigned *w, int words, int first, int step, float ratio) {
  for (int e = first; e < words; e += step) {
    const unsigned x = __ldcg(w + e);
    const uint32_t u0 = from_e4m3x2(x), u1 = from_e4m3x2(x >> 16);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&u0));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&u1));
    w[e] = to_e4m3x4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio);
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
          most = finite_max(most, fx[e]);
          if (pair) most = finite_max(most, fy[e]);
        }
      });
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      float scale = scale_for(most);
      if (in > 0 && old >= scale) {
        scale = old;
      } else {
        if (in > 0) requantise(reinterpret_cast<unsigned *>(block), in * a.D / 4, lane, 32, old / scale);
        __syncwarp();  // every lane has read the old scale
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

// ---- whole vectors ---------------------------------------------------------------
constexpr int kWThreads = 256;
constexpr int kWHeads = kWThreads / 64;  // kv heads of a thread block: two warps each
constexpr int kWRows = kScaleBlock / 2;  // rows of a warp
constexpr int kWTokens = 2;              // rows of q a thread block has at most

struct WholeArgs {
  RopeQ8Args r;
  int kv_parts, kv_blocks;  // parts of the kv heads (K's, then V's), thread blocks for K and V
  int q_tokens, q_parts;    // rows of q a thread block, and parts of a row
};

// (cos, sin) of a frequency's turns at a position, times scale.
__device__ __forceinline__ float2 angle_of(unsigned long long turns, int pos, float scale) {
  const unsigned long long turn = turns * (unsigned long long)(unsigned)pos;
  // the angle over pi, in [-1, 1): the fraction's top 32 bits, signed, times 2^-31
  const float t = (float)(int)(unsigned)(turn >> 32) * 4.656612873077393e-10f;
  float sn, c;
  sincospif(t, &sn, &c);
  return make_float2(c * scale, sn * scale);
}

// A token's (cos, sin) in shared memory: those of vector w of a head in float4s, one a row
// of the table, so that the lanes of a head read 16 bytes side by side.
template <int VE, bool IL, int D>
struct Angles {
  static constexpr int kOf = IL ? VE / 2 : VE;        // pairs of a vector
  static constexpr int kVectors = D / 2 / kOf;        // vectors that turn, at most
  static __device__ __forceinline__ int at(int j) {   // of pair j
    const int w = j / kOf, e = j % kOf;
    return ((e >> 1) * kVectors + w) * 4 + (e & 1) * 2;
  }
  // turns vector x (IL), or the pair (x, y)
  static __device__ __forceinline__ void turn(const float *table, int w, float (&x)[VE], float (&y)[VE]) {
#pragma unroll
    for (int c = 0; c < kOf / 2; ++c) {
      const float4 t = *reinterpret_cast<const float4 *>(table + (c * kVectors + w) * 4);
      if constexpr (IL) {
        const float p0 = x[4 * c], r0 = x[4 * c + 1], p1 = x[4 * c + 2], r1 = x[4 * c + 3];
        x[4 * c] = p0 * t.x - r0 * t.y;
        x[4 * c + 1] = r0 * t.x + p0 * t.y;
        x[4 * c + 2] = p1 * t.z - r1 * t.w;
        x[4 * c + 3] = r1 * t.z + p1 * t.w;
      } else {
        const float p0 = x[2 * c], r0 = y[2 * c], p1 = x[2 * c + 1], r1 = y[2 * c + 1];
        x[2 * c] = p0 * t.x - r0 * t.y;
        y[2 * c] = r0 * t.x + p0 * t.y;
        x[2 * c + 1] = p1 * t.z - r1 * t.w;
        y[2 * c + 1] = r1 * t.z + p1 * t.w;
      }
    }
  }
};

template <typename T, int VE>
__device__ __forceinline__ void to_floats(const Vec<T, VE> &v, float (&f)[VE]) {
#pragma unroll
  for (int e = 0; e < VE; ++e) f[e] = to_f32(v.e[e]);
}

// IL: interleaved pairs, of which rot / 2 turn; else the half layout, turned whole.
template <typename T, bool IL, int D>
__global__ void __launch_bounds__(kWThreads, sizeof(T) == 4 ? 3 : 4)
    rope_q8_whole_kernel(WholeArgs wa, PagedArgs b, int *d_status) {
  constexpr int VE = 16 / sizeof(T);
  using A = Angles<VE, IL, D>;
  constexpr int PV = IL ? D / VE : D / 2 / VE;   // units of a row: vectors, or pairs of them
  constexpr int U = kWRows * PV / 32;            // of a lane, eight rows a warp
  constexpr int UV = kWRows * D / VE / 32;       // vectors of V, the same
  static_assert(U >= 1 && 32 % PV == 0, "a lane's units lie in rows 32 / PV apart");
  const RopeQ8Args &a = wa.r;
  __shared__ __align__(16) float cs[kScaleBlock][D];
  __shared__ float s_most[kWThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = a.rot / 2, nturn = IL ? a.rot / VE : PV;  // pairs that turn, units that do
  grid_dependency_wait();
  if ((int)blockIdx.x >= wa.kv_blocks) {
    // ======================= q =================================================
    const int block = (int)blockIdx.x - wa.kv_blocks, part = block % wa.q_parts;
    const int row0 = block / wa.q_parts * wa.q_tokens, ntok = min(wa.q_tokens, b.num_rows - row0);
    const int of_token = a.H * PV, step = kWThreads * wa.q_parts;
    Vec<T, VE> x[kWTokens], y[kWTokens];
    auto load = [&](int it) {
#pragma unroll
      for (int t = 0; t < kWTokens; ++t) {
        if (t >= ntok || it >= of_token) break;
        const T *src = static_cast<const T *>(a.q) + (long long)(row0 + t) * a.q_stride + (it / PV) * D + (it % PV) * VE;
        x[t] = vec_load<T, VE>(src);
        if constexpr (!IL) y[t] = vec_load<T, VE>(src + D / 2);
      }
    };
    int it = part * kWThreads + tid;
    load(it);
    const unsigned long long turns = tid % (D / 2) < half ? turns_of(a.inv_freq[tid % (D / 2)]) : 0ull;
    allow_dependent_launch();
    if (part == 0)  // the status of every sequence, spread over the blocks
      for (long long i = (long long)(block / wa.q_parts) * kWThreads + tid; i < b.M;
           i += (long long)((b.num_rows + wa.q_tokens - 1) / wa.q_tokens) * kWThreads) {
        const int err = paged_seq(b, (int)i).err;
        if (err != KVS_OK) record_status(d_status, err);
      }
    int state[kWTokens];  // 0: nothing to write, 1: rotated, 2: NaN
    PagedSeq s{0, 0, 0, KVS_OK};
    int i = -1;
#pragma unroll
    for (int t = 0; t < kWTokens; ++t) {
      state[t] = 0;
      const int row = row0 + t;
      if (t >= ntok) break;
      if (i < 0 || row >= s.row0 + s.n) i = warp_find_seq(b, row, lane, s);
      if (i >= b.M || s.err == KVS_ERR_ROWS || row < s.row0 || row >= s.row0 + s.n) {
        i = -1;
        continue;
      }
      state[t] = s.err != KVS_OK ? 2 : 1;
      if (tid / (D / 2) == t && tid % (D / 2) < half)
        *reinterpret_cast<float2 *>(&cs[t][A::at(tid % (D / 2))]) = angle_of(turns, s.p + row - s.row0, a.scale);
    }
    __syncthreads();
    for (; it < of_token; load(it)) {
      const int w = it % PV, at = (it / PV) * D + w * VE;
#pragma unroll
      for (int t = 0; t < kWTokens; ++t) {
        if (t >= ntok || state[t] == 0) continue;
        T *to = static_cast<T *>(a.q_out) + (long long)(row0 + t) * a.q_out_stride + at;
        if (state[t] == 2 || w < nturn) {
          float fx[VE], fy[VE];
          to_floats<T, VE>(x[t], fx);
          if constexpr (!IL) to_floats<T, VE>(y[t], fy);
          A::turn(cs[t], w, fx, fy);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            x[t].e[e] = from_f32<T>(state[t] == 2 ? __int_as_float(0x7fc00000) : fx[e]);
            if constexpr (!IL) y[t].e[e] = from_f32<T>(state[t] == 2 ? __int_as_float(0x7fc00000) : fy[e]);
          }
        }
        vec_store<T, VE>(to, x[t]);
        if constexpr (!IL) vec_store<T, VE>(to + D / 2, y[t]);
      }
      it += step;
    }
    return;
  }
  // ========================= K or V =============================================
  const int part = (int)blockIdx.x % wa.kv_parts, first_row = (int)blockIdx.x / wa.kv_parts * a.group;
  const int end_row = min(first_row + a.group, b.num_rows);
  const bool is_k = part < wa.kv_parts / 2;
  const int g = (is_k ? part : part - wa.kv_parts / 2) * kWHeads + (warp >> 1);  // this warp's kv head
  const int first_tok = (warp & 1) * kWRows;                                     // and rows of a block
  const bool works = g < a.Hkv;
  const long long stride = is_k ? a.k_stride : a.v_stride;
  const T *rows = static_cast<const T *>(is_k ? a.k : a.v) + (works ? g * D : 0) + first_tok * stride;
  // this lane's units: K's are unit lane % PV of rows lane / PV + 32 / PV u, V's vector lane %
  // (D / VE) of rows lane / (D / VE) + ... (a pair of vectors half a head apart is two of f)
  constexpr int kOfRow = D / VE;
  const int kw = lane % PV, kt = lane / PV, vw = lane % kOfRow, vt = lane / kOfRow;
  float f[UV][VE];
  auto load = [&](const T *src, int n) {  // n rows of this warp's at most
    if (is_k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tok = kt + 32 / PV * u;
        if (tok >= n) continue;
        const T *at = src + tok * stride + kw * VE;
        to_floats<T, VE>(vec_load<T, VE>(at), f[u]);
        if constexpr (!IL) to_floats<T, VE>(vec_load<T, VE>(at + D / 2), f[U + u]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < UV; ++u) {
        const int tok = vt + 32 / kOfRow * u;
        if (tok < n) to_floats<T, VE>(vec_load<T, VE>(src + tok * stride + vw * VE), f[u]);
      }
    }
  };
  if (works && a.group == 1) load(rows + (long long)first_row * stride, 1 - first_tok);  // (usually all of it)
  constexpr int kServe = kWThreads / (D / 2);  // tokens whose angles are made at a time
  const int jf = tid % (D / 2), tf = tid / (D / 2);
  const unsigned long long turns = is_k && jf < half ? turns_of(a.inv_freq[jf]) : 0ull;
  allow_dependent_launch();
  PagedSeq s{0, 0, 0, KVS_OK};
  int i = -1;
  for (int row = first_row; row < end_row;) {  // (the same for every thread)
    if (i < 0 || row >= s.row0 + s.n) {
      i = warp_find_seq(b, row, lane, s);
      if (i >= b.M) return;  // rows behind the last sequence
    }
    if (s.err != KVS_OK || row < s.row0 || row >= s.row0 + s.n) {
      i = -1;
      ++row;
      continue;
    }
    const int t0 = row - s.row0;
    const int pos = s.p + t0, in = pos & (kScaleBlock - 1);
    if (t0 > 0 && in != 0) {  // an earlier row begins this block
      row += min(kScaleBlock - in, s.n - t0);
      continue;
    }
    const int ntok = min(kScaleBlock - in, s.n - t0), mine = ntok - first_tok;
    const int page = __ldca(b.page_table + (size_t)i * b.max_pages + (pos >> b.page_shift));
    if (works && (a.group != 1 || ntok > 1)) load(rows + (long long)row * stride, mine);
    const bool bad_page = (unsigned)page >= (unsigned)b.num_pages;
    if (bad_page && tid == 0 && part == 0) record_status(d_status, KVS_ERR_PAGE);
    const int slot = pos & ((1 << b.page_shift) - 1);
    const size_t head = (size_t)(bad_page ? 0 : page) * a.Hkv + g;
    float *scale_at = (is_k ? a.k_scales : a.v_scales) + (head << (b.page_shift - 4)) + (slot >> 4);
    const float old = in > 0 && works && !bad_page ? __ldcg(scale_at) : 0.f;
    __syncthreads();  // the tables of the block before have been read
    if (is_k && jf < half)
      for (int t = tf; t < ntok; t += kServe)
        *reinterpret_cast<float2 *>(&cs[t][A::at(jf)]) = angle_of(turns, pos + t, a.scale);
    if (is_k) __syncthreads();
    row += ntok;
    float most = 0.f;
    if (works && is_k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tok = kt + 32 / PV * u;
        if (tok >= mine) continue;
        if (kw < nturn) A::turn(cs[first_tok + tok], kw, f[u], f[IL ? u : U + u]);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          most = fmaxf(most, fabsf(f[u][e]));
          if constexpr (!IL) most = fmaxf(most, fabsf(f[U + u][e]));
        }
      }
    } else if (works) {
#pragma unroll
      for (int u = 0; u < UV; ++u)
        if (vt + 32 / kOfRow * u < mine)
#pragma unroll
          for (int e = 0; e < VE; ++e) most = fmaxf(most, fabsf(f[u][e]));
    }
    // (sizes are ordered as integers; a NaN was passed over, and infinities are once there are
    // some: finite_max for all takes 42.3 us where this takes 41.4)
    unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (top == 0x7f800000u) {
      most = 0.f;
#pragma unroll
      for (int u = 0; u < UV; ++u) {
        const int tok = is_k ? kt + 32 / PV * (u % U) : vt + 32 / kOfRow * u;
        if (tok < mine)
#pragma unroll
          for (int e = 0; e < VE; ++e) most = finite_max(most, f[u][e]);
      }
      top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    }
    if (lane == 0) s_most[warp] = __uint_as_float(top);
    __syncthreads();
    if (!works || bad_page) continue;
    uint8_t *block = (is_k ? a.k_pages : a.v_pages) + ((head << b.page_shift) + (slot - in)) * D;
    float scale = scale_for(fmaxf(s_most[warp & ~1], s_most[warp | 1]));
    if (in > 0 && old >= scale) {
      scale = old;
    } else {
      if (in > 0) requantise(reinterpret_cast<unsigned *>(block), in * D / 4, lane + 32 * (warp & 1), 64, old / scale);
      if (lane == 0 && first_tok == 0) *scale_at = scale;
    }
    const float inv = 1.f / scale;
    uint8_t *to = block + (in + first_tok) * D;
    if (is_k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tok = kt + 32 / PV * u;
        if (tok >= mine) continue;
        store_e4m3<VE>(to + tok * D + kw * VE, f[u], inv);
        if constexpr (!IL) store_e4m3<VE>(to + tok * D + kw * VE + D / 2, f[U + u], inv);
      }
    } else {
#pragma unroll
      for (int u = 0; u < UV; ++u) {
        const int tok = vt + 32 / kOfRow * u;
        if (tok < mine) store_e4m3<VE>(to + tok * D + vw * VE, f[u], inv);
      }
    }
  }
}

template <typename T, bool IL, int D>
int launch_whole(const RopeQ8Args &r, const PagedArgs &b, int *d_status, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return KVS_ERR_LAUNCH;
  WholeArgs a{r, 0, 0, 0, 0};
  // Few rows: a thread block a row (those that do not begin a block of 16 leave at
  // once); else 16 rows, which begin one block of a prompt.
  const bool few = b.num_rows <= 4 * sms;
  a.r.group = few ? 1 : kScaleBlock;
  a.kv_parts = 2 * ((r.Hkv + kWHeads - 1) / kWHeads);
  const long long kv = ((long long)b.num_rows + a.r.group - 1) / a.r.group * a.kv_parts;
  a.q_tokens = few ? 1 : kWTokens;
  const long long groups = ((long long)b.num_rows + a.q_tokens - 1) / a.q_tokens;
  // a row of q is split until every SM has a block or a thread one unit left
  const int units = r.H * (IL ? D : D / 2) / (16 / (int)sizeof(T));
  const long long most = (units + kWThreads - 1) / kWThreads, want = (2 * sms + groups - 1) / groups;
  a.q_parts = (int)(want < 1 ? 1 : want < most ? want : most);
  if (kv + groups * a.q_parts > 0x7fffffffll) return KVS_ERR_UNSUPPORTED;
  a.kv_blocks = (int)kv;
  const cudaError_t e = launch_pdl(rope_q8_whole_kernel<T, IL, D>, dim3((unsigned)(kv + groups * a.q_parts)),
                                   dim3(kWThreads), 0, stream, a, b, d_status);
  return e == cudaSuccess ? KVS_OK : KVS_ERR_LAUNCH;
}

// ---- any head ----------------------------------------------------------------------
template <typename T, int VE, bool IL>
int launch_rope(RopeQ8Args a, const PagedArgs &b, int *d_status, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return KVS_ERR_LAUNCH;
  // Few rows: a thread block a row (those that do not begin a block of 16 leave at
  // once); else 16 rows, which begin one block of a prompt.
  a.group = b.num_rows <= 4 * sms ? 1 : kScaleBlock;
  const int groups = (int)(((long long)b.num_rows + a.group - 1) / a.group);
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
  if ((interleaved || a.rot == 0) && n % kMost == 0)  // (nothing that turns is either layout)
    return a.D == 64 ? launch_whole<T, true, 64>(a, b, d_status, stream)
                     : launch_whole<T, true, 128>(a, b, d_status, stream);
  if (a.rot == a.D)
    return a.D == 64 ? launch_whole<T, false, 64>(a, b, d_status, stream)
                     : launch_whole<T, false, 128>(a, b, d_status, stream);
  if (n % kMost == 0) return launch_rope<T, kMost, false>(a, b, d_status, stream);
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
