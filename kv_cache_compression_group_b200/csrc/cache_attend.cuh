// Attention over the paged cache of block-quantised rows.
//
// For a new row at position p_q of a sequence, over the keys it sees,
//   s_t = cap tanh(scale (q . k_t) / cap) - slope (p_q - p_t),   o = sum_t softmax(s)_t v_t,
// with k_t, v_t = lo + code * step taken from the stored blocks.
#pragma once

#include "cache.cuh"

namespace jolt {

struct CacheAttendArgs {
  CacheArgs c;
  BatchArgs a;
  int nq, G;                 // query heads, query heads per KV head
  float scale, cap;          // cap 0: none
  int window;                // 0: none
  int words;
  const float* slopes;
  const int* positions;
  const uint32_t* mask;
  const float* prefix_out;
  const float* prefix_lse;
  const void* q;
  long long q_row, q_head;
  void* out;
  long long o_row, o_head;
};

// position of key t of a sequence whose new rows start at position `old` and row `row0`
__device__ __forceinline__ int key_position(const CacheAttendArgs& A, int row0, int old, int t) {
  return (A.positions && t >= old) ? A.positions[row0 + t - old] : t;
}

// whether row i (of n, at position pq) sees key t (at position pk)
__device__ __forceinline__ bool row_sees(const CacheAttendArgs& A, int row0, int old, int n, int i, int pq, int t,
                                         int pk) {
  if (A.window && (pq - pk >= A.window || t <= old - A.window)) return false;
  const int j = t - old;
  if (j < 0) return true;
  if (j >= n) return false;
  if (!A.mask) return j <= i;
  return (A.mask[(long long)(row0 + i) * A.words + (j >> 5)] >> (j & 31)) & 1u;
}

__device__ __forceinline__ float cache_value(const CacheArgs& c, int kv, long long row, int d) {
  const int b = c.bits[kv], nb = c.D / pc::BLK, bit = d * b;
  const long long at = row * nb;
  const uint32_t byte = c.codes[kv][at * (2 * b) + (bit >> 3)];
  const float2 s = __half22float2(c.scales[kv][at + d / pc::BLK]);
  return fmaf((float)((byte >> (bit & 7)) & ((1u << b) - 1u)), s.y, s.x);
}

// One CTA of D threads per (new row, query head): tiles of D keys, one key per thread for the
// scores, one feature per thread for the values.
template <typename T, int D>
__global__ void __launch_bounds__(D) cache_attend_kernel(CacheAttendArgs A) {
  __shared__ float qs[D], ps[D], red[D / 32];
  __shared__ long long rowof[D];
  const int r = blockIdx.x, j = blockIdx.y, h = j / A.G, tid = threadIdx.x;
  const int b = seq_of_row(A.a, r);
  int row0, n, len;
  if (b < 0 || !seq_of(A.a, A.c.page_shift, b, row0, n, len)) return;
  const int i = r - row0, old = len - n;
  qs[tid] = to_f32(reinterpret_cast<const T*>(A.q)[r * A.q_row + j * A.q_head + tid]);
  const int pq = A.positions ? A.positions[r] : old + i;
  const float slope = A.slopes ? A.slopes[j] : 0.f;
  float m = -INFINITY, l = 0.f, o = 0.f;
  const int first = A.window ? max(0, old - A.window + 1) : 0;
  __syncthreads();
  for (int t0 = first; t0 < len; t0 += D) {
    const int t = t0 + tid;
    float s = -INFINITY;
    rowof[tid] = -1;
    if (t < len) {
      const int page = page_at(A.a, A.c, b, t), pk = key_position(A, row0, old, t);
      if (page >= 0 && row_sees(A, row0, old, n, i, pq, t, pk)) {
        const long long row = row_index(A.c, page, h, t);
        rowof[tid] = row;
        s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(qs[d], cache_value(A.c, 0, row, d), s);
        s *= A.scale;
        if (A.cap > 0.f) s = A.cap * tanhf(s / A.cap);
        s -= slope * (float)(pq - pk);
      }
    }
    float mx = s;
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    for (int k = 0; k < D / 32; ++k) mx = fmaxf(mx, red[k]);
    const float mn = fmaxf(m, mx), f = m == -INFINITY ? 0.f : expf(m - mn);
    ps[tid] = s == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    __syncthreads();
    l *= f;
    o *= f;
    for (int k = 0; k < D; ++k)
      if (rowof[k] >= 0) {
        l += ps[k];
        o = fmaf(ps[k], cache_value(A.c, 1, rowof[k], tid), o);
      }
    __syncthreads();
  }
  if (A.prefix_out) {
    const float lp = A.prefix_lse[(long long)r * A.nq + j], mn = fmaxf(m, lp);
    const float f = m == -INFINITY ? 0.f : expf(m - mn), g = lp == -INFINITY ? 0.f : expf(lp - mn);
    o = f * o;
    if (g > 0.f) o = fmaf(g, A.prefix_out[((long long)r * A.nq + j) * D + tid], o);
    l = fmaf(f, l, g);
  }
  from_f32(l != 0.f ? o / l : 0.f, reinterpret_cast<T*>(A.out)[r * A.o_row + j * A.o_head + tid]);
}

}  // namespace jolt
