// How attention over the paged cache is split over thread blocks, and how the pieces are joined.
//
// A job is one KV head of one sequence (and, for long chunks, one tile of its rows); its keys are
// cut into units of a fixed number of tokens.  All units of all jobs, in order, are dealt out to
// the thread blocks in equal contiguous ranges, so a ragged batch and one long sequence load the
// GPU alike.  A job that one block has from its first unit to its last is finished there.  Of any
// other job every block leaves a piece (running maximum, sum, and unnormalised output of every
// row) in the scratch: in its slot 1 the job that begins in it, in its slot 0 the job that does
// not.  The block in which a job begins also leaves a note of it, and a second kernel joins the
// pieces of every noted job in their order, so results are the same in every run.
#pragma once

#include "cache.cuh"

namespace jolt {

struct CacheAttendArgs {
  CacheArgs c;
  BatchArgs a;
  int nq, G;                 // query heads, query heads per KV head
  float scale, cap, cap_inv; // cap 0: none; its reciprocal
  int window;                // 0: none
  int words;
  const float* slopes;
  const int* positions;
  const uint32_t* mask;
  const float* prefix_out;
  const float* prefix_lse;
  const void* q;
  int q_f16;                 // queries and outputs are fp16, else bf16
  long long q_row, q_head;
  void* out;
  long long o_row, o_head;
  bool q_vec, o_vec;         // rows and heads of q and of the output are 16-byte aligned
  // scratch
  int4* notes;               // [blocks]: {sequence, KV head, row tile or -1, blocks with a piece}
  float* pieces;             // [blocks][2][rows of a tile][D + 4]: D outputs, maximum, sum
};

namespace cs {
constexpr float LOG2E = 1.4426950408889634f;
constexpr float MASKED = -INFINITY;
// Weights are 2^(s - m + SHIFT): fp16 holds them normalised over 21 binary orders below the
// maximum, and the reference m may lag behind the true maximum by 2^LAG before the sums are
// rescaled (SHIFT + LAG = 15 keeps them below fp16's largest).
constexpr float SHIFT = 7.f, LAG = 8.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// start of block c's range when `total` units are dealt to `parts` blocks
__device__ __forceinline__ long long range_start(long long total, int parts, int c) { return total * c / parts; }
// number of blocks from c0 on whose ranges begin before unit `end`
__device__ __forceinline__ int pieces_until(long long total, int parts, int c0, long long end) {
  int c = (int)(end * parts / total);                  // range_start(c) <= end
  while (c > c0 && range_start(total, parts, c) >= end) --c;
  while (c + 1 < parts && range_start(total, parts, c + 1) < end) ++c;
  return c - c0 + 1;
}
}  // namespace cs

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

// s = cap tanh(s / cap).  tanh x = 1 - 2 / (e^(2x) + 1) is off by some 2^-23, so by 2^-17 of the score's
// unit at a cap of 64, far below the rounding of a weight to fp16.  A larger cap makes much of it: there,
// below |x| = 1/4, the series x - x^3/3 + 2x^5/15 - 17x^7/315 is used, whose next term is 62 x^9 / 2835,
// 2^-21.5 of x there.  Every call through the series: 120 us instead of 108 us (64 ragged sequences of up
// to 8192 tokens, one token each).
constexpr float MILD_CAP = 64.f;
__device__ __forceinline__ float cap_score(const CacheAttendArgs& A, float s) {
  const float e = cs::ex2(2.f * cs::LOG2E * A.cap_inv * s);
  const float far = A.cap - __fdividef(2.f * A.cap, e + 1.f);
  if (A.cap <= MILD_CAP) return far;
  const float x = s * A.cap_inv, x2 = x * x;
  const float near = fmaf(x2, fmaf(x2, fmaf(x2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f) * s;
  return fabsf(x) < 0.25f ? near : far;
}

__device__ __forceinline__ float ld_q(const CacheAttendArgs& A, long long at) {
  return A.q_f16 ? __half2float(reinterpret_cast<const __half*>(A.q)[at])
                 : __bfloat162float(reinterpret_cast<const bf16*>(A.q)[at]);
}

// Output element (row r, query head j, feature d): the joined sums o / l with reference maximum m
// (base 2), together with the row's prefix if there is one.  A row that saw nothing has l = 0.
__device__ __forceinline__ void store_out(const CacheAttendArgs& A, int D, int r, int j, int d, float o, float l,
                                          float m) {
  if (A.prefix_out) {
    const float lp = A.prefix_lse[(long long)r * A.nq + j] * cs::LOG2E, top = fmaxf(m, lp);
    const float f = l == 0.f ? 0.f : cs::ex2(m - top);
    const float g = lp == -INFINITY ? 0.f : cs::ex2(lp - top + cs::SHIFT);
    o *= f;
    l = fmaf(f, l, g);
    if (g != 0.f) o = fmaf(g, A.prefix_out[((long long)r * A.nq + j) * D + d], o);
  }
  const float y = l != 0.f ? o / l : 0.f;
  const long long at = r * A.o_row + j * A.o_head + d;
  if (A.q_f16) reinterpret_cast<__half*>(A.out)[at] = __float2half_rn(y);
  else reinterpret_cast<bf16*>(A.out)[at] = __float2bfloat16_rn(y);
}

// Join the pieces of the job that begins in block blockIdx.x.  Both kernels add a row's pieces in
// their order.

// Many rows, mostly of two or three pieces: a warp per row, no exchange between them.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) cache_join_rows_kernel(CacheAttendArgs A) {
  constexpr int REC = D + 4, V = D / 32;
  cs::wait_for_predecessor();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 note = A.notes[c0];
  const int b = note.x, h = note.y, tile = note.z, count = note.w;
  if (tile < 0) return;
  const int row0 = A.a.starts[b], R = (A.a.starts[b + 1] - row0) * A.G;
  const int mine = blockIdx.y * 8 + (threadIdx.x >> 5), row = tile * ROWS + mine;
  if (row >= R) return;
  const float* p = A.pieces + ((2ll * c0 + 1) * ROWS + mine) * REC;
  float o[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
#pragma unroll 2
  for (int k = 0; k < count; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(p + D);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[32 * i + lane];
    const float top = fmaxf(m, ml.x);
    const float f = l == 0.f ? 0.f : cs::ex2(m - top), g = ml.y == 0.f ? 0.f : cs::ex2(ml.x - top);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(g, v[i], f * o[i]);
    l = fmaf(g, ml.y, f * l);
    m = top;
    p += (k == 0 ? 1 : 2) * (long long)ROWS * REC;   // the next block's slot 0
  }
#pragma unroll
  for (int i = 0; i < V; ++i) store_out(A, D, row0 + row / A.G, h * A.G + row % A.G, 32 * i + lane, o[i], l, m);
}

// Few rows of few jobs, which may have many pieces each (one of every block where there is one job): a CTA
// takes 512 / D rows, a thread one feature; the pieces' maxima and sums first, then the weighted sums, eight
// loads under way.
constexpr int JOIN_MOST = 592;          // blocks of the launch whose pieces are joined
template <int D, int ROWS>
__global__ void __launch_bounds__(512) cache_join_kernel(CacheAttendArgs A) {
  constexpr int REC = D + 4, PER = 512 / D;
  __shared__ float2 ml[PER][JOIN_MOST];   // maximum and sum of every piece
  cs::wait_for_predecessor();
  const int c0 = blockIdx.x, slot = threadIdx.x / D, d = threadIdx.x % D;
  const int4 note = A.notes[c0];
  const int b = note.x, h = note.y, tile = note.z, count = note.w;
  if (tile < 0) return;
  const int row0 = A.a.starts[b], R = (A.a.starts[b + 1] - row0) * A.G;
  const int mine = blockIdx.y * PER + slot, row = tile * ROWS + mine;
  // record of the row in the k-th piece
  auto rec = [&](int k) { return A.pieces + ((2ll * (c0 + k) + (k == 0 ? 1 : 0)) * ROWS + mine) * REC; };
  if (row < R)
    for (int k = d; k < count; k += D) ml[slot][k] = *reinterpret_cast<const float2*>(rec(k) + D);
  __syncthreads();
  if (row >= R) return;
  float top = -INFINITY, sum = 0.f, y = 0.f;
#pragma unroll 8
  for (int k = 0; k < count; ++k) top = fmaxf(top, ml[slot][k].x);
#pragma unroll 8
  for (int k = 0; k < count; ++k) {
    const float2 x = ml[slot][k];
    const float f = x.y == 0.f ? 0.f : cs::ex2(x.x - top);
    y = fmaf(f, rec(k)[d], y);
    sum = fmaf(f, x.y, sum);
  }
  store_out(A, D, row0 + row / A.G, h * A.G + row % A.G, d, y, sum, top);
}

}  // namespace jolt
