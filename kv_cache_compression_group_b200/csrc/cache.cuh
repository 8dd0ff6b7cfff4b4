// Paged cache of block-quantised rows: how a batch's rows find their pages, and the kernels that
// write rows and read them back.  The stored form is the residual quantiser's: per 16 consecutive
// features lo = fp16_rd(min), step = fp16_ru((max - lo) / (2^b - 1)), code = rhe((x - lo) / step).
#pragma once

#include "common.cuh"
#include "fp16_exact.cuh"

namespace jolt {
namespace pc {
constexpr int BLK = 16;   // features per (lo, step) pair
}

// one layer's pool; index 0 = K, 1 = V
struct CacheArgs {
  unsigned char* codes[2];
  __half2* scales[2];
  int bits[2];
  int H, D, n_pages;
  int page_shift;          // log2(page_size)
};

struct BatchArgs {
  const int* table;        // [B][max_pages]
  const int* lens;         // [B]
  const int* starts;       // [B + 1]
  int B, max_pages, max_new, rows;
  uint32_t* status;
};

// sequence b of the batch: rows [row0, row0 + n), positions [len - n, len); false (and the status
// bit) when the entries do not describe one
__device__ __forceinline__ bool seq_of(const BatchArgs& a, int page_shift, int b, int& row0, int& n, int& len) {
  row0 = a.starts[b];
  const long long cnt = (long long)a.starts[b + 1] - row0;
  n = (int)cnt;
  len = a.lens[b];
  const bool ok = cnt >= 0 && cnt <= a.max_new && row0 >= 0 && row0 + cnt <= a.rows && len >= cnt &&
                  len <= ((long long)a.max_pages << page_shift);
  if (!ok) raise_status(a.status, DEV_ERR_BATCH);
  return ok;
}

// sequence that row r belongs to (the last one whose rows start at or before it), or -1.  With
// starts that are not ascending it still ends, and seq_of refuses what it finds.
__device__ __forceinline__ int seq_of_row(const BatchArgs& a, int r) {
  int lo = 0, hi = a.B;   // starts[lo] <= r < starts[hi]
  if (r < a.starts[0] || r >= a.starts[a.B]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.starts[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// page of position t of sequence b, or -1 (and the status bit) when the table names none
__device__ __forceinline__ int page_at(const BatchArgs& a, const CacheArgs& c, int b, int t) {
  const int p = a.table[(long long)b * a.max_pages + (t >> c.page_shift)];
  if ((unsigned)p < (unsigned)c.n_pages) return p;
  raise_status(a.status, DEV_ERR_BATCH);
  return -1;
}

// row of head h at position t inside its page: index of its first block
__device__ __forceinline__ long long row_index(const CacheArgs& c, int page, int h, int t) {
  return (((long long)page * c.H + h) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}

template <typename T>
struct Vec16;   // 16 consecutive elements, loaded or stored 16 bytes at a time where aligned

__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(float v, bf16& x) { x = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& x) { x = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, float& x) { x = v; }

template <typename T>
__device__ __forceinline__ void load16(const T* p, bool vec, float (&v)[16]) {
  union {
    uint4 w[sizeof(T)];
    T e[16];
  } u;
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) u.w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) u.e[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = to_f32(u.e[i]);
}

template <typename T>
__device__ __forceinline__ void store16(T* p, bool vec, const float (&v)[16]) {
  union {
    uint4 w[sizeof(T)];
    T e[16];
  } u;
#pragma unroll
  for (int i = 0; i < 16; ++i) from_f32(v[i], u.e[i]);
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) reinterpret_cast<uint4*>(p)[i] = u.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = u.e[i];
  }
}

// dense rows of K (0) and V (1); strides in elements
template <typename T>
struct RowsArgs {
  T* x[2];
  long long row[2], head[2];
  bool vec[2];
};

// Codes of one block of 16 values, packed into BITS / 2 words.  The quotient is formed in fp32
// with the reciprocal of the step; its error is below (levels + 1) 2^-22 (three roundings of at
// most levels, each 2^-24 relative), so only a quotient closer than that to a tie can round
// otherwise than the definition, and those are decided in fp64 like the definition's.
template <int BITS>
__device__ __forceinline__ void encode_block(const float (&v)[16], float lo, float step, uint32_t (&w)[BITS / 2]) {
  constexpr float LEV = (float)((1 << BITS) - 1);
  constexpr float EDGE = 0.5f - (LEV + 1.f) * 0x1p-22f;
#pragma unroll
  for (int i = 0; i < BITS / 2; ++i) w[i] = 0u;
  if (!(step > 0.f)) return;
  const float inv = 1.0f / step;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float t = (v[i] - lo) * inv;
    float c = rintf(t);
    if (fabsf(t - c) > EDGE) c = (float)rint(((double)v[i] - (double)lo) / (double)step);
    c = fminf(fmaxf(c, 0.f), LEV);
    w[i * BITS / 32] |= (uint32_t)c << (i * BITS % 32);
  }
}

template <int BITS>
__device__ __forceinline__ void write_block(unsigned char* codes, const float (&v)[16], float lo, float step) {
  uint32_t w[BITS / 2];
  encode_block<BITS>(v, lo, step, w);
  if constexpr (BITS == 2) *reinterpret_cast<uint32_t*>(codes) = w[0];
  else if constexpr (BITS == 4) *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread per block of 16 features; blockIdx.y = 0 for K, 1 for V.
template <typename T>
__global__ void __launch_bounds__(256) cache_write_kernel(CacheArgs c, BatchArgs a, RowsArgs<const T> x) {
  const int kv = blockIdx.y, nb = c.D / pc::BLK;
  const long long idx = blockIdx.x * 256ll + threadIdx.x;
  const int blk = (int)(idx % nb), h = (int)(idx / nb % c.H);
  const long long r = idx / nb / c.H;
  if (r >= a.rows) return;
  const int b = seq_of_row(a, (int)r);
  int row0, n, len;
  if (b < 0 || !seq_of(a, c.page_shift, b, row0, n, len)) return;
  const int t = len - n + ((int)r - row0), page = page_at(a, c, b, t);
  if (page < 0) return;
  float v[16];
  load16(x.x[kv] + r * x.row[kv] + h * x.head[kv] + blk * pc::BLK, x.vec[kv], v);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    bad |= !(fabsf(v[i]) <= kFp16Max);
    v[i] = v[i] != v[i] ? 0.f : fminf(fmaxf(v[i], -kFp16Max), kFp16Max);
  }
  if (bad) raise_status(a.status, DEV_ERR_NONFINITE);
  float mn = v[0], mx = v[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    mn = fminf(mn, v[i]);
    mx = fmaxf(mx, v[i]);
  }
  const int bits = c.bits[kv];
  const float lo = rd16(mn) + 0.f;   // +0 for a minimum of -0
  const float step = quant_step_cvt(mx, lo, bits);
  const long long at = row_index(c, page, h, t) * nb + blk;
  unsigned char* codes = c.codes[kv] + at * (2 * bits);
  if (bits == 2) write_block<2>(codes, v, lo, step);
  else if (bits == 4) write_block<4>(codes, v, lo, step);
  else write_block<8>(codes, v, lo, step);
  c.scales[kv][at] = __floats2half2_rn(lo, step);
}

// One thread per block of 16 features; blockIdx.y = 0 for K, 1 for V.
template <typename T>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheArgs c, BatchArgs a, RowsArgs<T> x) {
  const int kv = blockIdx.y, nb = c.D / pc::BLK;
  const long long idx = blockIdx.x * 256ll + threadIdx.x;
  const int blk = (int)(idx % nb), h = (int)(idx / nb % c.H);
  const long long r = idx / nb / c.H;
  if (r >= a.rows) return;
  const int b = seq_of_row(a, (int)r);
  int row0, n, len;
  if (b < 0 || !seq_of(a, c.page_shift, b, row0, n, len)) return;
  const int t = len - n + ((int)r - row0), page = page_at(a, c, b, t), bits = c.bits[kv];
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  float lo = 0.f, step = 0.f;
  if (page >= 0) {
    const long long at = row_index(c, page, h, t) * nb + blk;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(c.codes[kv] + at * (2 * bits));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < bits / 2) w[i] = src[i];
    const float2 s = __half22float2(c.scales[kv][at]);
    lo = s.x;
    step = s.y;
  }
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = fmaf((float)unpack_code(w, i, bits), step, lo);
  store16(x.x[kv] + r * x.row[kv] + h * x.head[kv] + blk * pc::BLK, x.vec[kv], v);
}

}  // namespace jolt
