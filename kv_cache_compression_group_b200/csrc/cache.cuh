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

namespace cs {
// Programmatic launch: the kernel before this one in its stream has ended and its writes are seen.
// (A kernel launched so may start while that one ends; the waiting is all that keeps them apart.)
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// the next kernel's blocks may be brought up from here on, to wait for this one's end
__device__ __forceinline__ void let_successor_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace cs

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

// Sequence that row r belongs to (the last one whose rows start at or before it), or -1; the whole
// warp asks for one row and narrows the range 32-fold with every load.  With starts that are not
// ascending it still ends, and seq_of refuses what it finds.
__device__ __forceinline__ int seq_of_row(const BatchArgs& a, int r, int lane) {
  int lo = 0, n = a.B + 1;               // the last start <= r is one of starts[lo .. lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < lo + n && a.starts[at] <= r);
    if (le == 0u) return -1;
    const int last = 31 - __clz(le);
    n = min(step, n - last * step);
    lo += last * step;
    if (step == 1) break;
  }
  return lo < a.B ? lo : -1;
}

// page of position t of sequence b, or -1 (and the status bit) when the table names none
__device__ __forceinline__ int page_at(const BatchArgs& a, const CacheArgs& c, int b, int t) {
  const int p = a.table[(long long)b * a.max_pages + (t >> c.page_shift)];
  if ((unsigned)p < (unsigned)c.n_pages) return p;
  raise_status(a.status, DEV_ERR_BATCH);
  return -1;
}

// row of head h at position t inside its page (a pool has fewer than 2^31 rows; their bytes may pass
// 32 bits: byte offsets are formed as 32 x 32 -> 64 bit products)
__device__ __forceinline__ uint32_t row_index(const CacheArgs& c, int page, int h, int t) {
  return (((uint32_t)page * c.H + h) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}
__device__ __forceinline__ unsigned long long row_bytes(uint32_t row, uint32_t bytes) {
  return (unsigned long long)row * bytes;
}

__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(float v, bf16& x) { x = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& x) { x = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, float& x) { x = v; }

// N consecutive elements as they lie in memory, 16 bytes at a time where they are aligned
template <int N, typename T>
union Raw16 {
  uint4 w[N * sizeof(T) / 16];
  T e[N];
  __device__ __forceinline__ Raw16() {}
};
template <int N, typename T>
__device__ __forceinline__ void load_raw(const T* p, bool vec, Raw16<N, T>& u) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) u.w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) u.e[i] = p[i];
  }
}
template <int N, typename T>
__device__ __forceinline__ void load_n(const T* p, bool vec, float (&v)[N]) {
  Raw16<N, T> u;
  load_raw(p, vec, u);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_f32(u.e[i]);
}
template <int N, typename T>
__device__ __forceinline__ void store_n(T* p, bool vec, const float (&v)[N]) {
  Raw16<N, T> u;
#pragma unroll
  for (int i = 0; i < N; ++i) from_f32(v[i], u.e[i]);
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = u.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = u.e[i];
  }
}

// dense rows of K (0) and V (1); strides in elements
template <typename T>
struct RowsArgs {
  T* x[2];
  long long row[2], head[2];
  bool vec[2];
  int per_warp;            // rows of a warp
};

// Both kernels: a thread has a block of 16 features, a warp one row of 32 / (D / 16) neighbouring
// heads at a time and per_warp rows one after the other, so that everything about the row (its
// sequence, position and page) is found once per warp.  blockIdx.y = group of heads, blockIdx.z = 0
// for K, 1 for V.
constexpr int ROW_WARPS = 8;
constexpr int READ_AHEAD = 4;   // rows of which a warp has its loads under way at once

// Walks rows of the batch; all lanes of a warp together.
struct RowCursor {
  int row0 = 0, end = -1;     // rows of the sequence in hand: [row0, end)
  int b = -1, t = 0, page = -1;
  bool ok = false;            // the sequence is one
  // to row r (from r - 1, or anywhere)
  __device__ __forceinline__ void to(const CacheArgs& c, const BatchArgs& a, int r, int lane) {
    bool look = true;
    if (r >= row0 && r < end) {
      ++t;
      look = (t & ((1 << c.page_shift) - 1)) == 0;
    } else {
      b = seq_of_row(a, r, lane);
      ok = false;
      row0 = r;
      end = r + 1;
      if (b >= 0) {
        int n, len;
        ok = seq_of(a, c.page_shift, b, row0, n, len) && r >= row0 && r < row0 + n;
        if (ok) {
          end = row0 + n;
          t = len - n + (r - row0);
        } else {
          row0 = r;
        }
      }
    }
    if (ok && look) page = page_at(a, c, b, t);
  }
};

// minimum and maximum of 16 values, NaN if one is
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ void block_range(const Raw16<16, float>& u, float& mn, float& mx) {
  mn = mx = u.e[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    mn = min_nan(mn, u.e[i]);
    mx = fmaxf(mx, u.e[i]);
  }
}
__device__ __forceinline__ void block_range(const Raw16<16, bf16>& u, float& mn, float& mx) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(u.e);
  __nv_bfloat162 a = p[0], b = p[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    a = __hmin2_nan(a, p[i]);
    b = __hmax2(b, p[i]);
  }
  mn = min_nan(__low2float(a), __high2float(a));
  mx = fmaxf(__low2float(b), __high2float(b));
}
__device__ __forceinline__ void block_range(const Raw16<16, __half>& u, float& mn, float& mx) {
  const __half2* p = reinterpret_cast<const __half2*>(u.e);
  __half2 a = p[0], b = p[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    a = __hmin2_nan(a, p[i]);
    b = __hmax2(b, p[i]);
  }
  mn = min_nan(__low2float(a), __high2float(a));
  mx = fmaxf(__low2float(b), __high2float(b));
}

// Quantise one block and store it; v is what its values count as (finite, within fp16's range).
// The quotient (x - lo) / step is formed in fp32 with the reciprocal of the step; its error is below
// (levels + 1) 2^-22 (the difference, the reciprocal and the product are each rounded by at most
// 2^-24 of themselves, 3 levels 2^-24 together), so only a quotient closer than that to a tie can round otherwise than the
// definition's.  Those few are decided by comparing x - lo with the tie itself in fp64, where
// tie * step is exact.
template <int BITS>
__device__ __forceinline__ void encode_block(const float (&v)[16], float mn, float mx, unsigned char* codes,
                                             __half2* scale) {
  constexpr float LEV = (float)((1 << BITS) - 1), NEAR = (LEV + 1.f) * 0x1p-22f;
  const float lo = __half2float(__float2half_rd(mn)) + 0.f;   // +0 for a minimum of -0
  const float step = quant_step_cvt(mx, lo, BITS);
  const float inv = step > 0.f ? __frcp_rn(step) : 0.f;
  float code[16];
  const float2 lo2 = make_float2(-lo, -lo), inv2 = make_float2(inv, inv), minus = make_float2(-1.f, -1.f);
  const float2 up = make_float2(kRoundShift, kRoundShift), down = make_float2(-kRoundShift, -kRoundShift);
#pragma unroll
  for (int q = 0; q < 16; q += 4) {
    float off = 0.f;
#pragma unroll
    for (int i = q; i < q + 4; i += 2) {
      // integer part onto the mantissa of 1.5 2^23, and how far from it the quotient is
      const float2 t = __fmul2_rn(__fadd2_rn(make_float2(v[i], v[i + 1]), lo2), inv2);
      const float2 k = __fadd2_rn(__fadd2_rn(t, up), down);
      const float2 e = __ffma2_rn(k, minus, t);
      off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
      code[i] = k.x;
      code[i + 1] = k.y;
    }
    if (off > 0.5f - NEAR) {
#pragma unroll
      for (int i = q; i < q + 4; ++i) {
        const float below = floorf((v[i] - lo) * inv);
        const double d = (double)v[i] - (double)lo, tie = ((double)below + 0.5) * (double)step;
        if (fabsf((v[i] - lo) * inv - below - 0.5f) <= NEAR)
          code[i] = d > tie ? below + 1.f : d < tie ? below : 2.f * rintf(0.5f * (below + 0.5f));
      }
    }
  }
  // 16 bits of codes as the digits of a number, taken off the mantissa of 2^23
  constexpr int DIG = 16 / BITS;
  constexpr float BASE = (float)(1 << BITS);
  uint32_t h[BITS];
#pragma unroll
  for (int k = 0; k < BITS; ++k) {
    float x = code[k * DIG + DIG - 1];
#pragma unroll
    for (int i = DIG - 2; i >= 0; --i) x = fmaf(x, BASE, code[k * DIG + i]);
    h[k] = __float_as_uint(x + 8388608.f);
  }
  uint32_t w[BITS / 2];
#pragma unroll
  for (int k = 0; k < BITS / 2; ++k) w[k] = __byte_perm(h[2 * k], h[2 * k + 1], 0x5410);
  if constexpr (BITS == 2) *reinterpret_cast<uint32_t*>(codes) = w[0];
  else if constexpr (BITS == 4) *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
  *scale = __floats2half2_rn(lo, step);
}

// Quantise rows into their pages.  65536 rows of 8 heads of 128 bf16 features, K at 8 and V at 4 bits: 268 MB in
// and 134 MB out, 61 us at the copy rate, take 107 us; the instructions bound it (issue 75 %, ALU 62 %).
// 5620 fp32 rows of 8 heads of 64 features at 2 bits, 23 MB in and 3 MB out: 14 us (issue 42 %).
template <typename T, int D>
__global__ void __launch_bounds__(ROW_WARPS * 32, sizeof(T) == 4 ? 3 : 4) cache_write_kernel(CacheArgs c, BatchArgs a, RowsArgs<const T> x) {
  constexpr int LANES = D / 16;                       // of a head
  const int kv = blockIdx.z, lane = threadIdx.x & 31, blk = lane % LANES;
  const int h = blockIdx.y * (32 / LANES) + lane / LANES;
  const int r0 = (blockIdx.x * ROW_WARPS + (threadIdx.x >> 5)) * x.per_warp, r1 = min(a.rows, r0 + x.per_warp);
  // (chosen, not indexed: an index known only at run time would move the parameters to local memory)
  const bool on = h < c.H, vec = kv ? x.vec[1] : x.vec[0];
  const int bits = kv ? c.bits[1] : c.bits[0];
  const long long pitch = kv ? x.row[1] : x.row[0];
  unsigned char* const pool = kv ? c.codes[1] : c.codes[0];
  __half2* const scales = kv ? c.scales[1] : c.scales[0];
  const T* src = (kv ? x.x[1] : x.x[0]) + h * (kv ? x.head[1] : x.head[0]) + blk * 16;
  RowCursor at;
  Raw16<16, T> u, next;
  cs::wait_for_predecessor();
  cs::let_successor_start();
  if (r0 < r1 && on) load_raw(src + r0 * pitch, vec, next);
  for (int r = r0; r < r1; ++r) {
    u = next;
    if (r + 1 < r1 && on) load_raw(src + (r + 1) * pitch, vec, next);
    at.to(c, a, r, lane);
    if (!at.ok || at.page < 0 || !on) continue;
    float mn, mx, v[16];
    block_range(u, mn, mx);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = to_f32(u.e[i]);
    if (!(mn >= -kFp16Max) || mx > kFp16Max) {        // a NaN is the minimum
      raise_status(a.status, DEV_ERR_NONFINITE);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] != v[i] ? 0.f : fminf(fmaxf(v[i], -kFp16Max), kFp16Max);
      mn = mx = v[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) {
        mn = fminf(mn, v[i]);
        mx = fmaxf(mx, v[i]);
      }
    }
    const long long block = (long long)row_index(c, at.page, h, at.t) * LANES + blk;
    unsigned char* codes = pool + block * (2 * bits);
    if (bits == 4) encode_block<4>(v, mn, mx, codes, scales + block);
    else if (bits == 8) encode_block<8>(v, mn, mx, codes, scales + block);
    else encode_block<2>(v, mn, mx, codes, scales + block);
  }
}

// Read stored rows back: lo + code * step in fp32, rounded once.  40 heads of 128 features at 4 bits to fp16, 104 MB
// in and 277 MB out, take 73 us (58 at the copy rate).  To fp32 (8 bits, 85 MB in, 268 MB out) 85 us
// instead of 54 with issue at 22 %: a lane's 16-byte stores of its own block touch twice the sectors they fill.
template <typename T, int D>
__global__ void __launch_bounds__(ROW_WARPS * 32) cache_read_kernel(CacheArgs c, BatchArgs a, RowsArgs<T> x) {
  constexpr int LANES = D / 16;
  const int kv = blockIdx.z, lane = threadIdx.x & 31, blk = lane % LANES;
  const int h = blockIdx.y * (32 / LANES) + lane / LANES;
  const int r0 = (blockIdx.x * ROW_WARPS + (threadIdx.x >> 5)) * x.per_warp, r1 = min(a.rows, r0 + x.per_warp);
  const bool on = h < c.H, vec = kv ? x.vec[1] : x.vec[0];
  const int bits = kv ? c.bits[1] : c.bits[0];
  const long long pitch = kv ? x.row[1] : x.row[0];
  const unsigned char* const pool = kv ? c.codes[1] : c.codes[0];
  const __half2* const scales = kv ? c.scales[1] : c.scales[0];
  T* dst = (kv ? x.x[1] : x.x[0]) + h * (kv ? x.head[1] : x.head[0]) + blk * 16;
  RowCursor at;
  cs::wait_for_predecessor();
  cs::let_successor_start();
  for (int r = r0; r < r1; r += READ_AHEAD) {
    // the loads of several rows first
    uint4 q[READ_AHEAD];
    __half2 sc[READ_AHEAD];
    unsigned write = 0;
#pragma unroll
    for (int k = 0; k < READ_AHEAD; ++k) {
      q[k] = make_uint4(0u, 0u, 0u, 0u);
      sc[k] = __floats2half2_rn(0.f, 0.f);
      if (r + k >= r1) continue;
      at.to(c, a, r + k, lane);
      if (!at.ok || !on) continue;
      write |= 1u << k;
      if (at.page < 0) continue;
      const long long block = (long long)row_index(c, at.page, h, at.t) * LANES + blk;
      const unsigned char* src = pool + block * (2 * bits);
      if (bits == 4) *reinterpret_cast<uint2*>(&q[k]) = *reinterpret_cast<const uint2*>(src);
      else if (bits == 8) q[k] = *reinterpret_cast<const uint4*>(src);
      else q[k].x = *reinterpret_cast<const uint32_t*>(src);
      sc[k] = scales[block];
    }
#pragma unroll
    for (int k = 0; k < READ_AHEAD; ++k) {
      if (!((write >> k) & 1u)) continue;
      const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
      const float2 s2 = __half22float2(sc[k]);
      float v[16];
      // a code under the exponent of 2^23, made exact by one subtraction
      if (bits == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float((w[i / 8] >> (4 * (i % 8)) & 0xfu) | 0x4B000000u);
      } else if (bits == 8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7650 + (i & 3)));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float((w[0] >> (2 * i) & 0x3u) | 0x4B000000u);
      }
      const float2 lo2 = make_float2(s2.x, s2.x), step2 = make_float2(s2.y, s2.y);
      const float2 down = make_float2(-8388608.f, -8388608.f);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float2 y = __ffma2_rn(__fadd2_rn(make_float2(v[i], v[i + 1]), down), step2, lo2);
        v[i] = y.x;
        v[i + 1] = y.y;
      }
      store_n(dst + (r + k) * pitch, vec, v);
    }
  }
}

}  // namespace jolt
