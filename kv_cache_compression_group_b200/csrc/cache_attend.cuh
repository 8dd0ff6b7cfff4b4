// Attention of a few rows per KV head (more than the codes' kernel takes, up to 32: small trees) over the
// paged cache.
//
// For a new row at position p_q of a sequence, over the keys it sees,
//   s_t = cap tanh(scale (q . k_t) / cap) - slope (p_q - p_t),   o = sum_t softmax(s)_t v_t,
// with k_t, v_t = lo + code * step taken from the stored blocks.
//
// The stored bytes are its floor (96 bytes per token and head of K or V at 4 bits and D = 128); what bounds it is
// latency, with the instructions that turn codes into operands: 32 rows over 4 sequences of up to 16384 tokens (8 KV
// heads, D = 64, 8 bits) take 60 us where the bytes take 10, with four n-tiles 247 registers (up to 255, and
// some spills, at D = 128), so 8 warps on an SM, and issue at 43 %.  So codes go from global memory to shared
// memory untouched (cp.async, a ring of 16-token stages per warp, no block-wide barrier in the
// loop), become fp16 pairs in registers, and enter m16n8k16 products as the wide operand:
//   S^T [16 tokens x 8 NT rows] = K [16 x D] Q^T,   O^T [D x 8 NT rows] += V^T [D x 16] P^T.
// The query rows of a KV head are the narrow side, so four heads cost one n-tile, not a padded
// 16- or 128-row tile; that is why this path is mma.sync and not tcgen05, whose smallest tile would
// be mostly padding here.  K and V rows keep the packed order of their features:
//   * a K fragment's features may be any 16, as long as Q^T's are the same: a thread takes the
//     packed words of D / 4 consecutive features, and Q^T is laid out to match once per job;
//   * V's fragment pairs two tokens of one feature.  ldmatrix.trans transposes 16-bit units, here
//     16 / bits codes of one token, so one shift and mask of its result gives the pair.
// A value is fp16(lo / 2 + step * (code / 2)): one rounding, of halves so that the top of fp16's range does
// not overflow; the factor returns in fp32.  The half is the code's, which is exact (half a step would lose
// a bit below 2^-13, times a code of up to 255: 6e-3 of 8-bit values of 1e-3, their quantiser 4e-3); only lo / 2 may
// lose its last bit, below 2^-13, so a value is off by at most 2^-11 of itself and 2^-23.
#pragma once

#include "cache_split.cuh"

namespace jolt {
namespace ca {
constexpr int WARPS = 4;
constexpr int TOK = 16;                  // tokens of a stage
constexpr int UNIT = WARPS * TOK;        // tokens of a unit of work

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm2t(uint32_t& r0, uint32_t& r1, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2u(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 u2h(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// The exponent of 512 in both halves, in a register the compiler cannot see through: with it, mask
// and exponent go in by one three-input logic operation (as two immediates they would take two).
__device__ __forceinline__ uint32_t magic512() {
  uint32_t x;
  asm volatile("mov.b32 %0, 0x60006000;" : "=r"(x));
  return x;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t magic) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(a), "r"(mask), "r"(magic));
  return y;
}

// Half of codes s of the two 16-bit halves of w as an fp16 pair: the code under the exponent of 512,
// where fp16's step is 1/2 (or there with the code 4^k times too large, where it is not shifted down),
// made exact by one subtraction (or fused multiply-add).
template <int BITS>
__device__ __forceinline__ __half2 half_code_pair(uint32_t w, int s, uint32_t magic) {
  const __half2 k512 = __float2half2_rn(-512.f);
  if constexpr (BITS == 2) {
    const uint32_t v = s < 4 ? w : w >> 8;
    const int p = 2 * (s & 3);
    const uint32_t x = and_or(v, 0x00030003u << p, magic);
    if (p == 0) return __hadd2(u2h(x), k512);
    const float f = 1.f / (float)(1 << p);
    return __hfma2(u2h(x), __float2half2_rn(f), __float2half2_rn(-512.f * f));
  } else if constexpr (BITS == 4) {
    const uint32_t v = s < 2 ? w : w >> 8;
    if ((s & 1) == 0) return __hadd2(u2h(and_or(v, 0x000f000fu, magic)), k512);
    return __hfma2(u2h(and_or(v, 0x00f000f0u, magic)), __float2half2_rn(0.0625f), __float2half2_rn(-32.f));
  } else {
    return __hadd2(u2h(__byte_perm(w, magic, s == 0 ? 0x5250 : 0x5351)), k512);
  }
}

// where 16-byte chunk ch of row `row` of a stage lies when rows have CH chunks: eight rows' equal
// chunks fall into eight different bank groups
template <int CH>
__device__ __forceinline__ int swizzled(int row, int ch) {
  return (row * CH + (CH == 1 ? ch : ch ^ ((row / (8 / CH)) & (CH - 1)))) * 16;
}

// Copy a stage's rows (16 x CH chunks, contiguous in the page) to shared memory.  dst0: where this
// lane's first chunk goes, swizzled<CH>(lane / CH, lane % CH); its next ones follow 512 bytes apart
// (with CH = 8 every other one in the other half of its row).
template <int CH>
__device__ __forceinline__ void copy_rows(uint32_t stage, uint32_t dst0, const unsigned char* src, int lane) {
#pragma unroll
  for (int i = 0; i < (CH + 1) / 2; ++i)
    if (CH > 1 || lane < 16) cp16(stage + (CH == 8 && (i & 1) ? dst0 ^ 64u : dst0) + 512 * i, src + 512 * i);
}

// S^T += K Q^T for 16 tokens; q(m, nt) gives B registers of product m and n-tile nt
template <int BITS, int D, int NT, typename QF>
__device__ __forceinline__ void scores(float (&s)[NT][4], uint32_t kc, uint32_t ksc, int lane, uint32_t magic, QF&& q) {
  constexpr int CH = D * BITS / 128, W = D / 4 * BITS / 32;   // chunks per row, words per thread and token
  const int g = lane >> 2, c = lane & 3;
  uint32_t w[2][W];
  __half2 sc[2][D / 64];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int row = g + 8 * t;
    if constexpr (W >= 4) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[t][4 * i]), "=r"(w[t][4 * i + 1]), "=r"(w[t][4 * i + 2]), "=r"(w[t][4 * i + 3])
                     : "r"(kc + swizzled<CH>(row, c * (W / 4) + i))
                     : "memory");
    } else if constexpr (W == 2) {
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                   : "=r"(w[t][0]), "=r"(w[t][1])
                   : "r"(kc + swizzled<CH>(row, c >> 1) + (c & 1) * 8)
                   : "memory");
    } else {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[t][0]) : "r"(kc + row * 16 + c * 4) : "memory");
    }
    if constexpr (D == 128) {
      uint2 v;
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                   : "=r"(v.x), "=r"(v.y)
                   : "r"(ksc + swizzled<2>(row, c >> 1) + (c & 1) * 8)
                   : "memory");
      sc[t][0] = u2h(v.x);
      sc[t][1] = u2h(v.y);
    } else {
      uint32_t v;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(ksc + row * 16 + c * 4) : "memory");
      sc[t][0] = u2h(v);
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) sc[t][i] = __hmul2(sc[t][i], __floats2half2_rn(0.5f, 1.f));
  }
  constexpr int PER = 32 / BITS;
#pragma unroll
  for (int m = 0; m < D / 16; ++m) {
    const int word = m * 4 / PER, pair = m * 4 % PER / 2, blk = word * PER / 16;
    uint32_t a[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const __half2 lo = __low2half2(sc[t][blk]), step = __high2half2(sc[t][blk]);
#pragma unroll
      for (int r = 0; r < 2; ++r) a[t][r] = h2u(__hfma2(half_code_pair<BITS>(w[t][word], pair + r, magic), step, lo));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint2 b = q(m, nt);
      mma16816(s[nt], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
    }
  }
}

// O^T += V^T P^T for 16 tokens.  live: per thread, masks of its token pairs (2c, 2c + 1) and
// (2c + 8, 2c + 9), zero where a token lies behind the sequence
template <int BITS, int D, int NT>
__device__ __forceinline__ void values(float (&o)[NT][D / 16][4], uint32_t vc, uint32_t vsc, int lane,
                                       const uint32_t (&p)[NT][2], uint32_t live0, uint32_t live1, uint32_t magic) {
  constexpr int CH = D * BITS / 128, CPU = 16 / BITS, SCH = D / 64;
  const int g = lane >> 2, c = lane & 3;
  // (lo, step) of the row's blocks: column 2 blk + {0, 1}, rows = tokens
  uint32_t sc[2 * SCH];
  {
    const int row = lane & 15, ch = lane >> 4;
    if constexpr (SCH == 2) {
      uint32_t r[4];
      ldsm4t(r, vsc + swizzled<2>(row, ch));
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = r[i];
    } else {
      ldsm2t(sc[0], sc[1], vsc + row * 16);
    }
#pragma unroll
    for (int i = 0; i < 2 * SCH; ++i)      // lanes of even columns g hold lo, of odd ones step
      sc[i] = h2u(__hmul2(u2h(sc[i]), __float2half2_rn(g & 1 ? 1.f : 0.5f))) & ((i & 1) ? live1 : live0);
  }
#pragma unroll
  for (int q2 = 0; q2 < CH; q2 += 2) {
    uint32_t r[4];
    if constexpr (CH == 1) ldsm2t(r[0], r[1], vc + (lane & 15) * 16);
    else ldsm4t(r, vc + swizzled<CH>(lane & 15, q2 + (lane >> 4)));
#pragma unroll
    for (int u = 0; u < (CH == 1 ? 1 : 2); ++u) {
      const int qc = q2 + u;
      const int blk = BITS == 8 ? qc : BITS == 4 ? 2 * qc + (g >> 2) : 4 * qc + (g >> 1);
      const int z = qc * (8 / BITS) / 4;               // scale chunk that holds the block
      const int src = 8 * (blk & 3) + c;
      const __half2 lo0 = u2h(__shfl_sync(0xffffffffu, sc[2 * z], src));
      const __half2 lo1 = u2h(__shfl_sync(0xffffffffu, sc[2 * z + 1], src));
      const __half2 st0 = u2h(__shfl_sync(0xffffffffu, sc[2 * z], src + 4));
      const __half2 st1 = u2h(__shfl_sync(0xffffffffu, sc[2 * z + 1], src + 4));
#pragma unroll
      for (int sp = 0; sp < CPU / 2; ++sp) {
        const uint32_t a0 = h2u(__hfma2(half_code_pair<BITS>(r[2 * u], 2 * sp, magic), st0, lo0));
        const uint32_t a1 = h2u(__hfma2(half_code_pair<BITS>(r[2 * u], 2 * sp + 1, magic), st0, lo0));
        const uint32_t a2 = h2u(__hfma2(half_code_pair<BITS>(r[2 * u + 1], 2 * sp, magic), st1, lo1));
        const uint32_t a3 = h2u(__hfma2(half_code_pair<BITS>(r[2 * u + 1], 2 * sp + 1, magic), st1, lo1));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][qc * (CPU / 2) + sp], a0, a1, a2, a3, p[nt][0], p[nt][1]);
      }
    }
  }
}

// stages of the ring and shared memory of a block
__host__ __device__ constexpr int stage_bytes(int D, int bk, int bv) { return TOK * (D * (bk + bv) / 8 + D / 2); }
__host__ __device__ constexpr int stages(int D, int bk, int bv) { return stage_bytes(D, bk, bv) > 3072 ? 3 : 4; }
template <int D, int NT>
struct Smem {
  static constexpr int QF = D / 16 * NT * 32 * 8;       // Q^T fragments
  static constexpr int MERGE = WARPS * 8 * NT * (D + 4) * 4;
  static constexpr int FIXED = QF + 8 * NT * 16 + 64;
  __host__ __device__ static constexpr int bytes(int bk, int bv) {
    const int ring = WARPS * stages(D, bk, bv) * stage_bytes(D, bk, bv);
    return FIXED + (ring > MERGE ? ring : MERGE);
  }
};

struct RowInfo {
  float mult;      // of a product with the normalised query, to scores in base 2 (without a cap)
  float slope;     // in base 2
  int pq;          // position
  int i;           // new row of the sequence, or -1 behind the last
};
}  // namespace ca

// Units of sequence b, and its first token (a multiple of 16)
__device__ __forceinline__ int cache_units(const CacheAttendArgs& A, int b, int unit, int& row0, int& n, int& len,
                                           int& first) {
  if (!seq_of(A.a, A.c.page_shift, b, row0, n, len) || n == 0) return 0;
  const int old = len - n;
  first = A.window ? max(0, old - A.window + 1) & ~15 : 0;
  return (len - first + unit - 1) / unit;
}

// The units of a block: all sequences' units are summed, and the sequence in which the block's range
// begins is looked for (by one warp, 32 sequences at a time).  false: the block has none.
struct BlockRange {
  long long total, w0, w1, base;   // units in all; this block's; first unit of sequence b
  int parts, b;                    // blocks that have units
};
template <int WARPS>
__device__ __forceinline__ bool block_units(const CacheAttendArgs& A, BlockRange& r) {
  constexpr int UNIT = WARPS * ca::TOK;
  __shared__ long long s_sum[WARPS], s_base;
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int row0, n, len, first;
  long long total = 0;
  for (int b = tid; b < A.a.B; b += WARPS * 32)
    total += (long long)cache_units(A, b, UNIT, row0, n, len, first) * A.c.H;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  r.total = 0;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) r.total += s_sum[k];
  r.parts = (int)min((long long)gridDim.x, r.total);
  if ((int)blockIdx.x >= r.parts) return false;
  r.w0 = cs::range_start(r.total, r.parts, blockIdx.x);
  r.w1 = cs::range_start(r.total, r.parts, blockIdx.x + 1);
  if (warp == 0) {
    long long base = 0;
    for (int b0 = 0; b0 < A.a.B; b0 += 32) {
      const int b = b0 + lane;
      long long u = b < A.a.B ? (long long)cache_units(A, b, UNIT, row0, n, len, first) * A.c.H : 0, sum = u;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, k);
        if (lane >= k) sum += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + sum > r.w0);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          s_b = b;
          s_base = base + sum - u;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __syncthreads();
  r.b = s_b;
  r.base = s_base;
  return true;
}

// The warps' sums of a job's rows joined, and stored or left as a piece.  merge: [warp][row][D + 4];
// the outputs are `factor` times what it holds.
template <int D, int ROWS, int WARPS>
__device__ __forceinline__ void merge_warps(const CacheAttendArgs& A, const float* merge, int b, int h, int row0, int R,
                                            int u0, int u1, int units, float factor, const BlockRange& range,
                                            long long base) {
  const int tid = threadIdx.x;
  const bool whole = u0 == 0 && u1 == units;
  for (int idx = tid; idx < ROWS * D; idx += WARPS * 32) {
    const int r = idx / D, d = idx % D;
    if (r >= R) break;
    float top = -INFINITY, y = 0.f, sum = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) top = fmaxf(top, merge[(k * ROWS + r) * (D + 4) + D]);
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float* rec = merge + (k * ROWS + r) * (D + 4);
      const float f = rec[D + 1] == 0.f ? 0.f : cs::ex2(rec[D] - top);
      y = fmaf(f, factor * rec[d], y);
      sum = fmaf(f, rec[D + 1], sum);
    }
    if (whole) {
      store_out(A, D, row0 + r / A.G, h * A.G + r % A.G, d, y, sum, top);
    } else {
      float* rec = A.pieces + ((2ll * blockIdx.x + (u0 == 0 ? 1 : 0)) * ROWS + r) * (D + 4);
      rec[d] = y;
      if (d == 0) {
        rec[D] = top;
        rec[D + 1] = sum;
      }
    }
  }
  if (!whole && u0 == 0 && tid == 0) {
    const long long end = base + (long long)(h + 1) * units;
    A.notes[blockIdx.x] = make_int4(b, h, 0, cs::pieces_until(range.total, range.parts, blockIdx.x, end));
  }
}

// What a warp needs of its job; the arrays are the kernel's registers.
template <int NT>
struct FewJob {
  int b, h, row0, n, len;
  int tw, count;           // first token of the warp's first stage; stages, UNIT tokens apart
  int edge, R;             // keys from `edge` on are inside every row's window; rows
  const float (&mult)[NT][2];
  const float (&slope)[NT][2];
  const int (&pq)[NT][2];
};

// A warp's stages, each of 16 tokens: copies run stages() - 1 ahead of the products.
template <int D, int NT, int KB, int VB, typename QF>
__device__ __forceinline__ void few_loop(const CacheAttendArgs& A, const FewJob<NT>& J, unsigned char* mine, int lane,
                                         QF&& q_of, float (&o)[NT][D / 16][4], float (&m_ref)[NT][2],
                                         float (&l)[NT][2]) {
  using namespace ca;
  constexpr int NST = stages(D, KB, VB), KBYTES = TOK * D * KB / 8, VBYTES = TOK * D * VB / 8, SBYTES = TOK * D / 4;
  constexpr int STAGE = KBYTES + VBYTES + 2 * SBYTES, KCH = D * KB / 128, VCH = D * VB / 128, SCH = D / 64;
  const int g = lane >> 2, c = lane & 3, len = J.len, old = J.len - J.n, count = J.count, tw = J.tw;
  const bool plain = A.cap == 0.f;
  const uint32_t magic = magic512(), ring = smem_addr(mine);
  const uint32_t kdst = swizzled<KCH>(lane / KCH, lane % KCH), vdst = KBYTES + SBYTES + swizzled<VCH>(lane / VCH, lane % VCH);
  const uint32_t ksd = KBYTES + swizzled<SCH>(lane / SCH, lane % SCH), vsd = ksd + SBYTES + VBYTES;
  const unsigned char* kc = A.c.codes[0] + lane * 16;
  const unsigned char* vc = A.c.codes[1] + lane * 16;
  const unsigned char* ks = reinterpret_cast<const unsigned char*>(A.c.scales[0]) + lane * 16;
  const unsigned char* vs = reinterpret_cast<const unsigned char*>(A.c.scales[1]) + lane * 16;
  const int* table = A.a.table + (long long)J.b * A.a.max_pages;
  // a stage's page is looked up one stage ahead of its copies
  int t_issue = tw, left = count;        // token of the next stage to copy; how many are to copy
  int page = left > 0 ? table[t_issue >> A.c.page_shift] : 0;
  uint32_t st_issue = 0;                 // its place in the ring
  unsigned lost = 0;                     // bit k: the stage k after the one in work has no page
  auto issue = [&](int ahead) {
    if (left > 0) {
      const int mine_page = page, t = t_issue;
      --left;
      t_issue += UNIT;
      if (left > 0) page = table[t_issue >> A.c.page_shift];
      if ((unsigned)mine_page < (unsigned)A.c.n_pages) {
        const uint32_t row = row_index(A.c, mine_page, J.h, t);
        const uint32_t dst = ring + st_issue;
        copy_rows<KCH>(dst, kdst, kc + row_bytes(row, D * KB / 8), lane);
        copy_rows<SCH>(dst, ksd, ks + row_bytes(row, D / 4), lane);
        copy_rows<VCH>(dst, vdst, vc + row_bytes(row, D * VB / 8), lane);
        copy_rows<SCH>(dst, vsd, vs + row_bytes(row, D / 4), lane);
      } else {
        lost |= 1u << ahead;
        raise_status(A.a.status, DEV_ERR_BATCH);
      }
      st_issue = st_issue == (NST - 1) * STAGE ? 0 : st_issue + STAGE;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) issue(i);
  uint32_t st = ring;
  for (int i = 0, t0 = tw; i < count; ++i, t0 += UNIT) {
    cp_wait<NST - 2>();
    __syncwarp();                        // everyone's copies of this stage are here, and the one before is read
    issue(NST - 1);
    const bool skip = lost & 1u;
    lost >>= 1;
    const uint32_t sta = st;
    st = st == ring + (NST - 1) * STAGE ? ring : st + STAGE;
    if (skip) continue;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[nt][k] = 0.f;
    scores<KB, D, NT>(s, sta, sta + KBYTES, lane, magic, q_of);
    // ---- scores to base 2: s[nt][2 t + k] is token g + 8 t, row 8 nt + 2 c + k ----
    const bool ragged = t0 + TOK > old || t0 < J.edge;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[nt][k] *= J.mult[nt][k & 1];
    if (!plain) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[nt][k] = cap_score(A, s[nt][k]) * cs::LOG2E;
    }
    if (ragged) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = t0 + g + 8 * (k >> 1);
        const int pk = t < len ? key_position(A, J.row0, old, t) : 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = 8 * nt + 2 * c + (k & 1);
          const bool sees = t < len && r < J.R && row_sees(A, J.row0, old, J.n, r / A.G, J.pq[nt][k & 1], t, pk);
          s[nt][k] = sees ? fmaf(-J.slope[nt][k & 1], (float)(J.pq[nt][k & 1] - pk), s[nt][k]) : -INFINITY;
        }
      }
    } else if (A.slopes) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          s[nt][k] = fmaf(-J.slope[nt][k & 1], (float)(J.pq[nt][k & 1] - (t0 + g + 8 * (k >> 1))), s[nt][k]);
    }
    // ---- running softmax over the tokens ----
    bool grow = false;
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mx[nt][k] = fmaxf(s[nt][k], s[nt][2 + k]);
        grow |= mx[nt][k] > m_ref[nt][k] + cs::LAG;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = mx[nt][k];
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, z));
          const float to = fmaxf(x, m_ref[nt][k]);
          const float f = m_ref[nt][k] == -INFINITY ? 0.f : cs::ex2(m_ref[nt][k] - to);
          m_ref[nt][k] = to;
          l[nt][k] *= f;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            o[nt][mt][k] *= f;
            o[nt][mt][2 + k] *= f;
          }
        }
      }
    }
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float ref = m_ref[nt][k & 1] == -INFINITY ? 0.f : m_ref[nt][k & 1] - cs::SHIFT;
        e[k] = cs::ex2(s[nt][k] - ref);
        l[nt][k & 1] += e[k];
      }
      p[nt][0] = transpose8(h2u(__floats2half2_rn(e[0], e[1])));
      p[nt][1] = transpose8(h2u(__floats2half2_rn(e[2], e[3])));
    }
    uint32_t live0 = 0xffffffffu, live1 = 0xffffffffu;
    if (t0 + TOK > len) {
      const int t = t0 + 2 * c;
      live0 = (t < len ? 0xffffu : 0u) | (t + 1 < len ? 0xffff0000u : 0u);
      live1 = (t + 8 < len ? 0xffffu : 0u) | (t + 9 < len ? 0xffff0000u : 0u);
    }
    values<VB, D, NT>(o, sta + KBYTES + SBYTES, sta + KBYTES + SBYTES + VBYTES, lane, p, live0, live1, magic);
  }
  cp_wait<0>();
}

template <int D, int NT, int KB, int VB>
__global__ void __launch_bounds__(ca::WARPS * 32, NT == 1 ? 4 : NT == 2 ? 3 : 2) cache_few_rows_kernel(CacheAttendArgs A) {
  using namespace ca;
  using S = Smem<D, NT>;
  extern __shared__ __align__(128) unsigned char ca_smem[];
  uint2* qf = reinterpret_cast<uint2*>(ca_smem);                        // [product][n-tile][lane]
  RowInfo* rows = reinterpret_cast<RowInfo*>(ca_smem + S::QF);          // [8 NT]
  unsigned char* ring = ca_smem + S::FIXED;
  float* merge = reinterpret_cast<float*>(ring);                        // [warp][row][D + 4], after the ring
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  constexpr int bk = KB, bv = VB;
  unsigned char* mine = ring + warp * stages(D, bk, bv) * stage_bytes(D, bk, bv);
  cs::wait_for_predecessor();
  cs::let_successor_start();
  BlockRange range;
  if (tid == 0) A.notes[blockIdx.x] = make_int4(0, 0, -1, 0);
  if (!block_units<WARPS>(A, range)) return;
  const long long w1 = range.w1;
  long long w = range.w0, base = range.base;
  int b = range.b, row0, n, len, first;
  const bool plain = A.cap == 0.f;

  while (w < w1 && b < A.a.B) {
    const int units = cache_units(A, b, UNIT, row0, n, len, first);
    if (w >= base + (long long)units * A.c.H) {   // next sequence (those without units are passed over)
      base += (long long)units * A.c.H;
      ++b;
      continue;
    }
    const int h = (int)((w - base) / units), u0 = (int)((w - base) % units);
    const int u1 = (int)min((long long)units, u0 + (w1 - w));
    const int old = len - n, R = n * A.G;
    // ---- queries: each row scaled by a power of two to the top of fp16's range, as B fragments ----
    __syncthreads();   // the previous job's fragments and merge buffer are read
    int pq_max = 0;
    for (int r = warp; r < 8 * NT; r += WARPS) {
      float x[D / 32], mx = 0.f;
      const bool is = r < R;
      const int j = h * A.G + r % A.G, i = r / A.G;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        x[k] = is ? ld_q(A, (row0 + i) * A.q_row + j * A.q_head + lane + 32 * k) : 0.f;
        mx = fmaxf(mx, fabsf(x[k]));
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      int e = 13;                                  // largest element into [2^13, 2^14)
      if (mx > 0.f && mx < INFINITY) e = ilogbf(mx);
      const float up = ldexpf(1.f, 13 - max(e, -100));
      if (lane == 0) {
        RowInfo ri;
        ri.i = is ? i : -1;
        ri.pq = is ? (A.positions ? A.positions[row0 + i] : old + i) : old;
        // two: the operands are halves
        ri.mult = A.scale * 2.f * ldexpf(1.f, max(e, -100) - 13) * (plain ? cs::LOG2E : 1.f);
        ri.slope = is && A.slopes ? A.slopes[j] * cs::LOG2E : 0.f;
        rows[r] = ri;
      }
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        // feature d belongs to thread column d / (D / 4); find its product, register and half
        const int d = lane + 32 * k, col = d / (D / 4), f = d % (D / 4), per = 32 / bk, in = f % per;
        int m, reg, hf;
        if (bk == 8) {
          m = f / 4;
          reg = in & 1;
          hf = in >> 1;
        } else {
          hf = in / (per / 2);
          const int pair = in % (per / 2);
          m = f / per * (per / 4) + pair / 2;
          reg = pair & 1;
        }
        reinterpret_cast<__half*>(qf)[(((m * NT + r / 8) * 32 + (r % 8) * 4 + col) * 2 + reg) * 2 + hf] =
            __float2half_rn(x[k] * up);
      }
    }
    __syncthreads();
    uint2 qr[NT <= 2 ? D / 16 : 1][NT <= 2 ? NT : 1];
    if constexpr (NT <= 2) {
#pragma unroll
      for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qr[m][nt] = qf[(m * NT + nt) * 32 + lane];
    }
    auto q_of = [&](int m, int nt) -> uint2 {
      if constexpr (NT <= 2) return qr[m][nt];
      else return qf[(m * NT + nt) * 32 + lane];
    };
    float mult[NT][2], slope[NT][2];
    int pq[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const RowInfo ri = rows[8 * nt + 2 * c + k];
        mult[nt][k] = ri.mult;
        slope[nt][k] = ri.slope;
        pq[nt][k] = ri.pq;
        pq_max = max(pq_max, ri.pq);
      }
    pq_max = __reduce_max_sync(0xffffffffu, pq_max);
    const int edge = A.window ? pq_max - A.window + 1 : 0;   // keys from here on are seen by the window

    float o[NT][D / 16][4], m_ref[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m_ref[nt][k] = -INFINITY;
        l[nt][k] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][mt][k] = 0.f;
    }

    // ---- this warp's share of the keys ----
    const int tw = first + u0 * UNIT + warp * TOK;
    int count = u1 - u0;
    if (tw + (count - 1) * UNIT >= len) count = tw < len ? (len - 1 - tw) / UNIT + 1 : 0;
    const FewJob<NT> job{b, h, row0, n, len, tw, count, edge, R, mult, slope, pq};
    few_loop<D, NT, KB, VB>(A, job, mine, lane, q_of, o, m_ref, l);
    // ---- the four warps' sums joined ----
    __syncthreads();
    const int cpu = 16 / bv;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum = l[nt][k];
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
        float* rec = merge + (warp * 8 * NT + 8 * nt + 2 * c + k) * (D + 4);
        if (g == 0) {
          rec[D] = m_ref[nt][k];
          rec[D + 1] = sum;
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          // features of product mt: chunk, then 16 / bits codes of unit g, pairs of them per product
          const int chunk = mt / (cpu / 2), d = chunk * (128 / bv) + g * cpu + 2 * (mt % (cpu / 2));
          rec[d] = o[nt][mt][k];
          rec[d + 1] = o[nt][mt][2 + k];
        }
      }
    __syncthreads();
    merge_warps<D, 8 * NT, WARPS>(A, merge, b, h, row0, R, u0, u1, units, 2.f, range, base);   // two: the operands are halves
    w += u1 - u0;
  }
}

}  // namespace jolt
