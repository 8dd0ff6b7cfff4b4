// Attention of the fewest rows per KV head (a single token's query group) over the paged cache: the
// products take the codes themselves, and the scales come in beside them.
//
// With k = lo + step c per block of 16 features,
//   q . k = sum_blocks step (q . c) + sum_blocks lo (sum of q over the block),
//   sum_t p_t v_t = sum_t (p_t step_t) c_t + sum_t p_t lo_t        (per block of the output),
// so the wide operand of a product may be the codes, and codes cost almost nothing to prepare: a code
// alone in a half, wherever it stands among the ten mantissa bits, is the subnormal number
// code * 4^k * 2^-24, exact in the products; the factor 4^k goes into q, or out of the output, the rest
// into fp32.  (Dequantising to fp16 first takes two more fp16 instructions per pair, on the pipe that
// bounds the other kernel, and rounds; here the scores are exact but for fp32 sums.)
// Every block has a scale of its own, and one 16-feature product holds codes of the two (4 bits) or
// four (2 bits) blocks of a 16-byte chunk.  They are told apart by the columns of the narrow side:
// with R rows in use, column n stands for row n % R and block n / R of the chunk.
//   K: column n of Q^T is zero outside its block's features, so S^T's columns are the blocks' partial
//      sums; each is multiplied by its token's step and the columns of a row are added.
//   V: column n of P^T is p times its block's step, rounded to fp16 once more; of an output row (a feature)
//      only the columns of its block are read.
// The sums with lo are one product more each: [tokens x blocks] lo with the blocks' sums of q (as two
// fp16 numbers, the second what the first leaves), and lo^T with p.
// Four rows at 4 bits (eight at 8, two at 2) fill one n-tile of eight columns; twice as many take two.
#pragma once

#include "cache_attend.cuh"

namespace jolt {
namespace cc {
// rows of an n-tile: the fewer the more blocks a chunk of K or V has
__host__ __device__ constexpr int rows_of(int kb, int vb) { return kb == 2 || vb == 2 ? 2 : kb == 4 || vb == 4 ? 4 : 8; }
// Weights are 2^(s - m + SHIFT) <= 2^(SHIFT + LAG) = 2^11, so that times a step below 32 they stay in
// fp16's range.  The steps of a block of features enter the products times a power of two, `up`, that keeps the
// largest so far below 32 (a larger one lowers `up`, and what was summed with it): without it the products of
// low weights and small steps would be subnormal (a weight of 2^-12 and steps of 4e-7 round to zero).  It is
// lowered to where the largest is below 4, so that it seldom has to be again (to below 32: 55 us instead of 52 us
// for the 40-head case), and together with the maximum, where the sums are rescaled anyway (on its own: 114 us
// instead of 109 us for the ragged batch, which it takes without `up` too; the 40-head case takes 49 us without).
constexpr float SHIFT = cs::SHIFT, LAG = 4.f, STEP_LIMIT = 32.f, UP_MOST = 0x1p15f;
constexpr int UP_LEAST = -11;               // fp16's largest number times 2^-11 is below 32

// codes s of the two halves of w, as 4^k 2^-24 times the code: k = factor of code_scale
template <int BITS>
__device__ __forceinline__ uint32_t codes_of(uint32_t w, int s) {
  if constexpr (BITS == 2) return (s < 4 ? w : w >> 8) & (0x00030003u << (2 * (s & 3)));
  else if constexpr (BITS == 4) return (s < 2 ? w : w >> 8) & (s & 1 ? 0x00f000f0u : 0x000f000fu);
  else return (s == 0 ? w : w >> 8) & 0x00ff00ffu;
}
// what takes the place of a code in its half away again
__host__ __device__ constexpr float code_scale(int bits, int s) {
  return bits == 2 ? (s & 3) == 0 ? 1.f : (s & 3) == 1 ? 0.25f : (s & 3) == 2 ? 0.0625f : 0.015625f
                   : bits == 4 ? (s & 1 ? 0.0625f : 1.f) : 1.f;
}
// D = A B, without an accumulator to set to zero first
__device__ __forceinline__ void mma16816_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 x;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a) : "memory");
  return x;
}

// Warps of a block: eight where two such blocks fit an SM, which halves the pieces to join (41 us
// instead of 45 us for one token over 65536 at 4 bits); but four at 2 bits, where a job is short for
// its blocks and their common barriers cost more (51 us instead of 54 us for the 40-head case).
template <int NT, int KB, int VB>
constexpr int warps_of() { return NT == 1 && KB > 2 && VB > 2 ? 8 : 4; }

template <int D, int NT, int KB, int VB>
struct Smem {
  static constexpr int WARPS = warps_of<NT, KB, VB>();
  static constexpr int ROWS = NT * rows_of(KB, VB);
  static constexpr int QF = (D / 16 + 1) * NT * 32 * 8;       // Q^T fragments, and those of the blocks' sums
  static constexpr int MERGE = WARPS * ROWS * (D + 4) * 4;
  static constexpr int RING = WARPS * ca::stages(D, KB, VB) * ca::stage_bytes(D, KB, VB);
  static constexpr int FIXED = (QF + ROWS * 16 + 127) / 128 * 128;
  static constexpr int BYTES = FIXED + (RING > MERGE ? RING : MERGE);
};
// blocks of an SM: by registers 16 warps, or 12 with two n-tiles; by shared memory what 228 KB hold with 1 KB for each
template <int D, int NT, int KB, int VB>
constexpr int blocks_per_sm() {
  const int by_smem = 228 * 1024 / (Smem<D, NT, KB, VB>::BYTES + 1024), by_regs = NT == 1 ? 16 / Smem<D, NT, KB, VB>::WARPS : 3;
  return by_smem < by_regs ? by_smem : by_regs;
}
}  // namespace cc

template <int D, int NT, int KB, int VB>
__global__ void __launch_bounds__(cc::warps_of<NT, KB, VB>() * 32,
                                  NT == 1 ? 16 / cc::warps_of<NT, KB, VB>() : 3) cache_codes_kernel(CacheAttendArgs A) {
  using namespace ca;
  using S = cc::Smem<D, NT, KB, VB>;
  constexpr int WARPS = S::WARPS, UNIT = WARPS * TOK;
  constexpr int RPT = cc::rows_of(KB, VB), ROWS = S::ROWS;
  constexpr int KBPC = 8 / KB, VBPC = 8 / VB;                 // blocks of a chunk
  constexpr int KPER = 32 / KB, CPU = 16 / VB;                // codes of a word of K, of a unit of V
  constexpr int KCH = D * KB / 128, VCH = D * VB / 128, SCH = D / 64;
  constexpr int NST = stages(D, KB, VB), KBYTES = TOK * D * KB / 8, VBYTES = TOK * D * VB / 8, SBYTES = TOK * D / 4;
  constexpr int STAGE = KBYTES + VBYTES + 2 * SBYTES;
  extern __shared__ __align__(128) unsigned char cc_smem[];
  uint2* qf = reinterpret_cast<uint2*>(cc_smem);              // [product, or D / 16: the sums][n-tile][lane]
  RowInfo* rows = reinterpret_cast<RowInfo*>(cc_smem + S::QF);
  float* merge = reinterpret_cast<float*>(cc_smem + S::FIXED);   // [warp][row][D + 4], after the ring
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_addr(cc_smem + S::FIXED) + warp * NST * STAGE, qfa = smem_addr(qf) + lane * 8;
  cs::wait_for_predecessor();
  cs::let_successor_start();
  BlockRange range;
  if (tid == 0) A.notes[blockIdx.x] = make_int4(0, 0, -1, 0);
  if (!block_units<WARPS>(A, range)) return;
  const long long w1 = range.w1;
  long long w = range.w0, base = range.base;
  int b = range.b, row0, n, len, first;
  const bool plain = A.cap == 0.f;
  // this lane's columns 2 c, 2 c + 1 of an n-tile: rows col_row, col_row + 1 of it, block group col_grp
  const int col_row = 2 * c % RPT, col_grp = 2 * c / RPT;
  const int b_grp = g / RPT;                                  // block group of column g (as operand B)
  // where this lane's copies go, and come from (see copy_rows)
  const uint32_t kdst = swizzled<KCH>(lane / KCH, lane % KCH), vdst = KBYTES + SBYTES + swizzled<VCH>(lane / VCH, lane % VCH);
  const uint32_t ksd = KBYTES + swizzled<SCH>(lane / SCH, lane % SCH), vsd = ksd + SBYTES + VBYTES;
  const unsigned char* const kc = A.c.codes[0] + lane * 16;
  const unsigned char* const vc = A.c.codes[1] + lane * 16;
  const unsigned char* const ks = reinterpret_cast<const unsigned char*>(A.c.scales[0]) + lane * 16;
  const unsigned char* const vs = reinterpret_cast<const unsigned char*>(A.c.scales[1]) + lane * 16;

  // Where this lane reads in a stage (128-byte aligned): word c of chunk q of K's row g is at k_at with q
  // xored into the chunk's bits, row g + 8 (the same swizzle) a constant further; so are the scales of
  // block col_grp % KBPC of K's chunks, and the chunks of V's row lane % 16.
  const uint32_t k_at = swizzled<KCH>(g, 0) + c * 4;
  const uint32_t ks_at = KBYTES + swizzled<SCH>(g, 0) + (col_grp % KBPC) * 4;
  const uint32_t lo_at = KBYTES + (D == 128 ? swizzled<2>(g, c >> 1) : g * 16) + (c & 1) * 8;
  const uint32_t v_at = KBYTES + SBYTES + swizzled<VCH>(lane & 15, VCH == 1 ? 0 : lane >> 4);
  const uint32_t vs_at = KBYTES + SBYTES + VBYTES + (SCH == 2 ? swizzled<2>(lane & 15, lane >> 4) : (lane & 15) * 16);

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
    __syncthreads();   // the previous job's fragments and merge buffer are read
    // ---- queries, scaled by a power of two to the top of fp16's range, as B fragments ----
    for (int r = warp; r < ROWS; r += WARPS) {
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
      if (mx > 0.f && mx < INFINITY) e = max(ilogbf(mx), -100);
      const float up = ldexpf(1.f, 13 - e);
      if (lane == 0) {
        RowInfo ri;
        ri.i = is ? i : -1;
        ri.pq = is ? (A.positions ? A.positions[row0 + i] : old + i) : old;
        ri.mult = A.scale * 16.f * ldexpf(1.f, e - 13) * (plain ? cs::LOG2E : 1.f);   // 16: see the sums below
        ri.slope = is && A.slopes ? A.slopes[j] * cs::LOG2E : 0.f;
        rows[r] = ri;
      }
      const int nt = r / RPT, rt = r % RPT;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        // feature d: word d / KPER of the row, pair `pair` of it, half hf; the word is thread column col's
        // of chunk q
        const int d = lane + 32 * k, word = d / KPER, in = d % KPER, hf = in / (KPER / 2), pair = in % (KPER / 2);
        const int q = word / 4, col = word % 4, m = q * (KPER / 4) + pair / 2, reg = pair & 1;
        const float y = x[k] * up;
        float sum = y;                                        // over the block's 16 features
#pragma unroll
        for (int z = 8; z > 0; z >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
        const __half value = __float2half_rn(y * cc::code_scale(KB, pair)), zero = __float2half_rn(0.f);
        // the sums divided by 16 (they may be 16 times as large as the queries), in two parts
        const __half hi = __float2half_rn(sum * 0.0625f), lo = __float2half_rn(sum * 0.0625f - __half2float(hi));
#pragma unroll
        for (int grp = 0; grp < 8 / RPT; ++grp) {
          const int column = grp * RPT + rt;
          const bool own = col * KBPC / 4 == grp % KBPC;
          __half* at = reinterpret_cast<__half*>(qf) + ((m * NT + nt) * 32 + column * 4 + col) * 4 + reg * 2 + hf;
          *at = own ? value : zero;
          if (lane % 16 == 0) {                               // block blk of the row
            const int blk = d / 16;
            const bool counts = grp % KBPC == 0;              // once per row, not once per column
            __half* sums = reinterpret_cast<__half*>(qf) + ((D / 16 * NT + nt) * 32 + column * 4) * 4;
            if constexpr (D == 128) {
              // products over 8 blocks (first register: hi) and the same 8 again (second: lo)
              sums[(blk / 2) * 4 + (blk & 1)] = counts ? hi : zero;
              sums[(blk / 2) * 4 + 2 + (blk & 1)] = counts ? lo : zero;
            } else {
              // 4 blocks (hi), the same 4 again (lo), and nothing
              sums[(blk / 2) * 4 + (blk & 1)] = counts ? hi : zero;
              sums[(2 + blk / 2) * 4 + (blk & 1)] = counts ? lo : zero;
              sums[(blk / 2) * 4 + 2 + (blk & 1)] = zero;
              sums[(2 + blk / 2) * 4 + 2 + (blk & 1)] = zero;
            }
          }
        }
      }
    }
    __syncthreads();
    float mult[NT][2], slope[NT][2];
    int pq[NT][2], pq_max = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const RowInfo ri = rows[RPT * nt + col_row + k];
        mult[nt][k] = ri.mult;
        slope[nt][k] = ri.slope;
        pq[nt][k] = ri.pq;
        pq_max = max(pq_max, ri.pq);
      }
    pq_max = __reduce_max_sync(0xffffffffu, pq_max);
    const int edge = A.window ? pq_max - A.window + 1 : 0;    // keys from here on are seen by the window
    float o[NT][D / 16][4], olo[NT][4], m_ref[NT][2], l[NT][2];
    // `up` of block 4 z + g / 2 in lanes of odd g, which hold the steps; the others hold lo, which stays as it
    // is.  o is as many times its sums.
    uint32_t up[SCH];
    const uint32_t limit = h2u(__float2half2_rn(g & 1 ? cc::STEP_LIMIT : INFINITY));
#pragma unroll
    for (int z = 0; z < SCH; ++z) up[z] = h2u(__float2half2_rn(g & 1 ? cc::UP_MOST : 1.f));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m_ref[nt][k] = -INFINITY;
        l[nt][k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        olo[nt][k] = 0.f;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) o[nt][mt][k] = 0.f;
      }
    }
    // ---- this warp's stages: 16 tokens, UNIT tokens apart; copies run NST - 1 ahead of the products ----
    const int tw = first + u0 * UNIT + warp * TOK;
    int count = u1 - u0;
    if (tw + (count - 1) * UNIT >= len) count = tw < len ? (len - 1 - tw) / UNIT + 1 : 0;
    const int* table = A.a.table + (long long)b * A.a.max_pages;
    int t_issue = tw, left = count;        // token of the next stage to copy; how many are to copy
    int page = left > 0 ? table[t_issue >> A.c.page_shift] : 0;   // looked up one stage ahead
    uint32_t st_issue = 0;                 // its place in the ring
    unsigned lost = 0;                     // bit k: the stage k after the one in work has no page
    auto issue = [&](int ahead) {
      if (left > 0) {
        const int mine_page = page, t = t_issue;
        --left;
        t_issue += UNIT;
        if (left > 0) page = table[t_issue >> A.c.page_shift];
        if ((unsigned)mine_page < (unsigned)A.c.n_pages) {
          const uint32_t row = row_index(A.c, mine_page, h, t);
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
      // ---- scores: s[nt][2 t + k] is token g + 8 t, column 2 c + k ----
      float s[NT][4];
      {
        // lo of blocks 2 c, 2 c + 1 with the blocks' sums
        uint32_t a[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint2 x = cc::lds64(sta + lo_at + 8 * t * SCH * 16);
          a[t] = __byte_perm(x.x, x.y, 0x5410);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = cc::lds64(qfa + (D / 16 * NT + nt) * 256);
          cc::mma16816_0(s[nt], a[0], a[1], a[0], a[1], q.x, q.y);
        }
      }
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[nt][k] = 0.f;
#pragma unroll
      for (int q = 0; q < KCH; ++q) {
        const uint32_t at = (sta + k_at) ^ (q * 16u);
        const uint32_t x0 = cc::lds32(at), x1 = cc::lds32(at + 8 * KCH * 16);
        const uint32_t sat = ((sta + ks_at) ^ (q * KBPC / 4 * 16u)) + (q * KBPC & 3) * 4;
        const float st0 = __high2float(u2h(cc::lds32(sat))), st1 = __high2float(u2h(cc::lds32(sat + 8 * SCH * 16)));
        float part[NT][4];
#pragma unroll
        for (int pp = 0; pp < KPER / 4; ++pp) {
          const uint32_t a0 = cc::codes_of<KB>(x0, 2 * pp), a1 = cc::codes_of<KB>(x1, 2 * pp);
          const uint32_t a2 = cc::codes_of<KB>(x0, 2 * pp + 1), a3 = cc::codes_of<KB>(x1, 2 * pp + 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 qv = cc::lds64(qfa + ((q * (KPER / 4) + pp) * NT + nt) * 256);
            if (pp == 0) cc::mma16816_0(part[nt], a0, a1, a2, a3, qv.x, qv.y);
            else mma16816(part[nt], a0, a1, a2, a3, qv.x, qv.y);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][0] = fmaf(st0, part[nt][0], acc[nt][0]);
          acc[nt][1] = fmaf(st0, part[nt][1], acc[nt][1]);
          acc[nt][2] = fmaf(st1, part[nt][2], acc[nt][2]);
          acc[nt][3] = fmaf(st1, part[nt][3], acc[nt][3]);
        }
      }
      // both sums over 16; the columns of a row added
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float y = fmaf(acc[nt][k], 0x1p20f, s[nt][k]);
          if constexpr (KBPC == 2 && RPT == 4) y += __shfl_xor_sync(0xffffffffu, y, 2);
          if constexpr (KBPC == 2 && RPT == 2) y += __shfl_xor_sync(0xffffffffu, y, 1);
          if constexpr (KBPC == 4) {
            y += __shfl_xor_sync(0xffffffffu, y, 1);
            y += __shfl_xor_sync(0xffffffffu, y, 2);
          }
          y *= mult[nt][k & 1];
          if (!plain) y = cap_score(A, y) * cs::LOG2E;
          s[nt][k] = y;
        }
      if (t0 + TOK > old || t0 < edge) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = t0 + g + 8 * (k >> 1);
          const int pk = t < len ? key_position(A, row0, old, t) : 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int r = RPT * nt + col_row + (k & 1);
            const bool sees = t < len && r < R && row_sees(A, row0, old, n, r / A.G, pq[nt][k & 1], t, pk);
            s[nt][k] = sees ? fmaf(-slope[nt][k & 1], (float)(pq[nt][k & 1] - pk), s[nt][k]) : -INFINITY;
          }
        }
      } else if (A.slopes) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            s[nt][k] = fmaf(-slope[nt][k & 1], (float)(pq[nt][k & 1] - (t0 + g + 8 * (k >> 1))), s[nt][k]);
      }
      // ---- the values' (lo, step) as columns, tokens as pairs, the steps times `up` ----
      auto load_scales = [&](uint32_t (&x)[2 * SCH]) {
        if constexpr (SCH == 2) ldsm4t(x, sta + vs_at);
        else ldsm2t(x[0], x[1], sta + vs_at);
        if (t0 + TOK > len) {              // what lies behind the sequence may be anything
          const int t = t0 + 2 * c;
          const uint32_t live0 = (t < len ? 0xffffu : 0u) | (t + 1 < len ? 0xffff0000u : 0u);
          const uint32_t live1 = (t + 8 < len ? 0xffffu : 0u) | (t + 9 < len ? 0xffff0000u : 0u);
#pragma unroll
          for (int k = 0; k < 2 * SCH; ++k) x[k] &= (k & 1) ? live1 : live0;
        }
      };
      uint32_t sc[2 * SCH];
      load_scales(sc);
#pragma unroll
      for (int k = 0; k < 2 * SCH; ++k) sc[k] = h2u(__hmul2(u2h(sc[k]), u2h(up[k / 2])));
      __half2 top = u2h(sc[0]);
#pragma unroll
      for (int k = 1; k < 2 * SCH; ++k) top = __hmax2(top, u2h(sc[k]));
      // ---- running softmax over the tokens ----
      bool grow = !__hblt2(top, u2h(limit));
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[nt][k] = fmaxf(s[nt][k], s[nt][2 + k]);
          grow |= mx[nt][k] > m_ref[nt][k] + cc::LAG;
        }
      if (__any_sync(0xffffffffu, grow)) {
        float f[NT][2], fu[SCH];           // what the sums are multiplied by, for the maximum and for `up`
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = mx[nt][k];
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, z));
            const float to = fmaxf(x, m_ref[nt][k]);
            f[nt][k] = m_ref[nt][k] == -INFINITY ? 0.f : cs::ex2(m_ref[nt][k] - to);
            m_ref[nt][k] = to;
            l[nt][k] *= f[nt][k];
            olo[nt][k] *= f[nt][k];
            olo[nt][2 + k] *= f[nt][k];
          }
        load_scales(sc);
#pragma unroll
        for (int z = 0; z < SCH; ++z) {
          const float2 x = __half22float2(__hmax2(u2h(sc[2 * z]), u2h(sc[2 * z + 1])));
          float most = g & 1 ? fmaxf(x.x, x.y) : 0.f, was = __low2float(u2h(up[z]));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          // the power of two that takes the largest into [2, 4)
          const int e = max(cc::UP_LEAST, 1 - ((int)(__float_as_uint(most) >> 23) - 127));
          const float to = most * was >= cc::STEP_LIMIT ? __uint_as_float((uint32_t)(e + 127) << 23) : was;
          fu[z] = to * __uint_as_float(0x7f000000u - __float_as_uint(was));   // to / was
          up[z] = h2u(__float2half2_rn(to));
          sc[2 * z] = h2u(__hmul2(u2h(sc[2 * z]), u2h(up[z])));
          sc[2 * z + 1] = h2u(__hmul2(u2h(sc[2 * z + 1]), u2h(up[z])));
        }
#pragma unroll
        for (int q = 0; q < VCH; ++q) {
          const int blk = q * VBPC + col_grp % VBPC;          // of this lane's columns
          const float fq = __shfl_sync(0xffffffffu, fu[q * VBPC / 4], 8 * (blk & 3) + 4);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float both = f[nt][k & 1] * fq;
#pragma unroll
              for (int sp = 0; sp < CPU / 2; ++sp) o[nt][q * (CPU / 2) + sp][k] *= both;
            }
        }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float ref = m_ref[nt][k & 1] == -INFINITY ? 0.f : m_ref[nt][k & 1] - cc::SHIFT;
          e[k] = cs::ex2(s[nt][k] - ref);
          l[nt][k & 1] += e[k];
        }
        p[nt][0] = transpose8(h2u(__floats2half2_rn(e[0], e[1])));
        p[nt][1] = transpose8(h2u(__floats2half2_rn(e[2], e[3])));
      }
      // ---- values ----
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma16816(olo[nt], sc[0], SCH == 2 ? sc[2 * (SCH - 1)] : 0u, sc[1], SCH == 2 ? sc[2 * (SCH - 1) + 1] : 0u, p[nt][0], p[nt][1]);
#pragma unroll
      for (int q2 = 0; q2 < VCH; q2 += 2) {
        uint32_t x[4];
        if constexpr (VCH == 1) ldsm2t(x[0], x[1], sta + v_at);
        else ldsm4t(x, (sta + v_at) ^ (q2 * 16u));
#pragma unroll
        for (int u = 0; u < (VCH == 1 ? 1 : 2); ++u) {
          const int q = q2 + u, blk = q * VBPC + b_grp % VBPC, z = q * VBPC / 4, src = 8 * (blk & 3) + 4 + c;
          const __half2 st0 = u2h(__shfl_sync(0xffffffffu, sc[2 * z], src));
          const __half2 st1 = u2h(__shfl_sync(0xffffffffu, sc[2 * z + 1], src));
          uint32_t ps[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            ps[nt][0] = h2u(__hmul2(u2h(p[nt][0]), st0));
            ps[nt][1] = h2u(__hmul2(u2h(p[nt][1]), st1));
          }
#pragma unroll
          for (int sp = 0; sp < CPU / 2; ++sp) {
            const uint32_t a0 = cc::codes_of<VB>(x[2 * u], 2 * sp), a1 = cc::codes_of<VB>(x[2 * u], 2 * sp + 1);
            const uint32_t a2 = cc::codes_of<VB>(x[2 * u + 1], 2 * sp), a3 = cc::codes_of<VB>(x[2 * u + 1], 2 * sp + 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][q * (CPU / 2) + sp], a0, a1, a2, a3, ps[nt][0], ps[nt][1]);
          }
        }
      }
    }
    cp_wait<0>();
    // ---- outputs to the merge buffer: of a feature, the columns of its block ----
    __syncthreads();
    const int own = g / VB;                  // block of unit g within its chunk
    float back[VCH];                         // what takes 2^-24 and `up` of that block away again
#pragma unroll
    for (int q = 0; q < VCH; ++q)
      back[q] = 0x1p24f / __low2float(u2h(__shfl_sync(0xffffffffu, up[q * VBPC / 4], 8 * ((q * VBPC + own) & 3) + 4)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum = l[nt][k];
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
        float* rec = merge + (warp * ROWS + RPT * nt + col_row + k) * (D + 4);
        if (g == 0 && col_grp == 0) {
          rec[D] = m_ref[nt][k];
          rec[D + 1] = sum;
        }
#pragma unroll
        for (int q = 0; q < VCH; ++q) {
          const int blk = q * VBPC + own;    // its lo sum: rows 2 (blk % 4) of the upper or lower half
          const float up = __shfl_sync(0xffffffffu, olo[nt][k], 8 * (blk & 3) + c);
          const float lower = __shfl_sync(0xffffffffu, olo[nt][2 + k], 8 * (blk & 3) + c);
          const float lo = blk >= 4 ? lower : up;
          if (col_grp == own) {
#pragma unroll
            for (int sp = 0; sp < CPU / 2; ++sp) {
              const int mt = q * (CPU / 2) + sp, d = q * (128 / VB) + g * CPU + 2 * sp;
              rec[d] = fmaf(o[nt][mt][k], back[q] * cc::code_scale(VB, 2 * sp), lo);
              rec[d + 1] = fmaf(o[nt][mt][2 + k], back[q] * cc::code_scale(VB, 2 * sp + 1), lo);
            }
          }
        }
      }
    __syncthreads();
    merge_warps<D, ROWS, WARPS>(A, merge, b, h, row0, R, u0, u1, units, 1.f, range, base);
    w += u1 - u0;
  }
}

}  // namespace jolt
