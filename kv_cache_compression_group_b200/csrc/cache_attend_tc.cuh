// Attention of many rows per KV head (wide trees, chunks of a prompt) over the paged cache, on the
// 5th-generation tensor cores.
//
// A job is 128 rows (new row x query head) of one KV head, or 256 where there are more; its keys come
// in tiles of 128 tokens.  One persistent CTA of 20 warps per SM:
//   * one warp walks the tiles and looks up their pages, several tiles ahead;
//   * eight dequantising warps take 16 tokens of every tile each: packed codes and (lo, step) pairs
//     straight to registers, one tile ahead, then fp16(lo / 2 + step * (code / 2)) into the
//     128-byte-swizzled operand tiles, two of K and two of V.  The features of a row keep the order
//     in which a packed word gives its pairs; Q is laid out in the same order, the output columns
//     are put back;
//   * two softmax warpgroups with score and output accumulators of their own (all 512 columns of
//     tensor memory).  With 256 rows each has 128 of them and both use every tile, which halves the
//     dequantisation; with 128 rows one takes the even and the other the odd tiles, joined at the
//     end.  A thread has one row: it reads its scores twice (maximum, then weights) and writes the
//     weights as fp16 over the scores.  The reference maximum may lag by 2^8, so rescaling O, a pass
//     through tensor memory, is rare after the first tiles;
//   * one thread issues the products, O += P V (P from tensor memory) and then the group's next
//     S = Q K^T, of the one group while the other is at its softmax.  (Scores in two halves of 64
//     keys, to overlap a group's products with its own softmax, were slower: a product with N = 64
//     waits for the shared memory that Q is read from again, and there are twice the commits.)
// What bounds it at D = 128: 2048 new rows of 32 query heads over 16384 tokens (8 KV heads, 4 bits) take 650 us,
// 5800 clocks for a tile of 256 rows and 128 tokens.  Its products take 2048 of them (tensor pipe 37 %), its
// exponentials 2048 at 16 per clock (that unit 38 %), instructions issue in 43 %: no unit is full, the rest is
// the roles' waiting for one another.  With 128 rows (wide trees, 124 us for 16 sequences of up to 8192 tokens)
// tensor pipe and exponentials are at 22 %, issue at 39 %.  The compiler holds every role to the launch's 96
// registers and spills: 466 to 502 bytes of stores and 592 to 804 of loads, by instance.
//
// Every wait is bounded; after one gave up, the roles keep their barrier schedule without waiting or
// issuing, so the CTA ends, and the issued products are drained before tensor memory is freed.
#pragma once

#include "cache_attend.cuh"
#include "umma.cuh"

namespace jolt {
namespace ct {
constexpr int TILE = 128;
constexpr int THREADS = 640;
constexpr int RING = 8;                        // tiles that the walk is ahead
constexpr int BOX = 128 * 128;                 // bytes of 128 rows x 64 fp16 features
template <int D>
struct Smem {
  static constexpr int OPND = D / 64 * BOX;    // bytes of a 128 x D operand tile
  static constexpr int Q = 0, K = OPND, V = 3 * OPND, Q2 = 5 * OPND;
  static constexpr int bytes(bool pair) { return (pair ? 6 : 5) * OPND + 1024; }
};
// fp16 A and B, fp32 accumulator, M = 128
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  umma::mma_bf16(d, a, b, id, acc);            // kind::f16; the types are the instruction descriptor's
}
// A (fp16 pairs) from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
        "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// 16 rows of a page, contiguous; address and size are multiples of 16 bytes
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// A bounded wait for a phase of a barrier that looks before anything else: reading the clock, as
// umma::mbar_wait does, or the flag takes longer than most waits.  A look lets the thread sleep for up
// to 20 us, so the bound is between some milliseconds and about three seconds; who gives up raises
// the flag, which ends the other waits too.
constexpr int LOOKS = 1 << 17;
__device__ __forceinline__ bool mbar_look(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  for (int i = 0; i < LOOKS; ++i) {
    if (mbar_look(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  return false;
}
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// the values of earlier loads may be used after this; they pass through it so that no use moves up
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15])
               :
               : "memory");
  asm volatile(""
               : "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]), "+r"(a[21]), "+r"(a[22]), "+r"(a[23]),
                 "+r"(a[24]), "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]), "+r"(a[30]), "+r"(a[31])
               :
               : "memory");
  asm volatile(""
               : "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                 "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15])
               :
               : "memory");
  asm volatile(""
               : "+r"(b[16]), "+r"(b[17]), "+r"(b[18]), "+r"(b[19]), "+r"(b[20]), "+r"(b[21]), "+r"(b[22]), "+r"(b[23]),
                 "+r"(b[24]), "+r"(b[25]), "+r"(b[26]), "+r"(b[27]), "+r"(b[28]), "+r"(b[29]), "+r"(b[30]), "+r"(b[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
      ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]),
        "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]),
        "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
// Registers of a thread of each role.  640 threads are launched with 96, 61440 in all, which the shares
// 256 x 120 + 256 x 88 + 128 x 64 use up.  (With fewer at the launch the softmax warps would wait for theirs
// forever: launch_many refuses a kernel that was compiled otherwise.)
constexpr int LAUNCH_REGS = 96, SOFTMAX_REGS = 120, DEQUANT_REGS = 88, ISSUE_REGS = 64;
static_assert(256 * SOFTMAX_REGS + 256 * DEQUANT_REGS + 128 * ISSUE_REGS <= THREADS * LAUNCH_REGS);
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// 16-byte piece `piece` (8 features) of row `row` of an operand tile
__device__ __forceinline__ uint32_t piece_addr(uint32_t tile, int row, int piece) {
  return tile + (piece >> 3) * BOX + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}
// feature at place p of a row as the dequantised words hold it
__device__ __forceinline__ constexpr int feature_at(int bits, int p) {
  const int per = 32 / bits, in = p & (per - 1);
  return (p - in) + (in >> 1) + (in & 1) * (per >> 1);
}

// one sequence's jobs, of ROWS rows
template <int ROWS>
struct Seq {
  int row0, n, len, first, tiles;      // tiles: of ROWS rows
  bool causal;
  // units of row tile rt: the keys that any of its rows may see
  __device__ int units(const CacheAttendArgs& A, int rt) const {
    int end = len;
    if (causal) end = min(len, len - n + min(n, ((rt + 1) * ROWS - 1) / A.G + 1));
    return (end - first + TILE - 1) / TILE;
  }
};
template <int ROWS>
__device__ __forceinline__ bool load_seq(const CacheAttendArgs& A, int b, Seq<ROWS>& s) {
  const int u = cache_units(A, b, TILE, s.row0, s.n, s.len, s.first);
  if (u == 0) return false;
  s.tiles = (int)(((long long)s.n * A.G + ROWS - 1) / ROWS);
  s.causal = A.mask == nullptr;
  return true;
}
template <int ROWS>
__device__ __forceinline__ long long seq_units(const CacheAttendArgs& A, int b) {
  Seq<ROWS> s;
  if (!load_seq(A, b, s)) return 0;
  if (!s.causal) return (long long)s.tiles * s.units(A, 0);
  long long sum = 0;
  for (int rt = 0; rt < s.tiles; ++rt) sum += s.units(A, rt);
  return sum;
}

// The jobs of a block's range [w, w1), in order; every thread walks its own copy.
template <int ROWS>
struct Jobs {
  long long w, w1, base;   // base: first unit of (b, h, rt)
  int b, h, rt;
  Seq<ROWS> s;
  int units, u0, u1;       // of the job, and of this block's part of it
  __device__ void start(const CacheAttendArgs& A, long long from, long long to, int b0, long long b0_base) {
    w = from;
    w1 = to;
    b = b0;
    base = b0_base;
    h = rt = 0;
    if (w >= w1) return;
    load_seq(A, b, s);
    const long long per = seq_units<ROWS>(A, b);
    h = (int)((w - base) / per);
    base += h * per;
    settle(A);
  }
  // the job that holds unit w
  __device__ void settle(const CacheAttendArgs& A) {
    for (;;) {
      if (rt == s.tiles) {
        rt = 0;
        if (++h == A.c.H) {
          h = 0;
          do ++b;
          while (b < A.a.B && !load_seq(A, b, s));
          if (b == A.a.B) {             // not reached while the batch stays as it was: w < w1
            w = w1;
            return;
          }
        }
      }
      units = s.units(A, rt);
      if (w < base + units) break;
      base += units;
      ++rt;
    }
    u0 = (int)(w - base);
    u1 = (int)min((long long)units, u0 + (w1 - w));
  }
  __device__ void next(const CacheAttendArgs& A) {
    w += u1 - u0;
    if (w < w1) settle(A);
  }
};

// ---- dequantisation: a warp's 16 tokens of a tile -----------------------------------------
// Lane l takes row l % 8 (and + 8) and 16-byte chunks of its codes, so that the 16-byte stores of
// eight lanes fall into eight rows, that is eight bank groups.
template <int BITS, int D>
struct Raw {
  static constexpr int CH = D * BITS / 128, N = CH / 2 > 0 ? CH / 2 : 1;   // chunks of a row; of a lane
  static constexpr int BLKS = 8 / BITS;                                    // (lo, step) pairs of a chunk
  __device__ static int row(int lane, int i) {
    if constexpr (CH >= 4) return (lane & 7) + 8 * (i / (CH / 4));
    else return (lane & 7) + 8 * ((lane >> 3) / CH & 1);
  }
  __device__ static int chunk(int lane, int i) {
    if constexpr (CH >= 4) return (lane >> 3) + 4 * (i % (CH / 4));
    else return (lane >> 3) % CH;
  }
};
// (Plain loads, not through the read-only path: the kernel may be brought up before the one that writes the rows has
// ended, so they are not constant while it lives.)
struct RawRegs {
  uint4 code[4];
  uint32_t scale[4];
};

template <int BITS, int D, bool ALL>
__device__ __forceinline__ void raw_load_rows(RawRegs& r, const unsigned char* codes, const __half2* scales, int lane,
                                              int live) {
  using W = Raw<BITS, D>;
#pragma unroll
  for (int i = 0; i < W::N; ++i) {
    const int row = W::row(lane, i), ch = W::chunk(lane, i);
    const bool on = (ALL || row < live) && (W::CH > 1 || lane < 16);
    const uint4* src = reinterpret_cast<const uint4*>(codes + row * (D * BITS / 8) + ch * 16);
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(scales + row * (D / 16) + ch * W::BLKS);
    if (!on) {
      r.code[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < W::BLKS; ++k) r.scale[i * W::BLKS + k] = 0u;
      continue;
    }
    r.code[i] = *src;
    if constexpr (W::BLKS == 1) {
      r.scale[i] = *sc;
    } else if constexpr (W::BLKS == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(sc);
      r.scale[2 * i] = v.x;
      r.scale[2 * i + 1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(sc);
      r.scale[0] = v.x;
      r.scale[1] = v.y;
      r.scale[2] = v.z;
      r.scale[3] = v.w;
    }
  }
}
template <int BITS, int D>
__device__ __forceinline__ void raw_load(RawRegs& r, const unsigned char* codes, const __half2* scales, long long row,
                                         int lane, int live) {
  codes += row_bytes((uint32_t)row, D * BITS / 8);
  scales += row_bytes((uint32_t)row, D / 16);
  if (live == 16) raw_load_rows<BITS, D, true>(r, codes, scales, lane, live);
  else raw_load_rows<BITS, D, false>(r, codes, scales, lane, live);
}

// rows `row16` .. + 15 of the operand tile
template <int BITS, int D>
__device__ __forceinline__ void raw_store(const RawRegs& r, uint32_t tile, int row16, int lane, uint32_t magic) {
  using W = Raw<BITS, D>;
  constexpr int PER = 32 / BITS;                // codes of a word
#pragma unroll
  for (int i = 0; i < W::N; ++i) {
    if (W::CH == 1 && lane >= 16) break;
    const int row = row16 + W::row(lane, i), ch = W::chunk(lane, i);
    const uint32_t words[4] = {r.code[i].x, r.code[i].y, r.code[i].z, r.code[i].w};
    uint32_t h[4 * PER / 2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 sc = __hmul2(ca::u2h(r.scale[i * W::BLKS + k * PER / 16]), __floats2half2_rn(0.5f, 1.f));
      const __half2 lo = __low2half2(sc), step = __high2half2(sc);
#pragma unroll
      for (int p = 0; p < PER / 2; ++p) h[k * PER / 2 + p] = ca::h2u(__hfma2(ca::half_code_pair<BITS>(words[k], p, magic), step, lo));
    }
#pragma unroll
    for (int k = 0; k < 4 * PER / 8; ++k)
      sts128(piece_addr(tile, row, ch * (4 * PER / 8) + k), h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
  }
}

}  // namespace ct

// 32 outputs of a row from place c0 on, in the order of the dequantised words: put back in order and
// stored (see store_out), or left as a piece
template <int D, int VB>
__device__ __forceinline__ void store_places(const CacheAttendArgs& A, int r, int j, int c0, const float (&v)[32],
                                             float l, float m) {
  float y[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) y[ct::feature_at(VB, e)] = v[e];
  if (A.prefix_out) {
    const float lp = A.prefix_lse[(long long)r * A.nq + j] * cs::LOG2E, top = fmaxf(m, lp);
    const float f = l == 0.f ? 0.f : cs::ex2(m - top);
    const float g = lp == -INFINITY ? 0.f : cs::ex2(lp - top + cs::SHIFT);
    const float* o = A.prefix_out + ((long long)r * A.nq + j) * D + c0;
    l = fmaf(f, l, g);
#pragma unroll
    for (int e = 0; e < 32; ++e) y[e] = g != 0.f ? fmaf(g, o[e], f * y[e]) : f * y[e];
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const long long at = r * A.o_row + j * A.o_head + c0;
  uint32_t h[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float a = l != 0.f ? y[2 * e] * inv : 0.f, b = l != 0.f ? y[2 * e + 1] * inv : 0.f;
    if (A.q_f16) {
      h[e] = ca::h2u(__floats2half2_rn(a, b));
    } else {
      const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
      h[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  uint16_t* out = reinterpret_cast<uint16_t*>(A.out) + at;
  if (A.o_vec) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      reinterpret_cast<uint4*>(out)[e] = make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      out[2 * e] = (uint16_t)h[e];
      out[2 * e + 1] = (uint16_t)(h[e] >> 16);
    }
  }
}

// PAIR: jobs of 256 rows, 128 for each softmax group, which both use every tile; else jobs of 128
// rows, whose even tiles are the one group's and whose odd tiles the other's.  Tile j of a job lies in
// operand buffers j % 2 either way.
template <int D, int KB, int VB, bool PAIR>
__global__ void __launch_bounds__(ct::THREADS, 1) cache_many_rows_kernel(CacheAttendArgs A) {
  using namespace ct;
  using S = Smem<D>;
  constexpr int ROWS = PAIR ? 256 : 128;
  extern __shared__ unsigned char ct_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)ct_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t bars[17 + 2 * RING];
  __shared__ uint32_t tmem_slot;
  __shared__ int aborted, s_b;
  __shared__ long long s_sum[THREADS / 32], s_base;
  __shared__ longlong2 s_ring[RING][8];                   // {first row in the pool, or -1 for the end; buffer, tokens}
  __shared__ __align__(16) uint16_t s_dead[2][2][8];      // [buffer][parity of its use][16 tokens each]
  __shared__ float s_max[2][2][128];                      // largest |q| of [group][half of the features][row]
  __shared__ float2 s_ml[2][128];                         // maximum and sum of [group][row]
  volatile int* abort_flag = &aborted;
  // the warp's number by a shuffle: so the compiler knows that it, and the roles' branches, are uniform
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t sma = umma::smem_u32(sm), bar0 = umma::smem_u32(bars);
  // barriers of buffer i: K written, K no longer needed, V written, V no longer needed; of group x:
  // S = Q K^T done, P written, Q laid out, the job's last O += P V done; all products done; of the ring
  auto k_full = [&](int i) { return bar0 + 8 * i; };
  auto k_free = [&](int i) { return bar0 + 16 + 8 * i; };
  auto v_full = [&](int i) { return bar0 + 32 + 8 * i; };
  auto v_free = [&](int i) { return bar0 + 48 + 8 * i; };
  auto s_done = [&](int x) { return bar0 + 64 + 8 * x; };
  auto p_full = [&](int x) { return bar0 + 80 + 8 * x; };
  auto q_full = [&](int x) { return bar0 + 96 + 8 * x; };
  auto o_done = [&](int x) { return bar0 + 112 + 8 * x; };
  auto ring_full = [&](int i) { return bar0 + 128 + 8 * i; };
  auto ring_free = [&](int i) { return bar0 + 128 + 8 * (RING + i); };
  const uint32_t drained = bar0 + 128 + 16 * RING;
  auto wait_warp = [&](uint32_t bar, uint32_t parity) {   // by whole warps
    ct::mbar_wait(bar, parity, abort_flag);
    __syncwarp();
  };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      umma::mbar_init(k_full(i), 8);
      umma::mbar_init(k_free(i), 1);
      umma::mbar_init(v_full(i), 8);
      umma::mbar_init(v_free(i), 1);
      umma::mbar_init(s_done(i), 1);
      umma::mbar_init(p_full(i), 4);
      umma::mbar_init(o_done(i), 1);
      umma::mbar_init(q_full(i), PAIR ? 4 : 8);
    }
    for (int i = 0; i < RING; ++i) {
      umma::mbar_init(ring_full(i), 1);
      umma::mbar_init(ring_free(i), 8);
    }
    umma::mbar_init(drained, 1);
    aborted = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  cs::wait_for_predecessor();
  cs::let_successor_start();
  if (tid == 0) A.notes[blockIdx.x] = make_int4(0, 0, -1, 0);
  // ---- this block's range of units ----
  long long total = 0;
  for (int b = tid; b < A.a.B; b += THREADS) total += seq_units<ROWS>(A, b) * A.c.H;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  total = 0;
  for (int k = 0; k < THREADS / 32; ++k) total += s_sum[k];
  const int parts = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= parts) return;   // the whole block
  const long long w0 = cs::range_start(total, parts, blockIdx.x), w1 = cs::range_start(total, parts, blockIdx.x + 1);
  if (warp == 0) {
    long long base = 0;
    for (int b0 = 0; b0 < A.a.B; b0 += 32) {
      const int b = b0 + lane;
      const long long u = b < A.a.B ? seq_units<ROWS>(A, b) * A.c.H : 0;
      long long sum = u;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, k);
        if (lane >= k) sum += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + sum > w0);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          s_b = b;
          s_base = base + sum - u;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(umma::smem_u32(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  Jobs<ROWS> jobs;
  jobs.start(A, w0, w1, s_b, s_base);

  if (warp >= 16) {
    regs_down<ISSUE_REGS>();
    if (warp == 17) {
      // ================= the walk over the tiles =================
      // lanes 0 .. 7: 16 tokens each
      int slot = 0;
      uint32_t round = 0;
      auto publish = [&](long long row, int buf, int live) {
        if (round > 0) wait_warp(ring_free(slot), (round - 1) & 1);
        if (lane < 8) s_ring[slot][lane] = make_longlong2(row, (long long)buf << 32 | (unsigned)live);
        __syncwarp();
        if (lane == 0) arrive(ring_full(slot));
        if (++slot == RING) {
          slot = 0;
          ++round;
        }
      };
      for (; jobs.w < jobs.w1; jobs.next(A))
        for (int tile = jobs.u0; tile < jobs.u1; ++tile) {
          const int t = jobs.s.first + tile * TILE + 16 * (lane & 7);
          long long row = 0;
          int live = 0;
          if (t < jobs.s.len) {
            const int page = page_at(A.a, A.c, jobs.b, t);
            if (page >= 0) {
              row = row_index(A.c, page, jobs.h, t);
              live = min(16, jobs.s.len - t);
            }
          }
          if (lane < 8 && live > 0) {
            // the rows into L2, as far ahead as the ring: the loads to registers are one tile ahead, which
            // covers L2's latency but not that of DRAM
            prefetch_l2(A.c.codes[0] + row * (D * KB / 8), 2 * D * KB);
            prefetch_l2(A.c.scales[0] + row * (D / 16), 4 * D);
            prefetch_l2(A.c.codes[1] + row * (D * VB / 8), 2 * D * VB);
            prefetch_l2(A.c.scales[1] + row * (D / 16), 4 * D);
          }
          __syncwarp();
          publish(row, (tile - jobs.u0) & 1, live);
        }
      publish(-1, 0, 0);
    } else if (warp == 16 && lane == 0) {
      // ================= the products =================
      // (One thread, and a wait only where a phase is new: what this thread spends between two
      // products is time in which none may run.)
      constexpr uint32_t id_s = idesc(128, false), id_o = idesc(D, true);
      const uint64_t kd = umma::smem_desc(sma + S::K, 16, 1024), vd = umma::smem_desc(sma + S::V, BOX, 1024);
      uint32_t k_par = 0u, v_par = 0u, p_par = 0u, q_par = 0u;   // bit i: parity of the next phase of barrier i
      bool go = true;
      auto wait = [&](uint32_t bar, uint32_t parity) { go = ct::mbar_wait(bar, parity, abort_flag) && go; };
      // S = Q K^T of group x with the K of buffer i; first / last: of those who need this K
      auto scores_of = [&](int x, int i, bool first, bool last) {
        if (first) {
          wait(k_full(i), (k_par >> i) & 1);
          k_par ^= 1u << i;
        }
        umma::fence_after_sync();
        const uint64_t qd = umma::smem_desc(sma + (PAIR && x ? S::Q2 : S::Q), 16, 1024);
        const uint64_t kh = kd + (uint64_t)((i * S::OPND) >> 4);
        if (!go) return;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = (uint64_t)(((k / 4) * BOX + (k % 4) * 32) >> 4);
          mma_ss(tmem + 128 * x, qd + off, kh + off, id_s, k != 0);
        }
        umma::mma_commit(s_done(x));
        if (last) umma::mma_commit(k_free(i));
      };
      for (; jobs.w < jobs.w1; jobs.next(A)) {
        const int count = jobs.u1 - jobs.u0;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          if (PAIR || x == 0) {
            wait(q_full(x), (q_par >> x) & 1);
            q_par ^= 1u << x;
          }
          if (PAIR || x < count) scores_of(x, PAIR ? 0 : x, !PAIR || x == 0, !PAIR || x == 1);
        }
#pragma unroll 1
        for (int e = 0; e < (PAIR ? 2 * count : count); ++e) {
          // tile jt, group x: in turn
          const int x = e & 1, jt = PAIR ? e >> 1 : e, i = jt & 1;
          const bool first = !PAIR || x == 0, last = !PAIR || x == 1, more = jt + (PAIR ? 1 : 2) < count;
          wait(p_full(x), (p_par >> x) & 1);
          p_par ^= 1u << x;
          if (first) {
            wait(v_full(i), (v_par >> i) & 1);
            v_par ^= 1u << i;
          }
          umma::fence_after_sync();
          if (go) {
            const uint64_t vh = vd + (uint64_t)((i * S::OPND) >> 4);
#pragma unroll
            for (int kk = 0; kk < TILE / 16; ++kk)
              mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + 8 * kk, vh + (uint64_t)((kk * 2048) >> 4), id_o,
                     (PAIR ? jt : jt >> 1) != 0 || kk != 0);
            if (!more) umma::mma_commit(o_done(x));
            if (last) umma::mma_commit(v_free(i));
          }
          if (more) scores_of(x, PAIR ? i ^ 1 : i, first, last);
        }
      }
      umma::mma_commit(drained);
      if (!umma::mbar_wait(drained, 0)) *abort_flag = 1;
      if (*abort_flag) raise_status(A.a.status, DEV_ERR_TIMEOUT);
    }
  } else if (warp >= 8) {
    // ================= dequantising warps =================
    regs_down<DEQUANT_REGS>();
    const int grp = warp - 8;                  // tokens 16 grp .. + 15 of every tile
    const uint32_t magic = ca::magic512();
    const unsigned char* const kc = A.c.codes[0];
    const unsigned char* const vc = A.c.codes[1];
    const __half2* const ks = A.c.scales[0];
    const __half2* const vs = A.c.scales[1];
    // Tiles are stored as K0 K1 V0 K2 V1 K3 V2 ...: the second group's next scores want K two tiles
    // ahead of the values that the first group's products have yet to release.
    struct Tile {
      long long row;      // of the pool, or -1 behind the last tile
      int live, buf;      // tokens that exist, buffers
    };
    RawRegs rk, rv;
    uint32_t used = 0u, k_par = 0u, v_par = 0u, round = 0;   // bit i: buffer i is in use (+ 2: its V); parities
    int slot = 0;
    auto take = [&]() {                        // the next tile of the walk
      const bool go = __all_sync(0xffffffffu, ct::mbar_wait(ring_full(slot), round & 1, abort_flag));
      const longlong2 e = s_ring[slot][grp];
      const Tile t{go ? e.x : -1, (int)e.y, (int)(e.y >> 32)};
      __syncwarp();
      if (lane == 0) arrive(ring_free(slot));
      if (++slot == RING) {
        slot = 0;
        ++round;
      }
      return t;
    };
    auto load_k = [&](const Tile& t) { raw_load<KB, D>(rk, kc, ks, t.row, lane, t.live); };
    auto load_v = [&](const Tile& t) { raw_load<VB, D>(rv, vc, vs, t.row, lane, t.live); };
    auto store_k = [&](const Tile& t) {
      const int i = t.buf;
      if ((used >> i) & 1u) wait_warp(k_free(i), (k_par >> i & 1u) ^ 1u);
      raw_store<KB, D>(rk, sma + S::K + i * S::OPND, 16 * grp, lane, magic);
      if (lane == 0) s_dead[i][k_par >> i & 1u][grp] = (uint16_t)(0xffffu << t.live);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(k_full(i));
      used |= 1u << i;
      k_par ^= 1u << i;
    };
    auto store_v = [&](const Tile& t) {
      const int i = t.buf;
      if ((used >> i) & 4u) wait_warp(v_free(i), (v_par >> i & 1u) ^ 1u);
      raw_store<VB, D>(rv, sma + S::V + i * S::OPND, 16 * grp, lane, magic);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(v_full(i));
      used |= 4u << i;
      v_par ^= 1u << i;
    };
    const Tile none{-1, 0, 0};
    Tile e0 = take(), e1 = none, e2 = none;
    if (e0.row >= 0) {
      load_k(e0);
      load_v(e0);
      e1 = take();
      store_k(e0);
      if (e1.row >= 0) {
        load_k(e1);
        e2 = take();
        store_k(e1);
        if (e2.row >= 0) load_k(e2);
      }
      for (;;) {
        const Tile e3 = e2.row >= 0 ? take() : none;
        store_v(e0);
        if (e1.row < 0) break;
        load_v(e1);
        if (e2.row >= 0) {
          store_k(e2);
          if (e3.row >= 0) load_k(e3);
        }
        e0 = e1;
        e1 = e2;
        e2 = e3;
      }
    }
  } else {
    regs_up<SOFTMAX_REGS>();
    // ================= softmax warpgroups =================
    const int x = warp >> 2, q4 = warp & 3, trow = 32 * q4 + lane;      // group, TMEM lanes, its row
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const uint32_t ts = tmem + 128 * x + lanes, to = tmem + 256 + 128 * x + lanes;
    const uint32_t qt = sma + (PAIR && x ? S::Q2 : S::Q);
    const bool plain = A.cap == 0.f, biased = A.slopes != nullptr;
    uint32_t s_par = 0u, o_par = 0u, dead_par = 0u;   // parities: of the barriers, and (bit i) of buffer i's use
    for (; jobs.w < jobs.w1; jobs.next(A)) {
      const Seq<ROWS>& s = jobs.s;
      const int old = s.len - s.n, R = s.n * A.G, count = jobs.u1 - jobs.u0;
      const int first_row = jobs.rt * ROWS + (PAIR ? 128 * x : 0), row = first_row + trow;
      const bool is = row < R;
      const int i = is ? row / A.G : 0, jq = jobs.h * A.G + (is ? row % A.G : 0);
      float down;
      // ---- Q: scaled to the top of fp16's range; without PAIR each group lays out half of the features ----
      {
        constexpr int PART = PAIR ? D : D / 2;
        const int f0 = PAIR ? 0 : x * (D / 2);
        float mx = 0.f;
        const long long at = (s.row0 + i) * A.q_row + jq * A.q_head + f0;
        auto load = [&](int k, float (&v)[16]) {
          if (!is) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          } else if (A.q_f16) {
            load_n(reinterpret_cast<const __half*>(A.q) + at + 16 * k, A.q_vec, v);
          } else {
            load_n(reinterpret_cast<const bf16*>(A.q) + at + 16 * k, A.q_vec, v);
          }
        };
#pragma unroll 1
        for (int k = 0; k < PART / 16; ++k) {
          float v[16];
          load(k, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(v[e]));
        }
        if constexpr (!PAIR) {
          s_max[0][x][trow] = mx;
          bar_sync(3, 256);
          mx = fmaxf(s_max[0][0][trow], s_max[0][1][trow]);
        }
        int e2 = 13;
        if (mx > 0.f && mx < INFINITY) e2 = max(ilogbf(mx), -100);
        const float up = ldexpf(1.f, 13 - e2);
        down = ldexpf(1.f, e2 - 13);
#pragma unroll 1
        for (int k = 0; k < PART / 16; ++k) {
          float v[16];
          load(k, v);
          uint32_t h[8];
          // places 2 e and 2 e + 1 of 16 features
#pragma unroll
          for (int e = 0; e < 8; ++e)
            h[e] = ca::h2u(__floats2half2_rn(v[feature_at(KB, 2 * e)] * up, v[feature_at(KB, 2 * e + 1)] * up));
          const int piece = f0 / 8 + 2 * k;
          sts128(piece_addr(qt, trow, piece), h[0], h[1], h[2], h[3]);
          sts128(piece_addr(qt, trow, piece + 1), h[4], h[5], h[6], h[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) arrive(q_full(PAIR ? x : 0));
      const float mult = A.scale * 2.f * down * (plain ? cs::LOG2E : 1.f);      // two: the operands are halves
      const float slope = is && biased ? A.slopes[jq] * cs::LOG2E : 0.f;
      const int pq = A.positions ? A.positions[s.row0 + i] : old + i;
      // keys before `sure` and from `edge` on are seen by every row of the group
      const int i0 = min(first_row / A.G, s.n - 1);
      const int sure = s.causal && !(A.window && A.positions) ? old + i0 + 1 : old;
      int edge = 0;
      if (A.window) {
        int top = old + s.n;
        if (A.positions) {
          top = old;
          for (int k = i0; k <= min(s.n - 1, (first_row + 127) / A.G); ++k) top = max(top, A.positions[s.row0 + k]);
        }
        edge = top - A.window + 1;
      }
      float m_ref = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      const int tiles = PAIR ? count : (count - x + 1) / 2;     // of this group in this part
      for (int k = 0; k < tiles; ++k) {
        const int jt = PAIR ? k : 2 * k + x, i_buf = jt & 1;
        const int t0 = s.first + (jobs.u0 + jt) * TILE;
        // S is there, s_dead (written before the K tile was), and the O += P V of the tile before, which
        // this S was queued behind, is over
        wait_warp(s_done(x), s_par);
        s_par ^= 1u;
        umma::fence_after_sync();
        const volatile uint32_t* dd = reinterpret_cast<const volatile uint32_t*>(s_dead[i_buf][dead_par >> i_buf & 1u]);
        dead_par ^= 1u << i_buf;
        const bool hidden = (dd[0] | dd[1] | dd[2] | dd[3]) != 0u || t0 + TILE > sure || t0 < edge;
        const bool special = hidden || biased || !plain;
        float mx = -INFINITY;
        if (!special) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c0 = 0; c0 < 128; c0 += 64) {
            uint32_t a[32], b[32];
            tmem_ld32_async(ts + c0, a);
            tmem_ld32_async(ts + c0 + 32, b);
            tmem_wait_ld(a, b);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              m4[e & 3] = fmaxf(m4[e & 3], fmaxf(__uint_as_float(a[e]), __uint_as_float(b[e])));
          }
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * mult;
        } else {
          // capped, biased and masked scores in base 2, written back
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            float v[32];
            __syncwarp();
            umma::tmem_ld32(ts + c0, v);
            const int t = t0 + c0;             // v[e]: key t + e
            uint32_t seen = 0xffffffffu;
            if (hidden) {
              seen = ~dd[c0 / 32];
              if (A.window) {
                // keys in the sequence at positions above pq - window; new rows below
                const int lowest = max(pq, old) - A.window + 1 - t;
                const int low = A.positions ? min(lowest, max(old - t, 0)) : lowest;
                if (low >= 32) seen = 0u;
                else if (low > 0) seen &= 0xffffffffu << low;
              }
              if (t + 32 > old) {
                const int j0 = t - old;        // new row of bit 0 (negative: earlier keys)
                uint32_t fresh;                // bits of the new rows that the row sees
                if (!A.mask) {
                  const int upto = i - j0;     // bits 0 .. upto
                  fresh = upto < 0 ? 0u : upto >= 31 ? 0xffffffffu : (2u << upto) - 1u;
                } else {
                  const uint32_t* words = A.mask + (long long)(s.row0 + i) * A.words;
                  const int wi = j0 >> 5, sh = j0 & 31;
                  const uint32_t lo = wi >= 0 && wi < A.words ? words[wi] : 0u;
                  const uint32_t hi = wi + 1 >= 0 && wi + 1 < A.words ? words[wi + 1] : 0u;
                  fresh = __funnelshift_r(lo, hi, sh);
                }
                const uint32_t new_bits = j0 >= 0 ? 0xffffffffu : 0xffffffffu << -j0;
                seen &= ~new_bits | fresh;
                if (A.window && A.positions)
                  for (int e = max(0, -j0); e < 32 && j0 + e < s.n; ++e)
                    if (pq - A.positions[s.row0 + j0 + e] >= A.window) seen &= ~(1u << e);
              }
            }
            const bool by_place = !A.positions || t + 32 <= old;
            const float base = (float)(pq - t);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float y = v[e] * mult;
              if (!plain) y = cap_score(A, y) * cs::LOG2E;
              if (biased) {
                float far = base - (float)e;
                if (!by_place && t + e < s.len) far = (float)(pq - key_position(A, s.row0, old, t + e));
                y = fmaf(-slope, far, y);
              }
              if (!((seen >> e) & 1u)) y = -INFINITY;
              mx = fmaxf(mx, y);
              v[e] = y;
            }
            __syncwarp();
            tmem_st16(ts + c0, *reinterpret_cast<const float(*)[16]>(v));
            tmem_st16(ts + c0 + 16, *reinterpret_cast<const float(*)[16]>(v + 16));
          }
          tmem_wait_st();
        }
        const float mul = special ? 1.f : mult;
        // ---- the reference maximum moves only when it lags: then O and l are rescaled ----
        const bool grow = mx > m_ref + cs::LAG;
        if (__any_sync(0xffffffffu, grow)) {
          const float to_m = fmaxf(mx, m_ref), f = m_ref == -INFINITY ? 0.f : cs::ex2(m_ref - to_m);
          m_ref = to_m;
          l2.x *= f;
          l2.y *= f;
          if (k > 0) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              float v[16];
              tmem_ld16(to + c0, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= f;
              tmem_st16(to + c0, v);
            }
          }
        }
        const float ref = m_ref == -INFINITY ? 0.f : cs::SHIFT - m_ref;
        const float2 mul2 = make_float2(mul, mul), ref2 = make_float2(ref, ref);
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 64) {
          uint32_t a[32], b[32], h[32];
          tmem_ld32_async(ts + c0, a);
          tmem_ld32_async(ts + c0 + 32, b);
          tmem_wait_ld(a, b);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t* v = e < 16 ? a + 2 * e : b + 2 * (e - 16);
            const float2 z = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), mul2, ref2);
            const float2 p = make_float2(cs::ex2(z.x), cs::ex2(z.y));
            l2 = __fadd2_rn(l2, p);
            h[e] = ca::h2u(__floats2half2_rn(p.x, p.y));
          }
          tmem_st32u(ts + c0 / 2, h);
        }
        tmem_wait_st();
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(p_full(x));
      }
      if (tiles > 0) {
        wait_warp(o_done(x), o_par);
        o_par ^= 1u;
      }
      const bool whole = jobs.u0 == 0 && jobs.u1 == jobs.units;
      const float l = l2.x + l2.y;
      const uint32_t o0 = tmem + 256 + lanes, o1 = o0 + 128;
      float f0 = 2.f, f1 = 0.f, top = m_ref, sum = l;        // two: the operands are halves
      int cb = 0, ce = D;
      if constexpr (!PAIR) {
        // the two groups' sums joined, half of the features by each
        s_ml[x][trow] = make_float2(m_ref, l);
        umma::fence_before_sync();
        bar_sync(3, 256);
        umma::fence_after_sync();
        const float2 g0 = s_ml[0][trow], g1 = s_ml[1][trow];
        top = fmaxf(g0.x, g1.x);
        f0 = g0.y == 0.f ? 0.f : 2.f * cs::ex2(g0.x - top);
        f1 = g1.y == 0.f ? 0.f : 2.f * cs::ex2(g1.x - top);
        sum = 0.5f * (g0.y * f0 + g1.y * f1);
        cb = x * (D / 2);
        ce = cb + D / 2;
      } else {
        umma::fence_after_sync();
      }
      float* rec = A.pieces + ((2ll * blockIdx.x + (jobs.u0 == 0 ? 1 : 0)) * ROWS + (row - jobs.rt * ROWS)) * (D + 4);
#pragma unroll 1
      for (int c0 = cb; c0 < ce; c0 += 32) {
        float v[32];
        __syncwarp();
        umma::tmem_ld32((PAIR && x ? o1 : o0) + c0, v);
        if constexpr (PAIR) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = sum != 0.f ? 2.f * v[e] : 0.f;
        } else {
          float v1[32];
          if (count > 1) umma::tmem_ld32(o1 + c0, v1);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float y = f0 != 0.f ? f0 * v[e] : 0.f;
            v[e] = count > 1 && f1 != 0.f ? fmaf(f1, v1[e], y) : y;
          }
        }
        if (!is) continue;
        if (whole) {
          store_places<D, VB>(A, s.row0 + i, jq, c0, v, sum, top);
        } else {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[feature_at(VB, e)] = v[e];
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(rec + c0 + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        }
      }
      if (!whole && is && (PAIR || x == 0)) {
        rec[D] = top;
        rec[D + 1] = sum;
      }
      if (!whole && jobs.u0 == 0 && tid == 0) {
        A.notes[blockIdx.x] = make_int4(
            jobs.b, jobs.h, jobs.rt, cs::pieces_until(total, parts, blockIdx.x, jobs.base + jobs.units));
      }
      // O is read (and, where the groups share it, Q no longer needed) before the next job's products
      umma::fence_before_sync();
      if constexpr (!PAIR) bar_sync(3, 256);
      umma::fence_after_sync();
    }
  }
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    umma::fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

}  // namespace jolt
