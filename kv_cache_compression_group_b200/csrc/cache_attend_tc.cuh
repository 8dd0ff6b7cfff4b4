// Attention of many rows per KV head (wide trees, chunks of a prompt) over the paged cache, on the
// 5th-generation tensor cores.
//
// A job is 128 rows (new row x query head) of one KV head; its keys come in tiles of 128 tokens.
// One persistent CTA of 16 warps per SM:
//   * eight dequantising warps take 16 tokens of every tile each: packed codes and (lo, step) pairs
//     straight to registers, one tile ahead, then fp16(lo / 2 + code * (step / 2)) into the
//     128-byte-swizzled operand tiles.  The features of a row keep the order in which a packed
//     word gives its pairs; Q is laid out in the same order, the output columns are put back.
//   * two softmax warpgroups take the even and the odd tiles of the job, each with operand tiles,
//     score and output accumulators, maximum and sum of its own (all 512 columns of tensor
//     memory), so that one group's exponentials overlap the other's products.  A thread has one
//     row: it reads its scores twice (maximum, then weights), writes the weights as fp16 over the
//     scores, and when its group has, one elected thread issues O += P V (P from tensor memory)
//     and the group's next S = Q K^T.  The reference maximum may lag by 2^8, so rescaling O, a pass
//     through tensor memory, is rare after the first tiles.
//   * at the end both groups' outputs are joined, half of the columns by each group.
// What bounds it at D = 128: the two products take 1024 cycles per tile, its 16384 exponentials
// 1024 at 16 per cycle, and the instructions of softmax and dequantisation about 1200 per scheduler.
//
// Every wait is bounded; after one gave up, the roles keep their barrier schedule without waiting or
// issuing, so the CTA ends, and the issued products are drained before tensor memory is freed.
#pragma once

#include "cache_attend.cuh"
#include "umma.cuh"

namespace jolt {
namespace ct {
constexpr int ROWS = 128, TILE = 128;
constexpr int THREADS = 512;
constexpr int BOX = 128 * 128;                 // bytes of 128 rows x 64 fp16 features
template <int D>
struct Smem {
  static constexpr int OPND = D / 64 * BOX;    // bytes of a 128 x D operand tile
  static constexpr int Q = 0, K = OPND, V = 3 * OPND, MISC = 5 * OPND;
  static constexpr int BYTES = MISC + 4096 + 1024;
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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
      ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
        "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]),
        "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]),
        "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 16-byte piece `piece` (8 features) of row `row` of an operand tile
__device__ __forceinline__ uint32_t piece_addr(uint32_t tile, int row, int piece) {
  return tile + (piece >> 3) * BOX + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}
// feature at place p of a row as the dequantised words hold it
__device__ __forceinline__ int feature_at(int bits, int p) {
  const int per = 32 / bits, in = p & (per - 1);
  return (p - in) + (in >> 1) + (in & 1) * (per >> 1);
}

// one sequence's jobs
struct Seq {
  int row0, n, len, first, tiles;      // tiles: of 128 rows
  bool causal;
  // units of row tile rt: the keys that any of its rows may see
  __device__ int units(const CacheAttendArgs& A, int rt) const {
    int end = len;
    if (causal) end = min(len, len - n + min(n, ((rt + 1) * ROWS - 1) / A.G + 1));
    return (end - first + TILE - 1) / TILE;
  }
};
__device__ __forceinline__ bool load_seq(const CacheAttendArgs& A, int b, Seq& s) {
  const int u = cache_units(A, b, TILE, s.row0, s.n, s.len, s.first);
  if (u == 0) return false;
  s.tiles = (int)(((long long)s.n * A.G + ROWS - 1) / ROWS);
  s.causal = A.mask == nullptr;
  return true;
}
__device__ __forceinline__ long long seq_units(const CacheAttendArgs& A, int b) {
  Seq s;
  if (!load_seq(A, b, s)) return 0;
  if (!s.causal) return (long long)s.tiles * s.units(A, 0);
  long long sum = 0;
  for (int rt = 0; rt < s.tiles; ++rt) sum += s.units(A, rt);
  return sum;
}

// The jobs of a block's range [w, w1), in order; every thread walks its own copy.
struct Jobs {
  long long w, w1, base;   // base: first unit of (b, h, rt)
  int b, h, rt;
  Seq s;
  int units, u0, u1;       // of the job, and of this block's part of it
  __device__ void start(const CacheAttendArgs& A, long long from, long long to, int b0, long long b0_base) {
    w = from;
    w1 = to;
    b = b0;
    base = b0_base;
    h = rt = 0;
    if (w >= w1) return;
    load_seq(A, b, s);
    const long long per = seq_units(A, b);
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
struct RawRegs {
  uint4 code[4];
  uint32_t scale[4];
};

template <int BITS, int D>
__device__ __forceinline__ void raw_load(RawRegs& r, const unsigned char* codes, const __half2* scales, int lane,
                                         int live) {
  using W = Raw<BITS, D>;
#pragma unroll
  for (int i = 0; i < W::N; ++i) {
    const int row = W::row(lane, i), ch = W::chunk(lane, i);
    r.code[i] = make_uint4(0u, 0u, 0u, 0u);
    const bool on = row < live && (W::CH > 1 || lane < 16);
    if (on) r.code[i] = __ldg(reinterpret_cast<const uint4*>(codes + row * (D * BITS / 8) + ch * 16));
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(scales + row * (D / 16) + ch * W::BLKS);
    if constexpr (W::BLKS == 1) {
      r.scale[i] = on ? __ldg(sc) : 0u;
    } else if constexpr (W::BLKS == 2) {
      const uint2 v = on ? __ldg(reinterpret_cast<const uint2*>(sc)) : make_uint2(0u, 0u);
      r.scale[2 * i] = v.x;
      r.scale[2 * i + 1] = v.y;
    } else {
      const uint4 v = on ? __ldg(reinterpret_cast<const uint4*>(sc)) : make_uint4(0u, 0u, 0u, 0u);
      r.scale[0] = v.x;
      r.scale[1] = v.y;
      r.scale[2] = v.z;
      r.scale[3] = v.w;
    }
  }
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
      const __half2 sc = __hmul2(ca::u2h(r.scale[i * W::BLKS + k * PER / 16]), __float2half2_rn(0.5f));
      const __half2 lo = __low2half2(sc), step = __high2half2(sc);
#pragma unroll
      for (int p = 0; p < PER / 2; ++p) h[k * PER / 2 + p] = ca::h2u(__hfma2(ca::code_pair<BITS>(words[k], p, magic), step, lo));
    }
#pragma unroll
    for (int k = 0; k < 4 * PER / 8; ++k)
      sts128(piece_addr(tile, row, ch * (4 * PER / 8) + k), h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
  }
}

template <int D>
__device__ __forceinline__ void load_bits(RawRegs& r, const CacheArgs& c, int kv, long long row, int lane, int live) {
  const int bits = c.bits[kv];
  const unsigned char* codes = c.codes[kv] + row * (D * bits / 8);
  const __half2* scales = c.scales[kv] + row * (D / 16);
  if (bits == 4) raw_load<4, D>(r, codes, scales, lane, live);
  else if (bits == 8) raw_load<8, D>(r, codes, scales, lane, live);
  else raw_load<2, D>(r, codes, scales, lane, live);
}
template <int D>
__device__ __forceinline__ void store_bits(const RawRegs& r, int bits, uint32_t tile, int row16, int lane,
                                           uint32_t magic) {
  if (bits == 4) raw_store<4, D>(r, tile, row16, lane, magic);
  else if (bits == 8) raw_store<8, D>(r, tile, row16, lane, magic);
  else raw_store<2, D>(r, tile, row16, lane, magic);
}
}  // namespace ct

template <int D>
__global__ void __launch_bounds__(ct::THREADS, 1) cache_many_rows_kernel(CacheAttendArgs A) {
  using namespace ct;
  using S = Smem<D>;
  extern __shared__ unsigned char ct_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)ct_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::MISC);      // 10 barriers
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::MISC + 96);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::MISC + 100);
  volatile uint16_t* dead = reinterpret_cast<volatile uint16_t*>(sm + S::MISC + 128);   // [group][parity][8]
  long long* s_sum = reinterpret_cast<long long*>(sm + S::MISC + 256);                  // [16]
  long long* s_base = s_sum + 16;
  int* s_b = reinterpret_cast<int*>(s_base + 1);
  float* s_max = reinterpret_cast<float*>(sm + S::MISC + 512);                          // [2][128]
  float* s_ml = s_max + 256;                                                            // [2][128][2]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sma = umma::smem_u32(sm), bar0 = umma::smem_u32(bars);
  // barriers of group x: K tile written, S = Q K^T done, V tile written, O += P V done
  auto k_full = [&](int x) { return bar0 + 8 * x; };
  auto s_done = [&](int x) { return bar0 + 16 + 8 * x; };
  auto v_full = [&](int x) { return bar0 + 32 + 8 * x; };
  auto o_done = [&](int x) { return bar0 + 48 + 8 * x; };
  auto drain = [&](int x) { return bar0 + 64 + 8 * x; };
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (*abort_flag) return false;
    if (umma::mbar_wait(bar, parity)) return true;
    *abort_flag = 1;
    return false;
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity) {   // by whole warps
    wait(bar, parity);
    __syncwarp();
  };

  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      umma::mbar_init(k_full(x), 8);
      umma::mbar_init(s_done(x), 1);
      umma::mbar_init(v_full(x), 8);
      umma::mbar_init(o_done(x), 1);
      umma::mbar_init(drain(x), 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    A.notes[blockIdx.x] = make_int4(0, 0, -1, 0);
  }
  // ---- this block's range of units ----
  long long total = 0;
  for (int b = tid; b < A.a.B; b += THREADS) total += seq_units(A, b) * A.c.H;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  total = 0;
  for (int k = 0; k < 16; ++k) total += s_sum[k];
  const int parts = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= parts) return;   // the whole block
  const long long w0 = cs::range_start(total, parts, blockIdx.x), w1 = cs::range_start(total, parts, blockIdx.x + 1);
  if (warp == 0) {
    long long base = 0;
    for (int b0 = 0; b0 < A.a.B; b0 += 32) {
      const int b = b0 + lane;
      const long long u = b < A.a.B ? seq_units(A, b) * A.c.H : 0;
      long long sum = u;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, k);
        if (lane >= k) sum += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + sum > w0);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          *s_b = b;
          *s_base = base + sum - u;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(umma::smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Jobs jobs;
  jobs.start(A, w0, w1, *s_b, *s_base);

  if (warp >= 8) {
    // ================= dequantising warps =================
    const int grp = warp - 8;                  // tokens 16 grp .. + 15 of every tile
    const uint32_t magic = ca::magic1024();
    RawRegs rk, rv;
    int tile = jobs.u0, j = 0;                 // tile of the job; its number in this block's part
    bool more = jobs.w < jobs.w1;
    uint32_t uses[2] = {0u, 0u};
    unsigned live = 0;                         // tokens of the 16 that exist
    long long row = 0;
    auto locate = [&]() {                      // the current tile's rows in the pool
      const int t = jobs.s.first + tile * TILE + 16 * grp;
      live = 0;
      if (t < jobs.s.len) {
        const int page = page_at(A.a, A.c, jobs.b, t);
        if (page >= 0) {
          row = row_index(A.c, page, jobs.h, t);
          live = min(16, jobs.s.len - t);
        }
      }
    };
    if (more) {
      locate();
      load_bits<D>(rk, A.c, 0, row, lane, live);
      load_bits<D>(rv, A.c, 1, row, lane, live);
    }
    while (more) {
      const int x = j & 1;
      const unsigned now_live = live;
      if (uses[x]) wait_warp(s_done(x), (uses[x] - 1) & 1);
      store_bits<D>(rk, A.c.bits[0], sma + S::K + x * S::OPND, 16 * grp, lane, magic);
      if (lane == 0) dead[(2 * x + (uses[x] & 1)) * 8 + grp] = (uint16_t)(0xffffu << now_live);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(k_full(x));
      // the next tile, its keys under way before the values of this one
      ++tile;
      ++j;
      if (tile == jobs.u1) {
        jobs.next(A);
        more = jobs.w < jobs.w1;
        tile = jobs.u0;
        j = 0;
      }
      if (more) {
        locate();
        load_bits<D>(rk, A.c, 0, row, lane, live);
      }
      if (uses[x]) wait_warp(o_done(x), (uses[x] - 1) & 1);
      store_bits<D>(rv, A.c.bits[1], sma + S::V + x * S::OPND, 16 * grp, lane, magic);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(v_full(x));
      ++uses[x];
      if (more) load_bits<D>(rv, A.c, 1, row, lane, live);
    }
  } else {
    // ================= softmax warpgroups =================
    const int x = warp >> 2, q4 = warp & 3, trow = 32 * q4 + lane;      // group, TMEM lanes, row of the tile
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const uint32_t ts = tmem + 128 * x + lanes, to = tmem + 256 + 128 * x + lanes;
    const bool plain = A.cap == 0.f, biased = A.slopes != nullptr;
    const bool issuer = (tid & 127) == 0;
    const uint32_t id_s = idesc(128, false), id_o = idesc(D, true);
    uint32_t uses = 0;                         // tiles of this group so far
    auto issue_scores = [&]() {                // next S = Q K^T of this group; its tile is use number `uses`
      if (!wait(k_full(x), uses & 1)) return;
      umma::fence_after_sync();
      const uint32_t kt = sma + S::K + x * S::OPND;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k / 4) * BOX + (k % 4) * 32;
        mma_ss(tmem + 128 * x, umma::smem_desc(sma + S::Q + off, 16, 1024), umma::smem_desc(kt + off, 16, 1024), id_s,
               k != 0);
      }
      umma::mma_commit(s_done(x));
    };
    for (; jobs.w < jobs.w1; jobs.next(A)) {
      const Seq& s = jobs.s;
      const int old = s.len - s.n, R = s.n * A.G, count = jobs.u1 - jobs.u0;
      const int row = jobs.rt * ROWS + trow;
      const bool is = row < R;
      const int i = is ? row / A.G : 0, jq = jobs.h * A.G + (is ? row % A.G : 0);
      float down;
      // ---- Q: row trow, half x of its features, scaled to the top of fp16's range ----
      {
        float mx = 0.f;
        const long long at = (s.row0 + i) * A.q_row + jq * A.q_head + x * (D / 2);
        const bool vec = A.q_vec;
        for (int k = 0; k < D / 32; ++k) {
          float v[16];
          if (!is) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          } else if (A.q_f16) load_n(reinterpret_cast<const __half*>(A.q) + at + 16 * k, vec, v);
          else load_n(reinterpret_cast<const bf16*>(A.q) + at + 16 * k, vec, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(v[e]));
        }
        s_max[128 * x + trow] = mx;
        bar_sync(3, 256);                      // and: the previous job's Q and sums are read
        mx = fmaxf(s_max[trow], s_max[128 + trow]);
        int e2 = 13;
        if (mx > 0.f && mx < INFINITY) e2 = max(ilogbf(mx), -100);
        const float up = ldexpf(1.f, 13 - e2);
        down = ldexpf(1.f, e2 - 13);
        for (int k = 0; k < D / 32; ++k) {
          float v[16];
          if (!is) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          } else if (A.q_f16) load_n(reinterpret_cast<const __half*>(A.q) + at + 16 * k, vec, v);
          else load_n(reinterpret_cast<const bf16*>(A.q) + at + 16 * k, vec, v);
          uint32_t h[8];
          const int bk = A.c.bits[0];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // places 2 e and 2 e + 1 of 16 features (feature_at, for each packing)
            const float a4 = v[(e / 4) * 8 + (e & 3)], b4 = v[(e / 4) * 8 + (e & 3) + 4];
            const float a8 = v[(e / 2) * 4 + (e & 1)], b8 = v[(e / 2) * 4 + (e & 1) + 2];
            const float a = bk == 4 ? a4 : bk == 8 ? a8 : v[e], b = bk == 4 ? b4 : bk == 8 ? b8 : v[e + 8];
            h[e] = ca::h2u(__floats2half2_rn(a * up, b * up));
          }
          const int piece = x * (D / 16) + 2 * k;
          sts128(piece_addr(sma + S::Q, trow, piece), h[0], h[1], h[2], h[3]);
          sts128(piece_addr(sma + S::Q, trow, piece + 1), h[4], h[5], h[6], h[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      bar_sync(3, 256);
      const float mult = A.scale * 2.f * down * (plain ? cs::LOG2E : 1.f);      // two: the operands are halves
      const float slope = is && biased ? A.slopes[jq] * cs::LOG2E : 0.f;
      const int pq = A.positions ? A.positions[s.row0 + i] : old + i;
      // keys before `sure` and from `edge` on are seen by every row of the tile
      const int i0 = jobs.rt * ROWS / A.G;
      const int sure = s.causal && !(A.window && A.positions) ? old + min(s.n, i0 + 1) : old;
      int edge = 0;
      if (A.window) {
        int top = old + s.n;
        if (A.positions) {
          top = old;
          for (int k = i0; k <= min(s.n - 1, (jobs.rt * ROWS + ROWS - 1) / A.G); ++k)
            top = max(top, A.positions[s.row0 + k]);
        }
        edge = top - A.window + 1;
      }
      float m_ref = -INFINITY, l = 0.f;
      const int mine = (count - x + 1) / 2;    // tiles x, x + 2, ... of the part
      if (issuer && mine > 0) issue_scores();
      for (int k = 0; k < mine; ++k, ++uses) {
        const int t0 = s.first + (jobs.u0 + 2 * k + x) * TILE;
        wait_warp(s_done(x), uses & 1);        // S is there, and `dead`, written before the K tile was
        umma::fence_after_sync();
        const volatile uint32_t* dd = reinterpret_cast<const volatile uint32_t*>(dead + (2 * x + (uses & 1)) * 8);
        const uint32_t d4[4] = {dd[0], dd[1], dd[2], dd[3]};
        const bool hidden = (d4[0] | d4[1] | d4[2] | d4[3]) != 0u || t0 + TILE > sure || t0 < edge;
        const bool special = hidden || biased || !plain;
        float mx = -INFINITY;
        if (!special) {
#pragma unroll
          for (int c0 = 0; c0 < 128; c0 += 32) {
            float v[32];
            umma::tmem_ld32(ts + c0, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, v[e]);
          }
          mx *= mult;
        } else {
          // capped, biased and masked scores in base 2, written back
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            float v[32];
            umma::tmem_ld32(ts + c0, v);
            uint32_t seen = 0xffffffffu;
            if (hidden) {
              seen = ~d4[c0 / 32];
              const int t = t0 + c0;           // bit e: key t + e
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
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float y = v[e] * mult;
              if (!plain) y = cap_score(y, A.cap) * cs::LOG2E;
              v[e] = y;
            }
            if (biased) {
              const bool by_place = !A.positions || t0 + c0 + 32 <= old;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int t = t0 + c0 + e;
                const int pk = by_place ? t : (t < s.len ? key_position(A, s.row0, old, t) : 0);
                v[e] = fmaf(-slope, (float)(pq - pk), v[e]);
              }
            }
            if (hidden) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = (seen >> e) & 1u ? v[e] : -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, v[e]);
            tmem_st32(ts + c0, v);
          }
          tmem_wait_st();
        }
        const float mul = special ? 1.f : mult;
        // ---- the reference maximum moves only when it lags: then O and l are rescaled ----
        const bool grow = mx > m_ref + cs::LAG;
        if (__any_sync(0xffffffffu, grow)) {
          const float to_m = fmaxf(mx, m_ref), f = m_ref == -INFINITY ? 0.f : cs::ex2(m_ref - to_m);
          m_ref = to_m;
          l *= f;
          if (k > 0) {
            wait_warp(o_done(x), (uses - 1) & 1);
            umma::fence_after_sync();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              float v[32];
              umma::tmem_ld32(to + c0, v);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] *= f;
              tmem_st32(to + c0, v);
            }
            tmem_wait_st();
          }
        }
        const float ref = m_ref == -INFINITY ? 0.f : cs::SHIFT - m_ref;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          float v[32];
          umma::tmem_ld32(ts + c0, v);
          uint32_t h[16];
          float a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = cs::ex2(fmaf(v[2 * e], mul, ref)), p1 = cs::ex2(fmaf(v[2 * e + 1], mul, ref));
            a0 += p0;
            a1 += p1;
            h[e] = ca::h2u(__floats2half2_rn(p0, p1));
          }
          l += a0 + a1;
          tmem_st16(ts + c0 / 2, h);
        }
        tmem_wait_st();
        umma::fence_before_sync();
        bar_sync(1 + x, 128);
        if (issuer) {
          umma::fence_after_sync();
          if (wait(v_full(x), uses & 1)) {
            umma::fence_after_sync();
            const uint32_t vt = sma + S::V + x * S::OPND;
#pragma unroll
            for (int kk = 0; kk < TILE / 16; ++kk)
              mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + 8 * kk, umma::smem_desc(vt + kk * 2048, BOX, 1024), id_o,
                     (k | kk) != 0);
            umma::mma_commit(o_done(x));
          }
          if (k + 1 < mine) {
            ++uses;
            issue_scores();
            --uses;
          }
        }
      }
      // ---- the two groups' sums joined, half of the features by each ----
      if (mine > 0) wait_warp(o_done(x), (uses - 1) & 1);
      s_ml[2 * (128 * x + trow)] = m_ref;
      s_ml[2 * (128 * x + trow) + 1] = l;
      umma::fence_before_sync();
      bar_sync(3, 256);
      umma::fence_after_sync();
      const float m0 = s_ml[2 * trow], l0 = s_ml[2 * trow + 1], m1 = s_ml[2 * (128 + trow)], l1 = s_ml[2 * (128 + trow) + 1];
      const float top = fmaxf(m0, m1);
      const float f0 = l0 == 0.f ? 0.f : cs::ex2(m0 - top), f1 = l1 == 0.f ? 0.f : cs::ex2(m1 - top);
      const float sum = l0 * f0 + l1 * f1;
      const bool whole = jobs.u0 == 0 && jobs.u1 == jobs.units, two = count > 1;
      float* rec = A.pieces + ((2ll * blockIdx.x + (jobs.u0 == 0 ? 1 : 0)) * ROWS + trow) * (D + 4);
      const uint32_t o0 = tmem + 256 + lanes, o1 = o0 + 128;
#pragma unroll 1
      for (int c0 = x * (D / 2); c0 < (x + 1) * (D / 2); c0 += 32) {
        float v[32], v1[32];
        __syncwarp();
        umma::tmem_ld32(o0 + c0, v);
        if (two) umma::tmem_ld32(o1 + c0, v1);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float y = f0 != 0.f ? 2.f * f0 * v[e] : 0.f;       // two: the operands are halves
          if (two && f1 != 0.f) y = fmaf(2.f * f1, v1[e], y);
          v[e] = y;
        }
        if (!is) continue;
        const int bv = A.c.bits[1];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int d = feature_at(bv, c0 + e);
          if (whole) store_out(A, D, s.row0 + i, jq, d, v[e], sum, top);
          else rec[d] = v[e];
        }
      }
      if (!whole && is && x == 0) {
        rec[D] = top;
        rec[D + 1] = sum;
      }
      if (!whole && jobs.u0 == 0 && tid == 0) {
        A.notes[blockIdx.x] = make_int4(
            jobs.b, jobs.h, jobs.rt, cs::pieces_until(total, parts, blockIdx.x, jobs.base + jobs.units));
      }
      umma::fence_before_sync();
      bar_sync(3, 256);     // O is read before the next job's first product writes it
      umma::fence_after_sync();
    }
    if (issuer) {
      umma::mma_commit(drain(x));
      if (!umma::mbar_wait(drain(x), 0)) *abort_flag = 1;
      if (*abort_flag) raise_status(A.a.status, DEV_ERR_TIMEOUT);
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    umma::fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

}  // namespace jolt
