// Launch of the cache attention kernels: which kernel takes how many rows, how many blocks, and
// the join behind it.  The kernels' instances for every pair of bit-widths are compiled in
// sources of their own, beside one another.
#pragma once

#include "cache_attend.cuh"
#include "cache_attend_codes.cuh"
#include "cache_attend_tc.cuh"
#include "host.cuh"

namespace jolt {

// Rows of one KV head that the narrow kernels take.  32 rows of 8 KV heads there and in the tensor-core kernel,
// whose tiles have 128 rows, in us, at 2, 4 and 8 bits:
//   16 sequences of 8192 tokens:  D = 64: 80, 84, 88 and 119, 109, 112;  D = 128: 121, 127, 131 and 131, 135, 152
//   one of 65536 tokens:          D = 64: 49, 49, 52 and 70, 64, 68;     D = 128: 66, 71, 74 and 80, 91, 96
//   one of 2000 tokens:           D = 64: 22.7 and 20.7;                 D = 128: 27 and 27
// With 17 rows the narrow ones take 5 to 10 % less, the other as long.
inline constexpr int FEW_ROWS = 32;

inline constexpr int MANY_BLOCKS = 148;   // of the tensor-core kernel: one per SM

// What the scratch holds for calls with so many rows of a KV head: pieces of this many blocks, two of each, of this
// many rows.  Every launch asserts that its blocks and pieces fit.
inline constexpr int scratch_blocks(long long rows) { return rows > FEW_ROWS ? MANY_BLOCKS : 148 * (rows <= 16 ? 4 : 2); }
inline constexpr int scratch_rows(long long rows) {
  return rows > 128 ? 256 : rows > FEW_ROWS ? 128 : rows <= 16 ? 16 : 32;
}
inline constexpr bool scratch_fits(int blocks, int piece_rows, long long rows) {
  return blocks <= scratch_blocks(rows) && blocks * piece_rows <= scratch_blocks(rows) * scratch_rows(rows);
}

template <int D, int NT, int KB, int VB>
jolt_status launch_codes(const CacheAttendArgs& A, cudaStream_t st) {
  using S = cc::Smem<D, NT, KB, VB>;
  constexpr int blocks = 148 * cc::blocks_per_sm<D, NT, KB, VB>();
  static_assert(blocks <= JOIN_MOST && scratch_fits(blocks, S::ROWS, S::ROWS));
  CUDA_TRY(cudaFuncSetAttribute(cache_codes_kernel<D, NT, KB, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES));
  CUDA_TRY(launch_after(cache_codes_kernel<D, NT, KB, VB>, dim3(blocks), S::WARPS * 32, S::BYTES, st, A));
  CUDA_TRY(launch_after(cache_join_kernel<D, S::ROWS>, dim3(blocks, (unsigned)ceil_div(A.a.max_new * A.G, 512 / D)), 512, 0, st, A));
  return JOLT_OK;
}

// As many blocks as the GPU holds at once: by registers 4, 3 or 2 per SM, by shared memory what 228 KB hold with
// 1 KB reserved for each.
template <int D, int NT, int KB, int VB>
jolt_status launch_few(const CacheAttendArgs& A, cudaStream_t st) {
  constexpr int smem = ca::Smem<D, NT>::bytes(KB, VB);
  constexpr int by_regs = NT == 1 ? 4 : NT == 2 ? 3 : 2, by_smem = 228 * 1024 / (smem + 1024);
  constexpr int blocks = 148 * (by_regs < by_smem ? by_regs : by_smem);
  static_assert(blocks <= JOIN_MOST && scratch_fits(blocks, 8 * NT, 8 * NT));
  CUDA_TRY(cudaFuncSetAttribute(cache_few_rows_kernel<D, NT, KB, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  CUDA_TRY(launch_after(cache_few_rows_kernel<D, NT, KB, VB>, dim3(blocks), ca::WARPS * 32, smem, st, A));
  CUDA_TRY(launch_after(cache_join_kernel<D, 8 * NT>, dim3(blocks, (unsigned)ceil_div(A.a.max_new * A.G, 512 / D)), 512, 0, st, A));
  return JOLT_OK;
}

template <int D, int KB, int VB, bool PAIR>
jolt_status launch_many(const CacheAttendArgs& A, cudaStream_t st) {
  constexpr int smem = ct::Smem<D>::bytes(PAIR), rows = PAIR ? 256 : 128;
  static_assert(scratch_fits(MANY_BLOCKS, rows, rows));
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, cache_many_rows_kernel<D, KB, VB, PAIR>) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < ct::LAUNCH_REGS) return fail(JOLT_ERR_CUDA, "the kernel has %d registers at its launch, needs %d", regs, ct::LAUNCH_REGS);
  CUDA_TRY(cudaFuncSetAttribute(cache_many_rows_kernel<D, KB, VB, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  CUDA_TRY(launch_after(cache_many_rows_kernel<D, KB, VB, PAIR>, dim3(MANY_BLOCKS), ct::THREADS, smem, st, A));
  CUDA_TRY(launch_after(cache_join_rows_kernel<D, rows>, dim3(MANY_BLOCKS, rows / 8), 256, 0, st, A));
  return JOLT_OK;
}

template <int D, bool PAIR>
jolt_status launch_many_bits(const CacheAttendArgs& A, cudaStream_t st) {
  switch (A.c.bits[0] * 16 + A.c.bits[1]) {
    case 0x22: return launch_many<D, 2, 2, PAIR>(A, st);
    case 0x24: return launch_many<D, 2, 4, PAIR>(A, st);
    case 0x28: return launch_many<D, 2, 8, PAIR>(A, st);
    case 0x42: return launch_many<D, 4, 2, PAIR>(A, st);
    case 0x44: return launch_many<D, 4, 4, PAIR>(A, st);
    case 0x48: return launch_many<D, 4, 8, PAIR>(A, st);
    case 0x82: return launch_many<D, 8, 2, PAIR>(A, st);
    case 0x84: return launch_many<D, 8, 4, PAIR>(A, st);
    default: return launch_many<D, 8, 8, PAIR>(A, st);
  }
}

// A few rows: the codes' kernel where they fit two of its n-tiles, else the other.  (8 sequences of up to
// 8192 tokens, 8 KV heads, D = 128, 4 bits: 31 us for 4 rows and 39 us for 8 with one and two n-tiles;
// with four, 60 us for 12 rows, where the other kernel, which prepares its operands once for all rows,
// takes about 40 us.)
template <int D, int KB, int VB>
jolt_status launch_few_rows_of(const CacheAttendArgs& A, cudaStream_t st) {
  constexpr int R = cc::rows_of(KB, VB);
  const long long rows = (long long)A.a.max_new * A.G;
  if (rows <= R) return launch_codes<D, 1, KB, VB>(A, st);
  if (rows <= 2 * R) return launch_codes<D, 2, KB, VB>(A, st);
  if constexpr (R == 2)
    if (rows <= 8) return launch_few<D, 1, KB, VB>(A, st);
  if constexpr (R < 8)
    if (rows <= 16) return launch_few<D, 2, KB, VB>(A, st);
  return launch_few<D, 4, KB, VB>(A, st);
}

template <int D>
jolt_status launch_few_bits(const CacheAttendArgs& A, cudaStream_t st) {
  switch (A.c.bits[0] * 16 + A.c.bits[1]) {
    case 0x22: return launch_few_rows_of<D, 2, 2>(A, st);
    case 0x24: return launch_few_rows_of<D, 2, 4>(A, st);
    case 0x28: return launch_few_rows_of<D, 2, 8>(A, st);
    case 0x42: return launch_few_rows_of<D, 4, 2>(A, st);
    case 0x44: return launch_few_rows_of<D, 4, 4>(A, st);
    case 0x48: return launch_few_rows_of<D, 4, 8>(A, st);
    case 0x82: return launch_few_rows_of<D, 8, 2>(A, st);
    case 0x84: return launch_few_rows_of<D, 8, 4>(A, st);
    default: return launch_few_rows_of<D, 8, 8>(A, st);
  }
}

// up to FEW_ROWS rows of a KV head, and the join
template <int D>
jolt_status launch_few_rows(const CacheAttendArgs& A, cudaStream_t st);

// the tensor-core kernel with jobs of 128 rows or (pair) 256, and its join
template <int D>
jolt_status launch_many_rows(const CacheAttendArgs& A, bool pair, cudaStream_t st);

}  // namespace jolt
