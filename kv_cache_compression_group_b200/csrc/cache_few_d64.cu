// The narrow cache attention kernel for head_dim 64, all bit-widths.
#include "cache_launch.cuh"

namespace jolt {
template <>
jolt_status launch_few_rows<64>(const CacheAttendArgs& A, int nt, cudaStream_t st) {
  return nt == 1 ? launch_few_bits<64, 1>(A, st) : nt == 2 ? launch_few_bits<64, 2>(A, st) : launch_few_bits<64, 4>(A, st);
}
}  // namespace jolt
