// The narrow cache attention kernel for head_dim 128, all bit-widths.
#include "cache_launch.cuh"

namespace jolt {
template <>
jolt_status launch_few_rows<128>(const CacheAttendArgs& A, int nt, cudaStream_t st) {
  return nt == 1 ? launch_few_bits<128, 1>(A, st) : nt == 2 ? launch_few_bits<128, 2>(A, st) : launch_few_bits<128, 4>(A, st);
}
}  // namespace jolt
