// The narrow cache attention kernels for head_dim 64, all bit-widths.
#include "cache_launch.cuh"

namespace jolt {
template <>
jolt_status launch_few_rows<64>(const CacheAttendArgs& A, cudaStream_t st) {
  return launch_few_bits<64>(A, st);
}
}  // namespace jolt
