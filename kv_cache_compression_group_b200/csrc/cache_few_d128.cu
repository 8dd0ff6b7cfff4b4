// The narrow cache attention kernels for head_dim 128, all bit-widths.
#include "cache_launch.cuh"

namespace jolt {
template <>
jolt_status launch_few_rows<128>(const CacheAttendArgs& A, cudaStream_t st) {
  return launch_few_bits<128>(A, st);
}
}  // namespace jolt
