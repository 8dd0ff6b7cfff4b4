// The tensor-core cache attention kernel for head_dim 64, all bit-widths.
#include "cache_launch.cuh"

namespace jolt {
template <>
jolt_status launch_many_rows<64>(const CacheAttendArgs& A, bool pair, cudaStream_t st) {
  return pair ? launch_many_bits<64, true>(A, st) : launch_many_bits<64, false>(A, st);
}
}  // namespace jolt
