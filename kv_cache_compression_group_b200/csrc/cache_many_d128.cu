// The tensor-core cache attention kernel for head_dim 128, all bit-widths.
#include "cache_launch.cuh"

namespace jolt {
template <>
jolt_status launch_many_rows<128>(const CacheAttendArgs& A, bool pair, cudaStream_t st) {
  return pair ? launch_many_bits<128, true>(A, st) : launch_many_bits<128, false>(A, st);
}
}  // namespace jolt
