// Scored backward kernel instantiations, head dimension 64.
#include "scored_launch.cuh"

namespace fa {
template int launch_bwd_scored<64, kSink>(bool, bool, const CUtensorMap*, const BwdParams&, int, cudaStream_t);
}  // namespace fa
