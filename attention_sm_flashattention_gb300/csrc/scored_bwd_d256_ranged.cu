// Scored backward kernel instantiations, head dimension 256.
#include "scored_launch.cuh"

namespace fa {
template int launch_bwd_scored<256, kRanged>(bool, bool, const CUtensorMap*, const BwdParams&, int, cudaStream_t);
}  // namespace fa
