// Scored backward kernel instantiations, head dimension 128.
#include "scored_launch.cuh"

namespace fa {
template int launch_bwd_scored<128, kCapBias>(bool, bool, const CUtensorMap*, const BwdParams&, int, cudaStream_t);
}  // namespace fa
