// Scored forward kernel instantiations over a paged K/V cache, head dimension 128.
#include "scored_launch.cuh"

namespace fa {
template int launch_fwd_paged_scored<128, kBias>(bool, bool, const CUtensorMap*, const FwdParams&, int, cudaStream_t);
}  // namespace fa
