// Scored forward kernel instantiations over a paged K/V cache, head dimension 256.
#include "scored_launch.cuh"

namespace fa {
template int launch_fwd_paged_scored<256, kSinkCap>(bool, bool, const CUtensorMap*, const FwdParams&, int, cudaStream_t);
}  // namespace fa
