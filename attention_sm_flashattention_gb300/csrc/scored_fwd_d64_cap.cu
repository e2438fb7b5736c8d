// Scored forward kernel instantiations over dense K/V, head dimension 64.
#include "scored_launch.cuh"

namespace fa {
template int launch_fwd_scored<64, kCap>(bool, bool, const CUtensorMap*, const FwdParams&, int, cudaStream_t);
}  // namespace fa
