// Scored forward kernel instantiations over dense K/V, head dimension 256.
#include "scored_launch.cuh"

namespace fa {
template int launch_fwd_scored<256, kCap>(bool, bool, const CUtensorMap*, const FwdParams&, int, cudaStream_t);
}  // namespace fa
