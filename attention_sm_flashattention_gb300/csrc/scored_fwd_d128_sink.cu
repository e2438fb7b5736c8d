// Scored forward kernel instantiations over dense K/V, head dimension 128.
#include "scored_launch.cuh"

namespace fa {
template int launch_fwd_scored<128, kSink>(bool, bool, const CUtensorMap*, const FwdParams&, int, cudaStream_t);
}  // namespace fa
