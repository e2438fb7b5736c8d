// Scored forward kernel instantiations over dense K/V, head dimension 256.
#include "fa_fwd.cuh"

namespace fa {

int launch_fwd_scored_d256(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                         cudaStream_t stream) {
  if (bf16)
    return causal ? launch_fwd<256, true, true, kScored>(maps, prm, num_sms, stream)
                  : launch_fwd<256, false, true, kScored>(maps, prm, num_sms, stream);
  return causal ? launch_fwd<256, true, false, kScored>(maps, prm, num_sms, stream)
                : launch_fwd<256, false, false, kScored>(maps, prm, num_sms, stream);
}

}  // namespace fa
