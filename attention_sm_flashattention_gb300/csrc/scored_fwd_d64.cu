// Scored forward kernel instantiations over dense K/V, head dimension 64.
#include "fa_fwd.cuh"

namespace fa {

int launch_fwd_scored_d64(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                         cudaStream_t stream) {
  if (bf16)
    return causal ? launch_fwd<64, true, true, kScored>(maps, prm, num_sms, stream)
                  : launch_fwd<64, false, true, kScored>(maps, prm, num_sms, stream);
  return causal ? launch_fwd<64, true, false, kScored>(maps, prm, num_sms, stream)
                : launch_fwd<64, false, false, kScored>(maps, prm, num_sms, stream);
}

}  // namespace fa
