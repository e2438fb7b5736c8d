// Scored forward kernel instantiations over a paged K/V cache, whole or with
// split key ranges (then followed by the merge of the slices), head dimension
// 256.
#include "fa_fwd.cuh"

namespace fa {

int launch_fwd_paged_scored_d256(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                               cudaStream_t stream) {
  if (prm.splits == 1) {
    if (bf16)
      return causal ? launch_fwd<256, true, true, kPagedScored>(maps, prm, num_sms, stream)
                    : launch_fwd<256, false, true, kPagedScored>(maps, prm, num_sms, stream);
    return causal ? launch_fwd<256, true, false, kPagedScored>(maps, prm, num_sms, stream)
                  : launch_fwd<256, false, false, kPagedScored>(maps, prm, num_sms, stream);
  }
  int rc;
  if (bf16)
    rc = causal ? launch_fwd<256, true, true, kPagedSplitScored>(maps, prm, num_sms, stream)
                : launch_fwd<256, false, true, kPagedSplitScored>(maps, prm, num_sms, stream);
  else
    rc = causal ? launch_fwd<256, true, false, kPagedSplitScored>(maps, prm, num_sms, stream)
                : launch_fwd<256, false, false, kPagedSplitScored>(maps, prm, num_sms, stream);
  if (rc != 0) return rc;
  return launch_split_combine(prm.part_o, prm.part_lse, prm.o, prm.lse, static_cast<long long>(prm.heads) * prm.Nq,
                              256, prm.splits, bf16, num_sms, stream);
}

}  // namespace fa
