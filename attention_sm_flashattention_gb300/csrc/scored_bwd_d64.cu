// Scored backward kernel instantiations, head dimension 64.
#include "fa_bwd2.cuh"

namespace fa {

int launch_bwd_scored_d64(bool causal, bool bf16, const CUtensorMap* maps, const BwdParams& prm, int grid,
                         cudaStream_t stream) {
  if (bf16)
    return causal ? launch_bwd2<64, true, true, true>(maps, prm, grid, stream)
                  : launch_bwd2<64, false, true, true>(maps, prm, grid, stream);
  return causal ? launch_bwd2<64, true, false, true>(maps, prm, grid, stream)
                : launch_bwd2<64, false, false, true>(maps, prm, grid, stream);
}

}  // namespace fa
