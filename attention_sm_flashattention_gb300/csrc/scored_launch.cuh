// Launchers of the scored kernels for one head dimension and kind of score;
// each is instantiated in a translation unit of its own.
#pragma once

#include "fa_bwd256.cuh"
#include "fa_fwd.cuh"
#include "fa_fwd256.cuh"

namespace fa {

template <int D, int SCORE>
int launch_fwd_scored(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                      cudaStream_t stream) {
  auto go = [&](auto c, auto b) {
    constexpr bool C = decltype(c)::value, B = decltype(b)::value;
    if constexpr (fwd_scored_block_n(D, score_biases(SCORE)) != fwd_block_n(D)) {
      return launch_fwd256<C, B, SCORE>(maps, prm, num_sms, stream);
    } else {
      return launch_fwd<D, C, B, kScored, SCORE>(maps, prm, num_sms, stream);
    }
  };
  if (bf16) return causal ? go(std::true_type{}, std::true_type{}) : go(std::false_type{}, std::true_type{});
  return causal ? go(std::true_type{}, std::false_type{}) : go(std::false_type{}, std::false_type{});
}

// Whole key ranges, or split ones followed by the merge of the slices.
// prm.token: heads of at most 32 rows (kPagedToken, D <= 128), four slices per
// unit.
template <int D, int SCORE>
int launch_fwd_paged_scored(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                            cudaStream_t stream) {
  if (prm.splits == 1 && !prm.token) {
    if (bf16)
      return causal ? launch_fwd<D, true, true, kPagedScored, SCORE>(maps, prm, num_sms, stream)
                    : launch_fwd<D, false, true, kPagedScored, SCORE>(maps, prm, num_sms, stream);
    return causal ? launch_fwd<D, true, false, kPagedScored, SCORE>(maps, prm, num_sms, stream)
                  : launch_fwd<D, false, false, kPagedScored, SCORE>(maps, prm, num_sms, stream);
  }
  if constexpr (D != 256) {
    if (prm.token) {
      int rc;
      if (bf16)
        rc = causal ? launch_fwd<D, true, true, kPagedToken, SCORE>(maps, prm, num_sms, stream)
                    : launch_fwd<D, false, true, kPagedToken, SCORE>(maps, prm, num_sms, stream);
      else
        rc = causal ? launch_fwd<D, true, false, kPagedToken, SCORE>(maps, prm, num_sms, stream)
                    : launch_fwd<D, false, false, kPagedToken, SCORE>(maps, prm, num_sms, stream);
      if (rc != 0) return rc;
      return launch_split_merge(prm.part_o, prm.part_lse, prm.o, prm.lse, static_cast<long long>(prm.heads) * prm.Nq, D,
                                4 * prm.splits, bf16, stream);
    }
  }
  int rc;
  if (bf16)
    rc = causal ? launch_fwd<D, true, true, kPagedSplitScored, SCORE>(maps, prm, num_sms, stream)
                : launch_fwd<D, false, true, kPagedSplitScored, SCORE>(maps, prm, num_sms, stream);
  else
    rc = causal ? launch_fwd<D, true, false, kPagedSplitScored, SCORE>(maps, prm, num_sms, stream)
                : launch_fwd<D, false, false, kPagedSplitScored, SCORE>(maps, prm, num_sms, stream);
  if (rc != 0) return rc;
  return launch_split_merge(prm.part_o, prm.part_lse, prm.o, prm.lse, static_cast<long long>(prm.heads) * prm.Nq, D,
                            prm.splits, bf16, stream);
}

template <int D, int SCORE>
int launch_bwd_scored(bool causal, bool bf16, const CUtensorMap* maps, const BwdParams& prm, int grid,
                      cudaStream_t stream) {
  auto go = [&](auto launch) { return launch(maps, prm, grid, stream); };
  if constexpr (D == 256) {
    if (bf16) return causal ? go(launch_bwd256<true, true, SCORE>) : go(launch_bwd256<false, true, SCORE>);
    return causal ? go(launch_bwd256<true, false, SCORE>) : go(launch_bwd256<false, false, SCORE>);
  } else {
    if (bf16) return causal ? go(launch_bwd2<D, true, true, SCORE>) : go(launch_bwd2<D, false, true, SCORE>);
    return causal ? go(launch_bwd2<D, true, false, SCORE>) : go(launch_bwd2<D, false, false, SCORE>);
  }
}

}  // namespace fa
