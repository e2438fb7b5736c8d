// Launchers of the scored kernels for one head dimension and kind of score;
// each is instantiated in a translation unit of its own.
#pragma once

#include "fa_bwd256.cuh"
#include "fa_fwd.cuh"
#include "fa_fwd256.cuh"

namespace fa {

// Calls go(causal, bf16) with both as compile-time truth values (kinds with
// sinks are causal, and have no other kernels).
template <int SCORE, typename F>
int with_flags(bool causal, bool bf16, F&& go) {
  if constexpr (!score_sinks(SCORE)) {
    if (!causal) return bf16 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
  }
  return bf16 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
}

template <int D, int SCORE>
int launch_fwd_scored(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                      cudaStream_t stream) {
  return with_flags<SCORE>(causal, bf16, [&](auto c, auto b) {
    constexpr bool C = decltype(c)::value, B = decltype(b)::value;
    if constexpr (fwd_scored_block_n(D, score_biases(SCORE)) != fwd_block_n(D)) {
      return launch_fwd256<C, B, SCORE>(maps, prm, num_sms, stream);
    } else {
      return launch_fwd<D, C, B, kScored, SCORE>(maps, prm, num_sms, stream);
    }
  });
}

// Whole key ranges, or split ones followed by the merge of the slices.
// prm.token: heads of at most 32 rows (kPagedToken, D <= 128), four slices per
// unit.
template <int D, int SCORE>
int launch_fwd_paged_scored(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                            cudaStream_t stream) {
  auto run = [&](auto mode) {
    return with_flags<SCORE>(causal, bf16, [&](auto c, auto b) {
      return launch_fwd<D, decltype(c)::value, decltype(b)::value, decltype(mode)::value, SCORE>(maps, prm, num_sms, stream);
    });
  };
  auto merge = [&](int slices) {
    return launch_split_merge(prm.part_o, prm.part_lse, prm.o, prm.lse, static_cast<long long>(prm.heads) * prm.Nq, D,
                              slices, bf16, stream);
  };
  if (prm.splits == 1 && !prm.token) return run(std::integral_constant<int, kPagedScored>{});
  if constexpr (D != 256) {
    if (prm.token) {
      const int rc = run(std::integral_constant<int, kPagedToken>{});
      return rc != 0 ? rc : merge(4 * prm.splits);
    }
  }
  const int rc = run(std::integral_constant<int, kPagedSplitScored>{});
  return rc != 0 ? rc : merge(prm.splits);
}

template <int D, int SCORE>
int launch_bwd_scored(bool causal, bool bf16, const CUtensorMap* maps, const BwdParams& prm, int grid,
                      cudaStream_t stream) {
  return with_flags<SCORE>(causal, bf16, [&](auto c, auto b) {
    constexpr bool C = decltype(c)::value, B = decltype(b)::value;
    if constexpr (D == 256) {
      return launch_bwd256<C, B, SCORE>(maps, prm, grid, stream);
    } else {
      return launch_bwd2<D, C, B, SCORE>(maps, prm, grid, stream);
    }
  });
}

}  // namespace fa
