// Scores that are capped, biased by distance and restricted to a range of keys
// per query (ScoreRule): the arithmetic that the scored instantiations of the
// forward and backward kernels share.
//
// Everything is in base-2 units, as in the kernels: y = x * log2(e).
//   cap    tanh(x / cap) = 1 - 2 r with r = 1 / (1 + exp(2 x / cap)), so
//          y = C - 2 C r, C = cap * log2(e): one exp2 and one reciprocal per
//          score, exact at both ends (exp2 -> 0 or inf gives r = 1 or 0).  Its
//          error is absolute, a few 2^-24 of C, which is what a softmax feels
//          (a relative error of p); a tanh with a relative error of 2^-11, the
//          hardware's, would move p by 2^-11 * cap.  The derivative
//          1 - tanh^2 = 4 r (1 - r) keeps its relative precision.
//   bias   y -= slope * log2(e) * |position - key|: positions and keys are
//          whole numbers below 2^24, exact in fp32 (further ones round to
//          2^-24 of the distance).
//   range  hidden scores are replaced (never added to), so that a NaN or an
//          infinity in a hidden key's score does not spread.
#pragma once

#include <type_traits>

#include "fa_kernels.h"
#include "ptx.cuh"

namespace fa {

constexpr float kLog2E = 1.4426950408889634f;
constexpr int kNoKey = 0x7fffffff;

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Keys [lo, hi) that a query row sees (lo >= hi: none).
struct KeyRange {
  int lo, hi;
};

// Row i of sequence z, i < q_len (the caller's bound), nk keys.
template <bool CAUSAL>
__device__ __forceinline__ KeyRange score_row(const ScoreRule& rule, int z, int i, int nk, int off) {
  KeyRange r{0, nk};
  if (rule.rows != nullptr) {
    const int2 g = __ldg(rule.rows + static_cast<size_t>(z) * rule.row_count + i);
    r.lo = max(g.x, 0);
    r.hi = min(g.y, nk);
  }
  if (CAUSAL) {
    r.hi = min(r.hi, i + off + 1);
    if (rule.window > 0) r.lo = max(r.lo, i + off - rule.window + 1);
  }
  return r;
}

// What the rows [i0, i1] of a query tile see together: keys outside
// [lo, hi) are hidden from all of them, keys inside [all_lo, all_hi) are
// hidden from none.
struct KeySpan {
  int lo, hi, all_lo, all_hi;
};

// `tile` is the 128-row tile that holds rows i0 .. i1 (i1 < i0: no row).
template <bool CAUSAL>
__device__ __forceinline__ KeySpan score_span(const ScoreRule& rule, int z, int tile, int i0, int i1, int nk, int off) {
  if (i1 < i0) return KeySpan{0, 0, kNoKey, 0};
  KeySpan s{0, nk, 0, nk};
  if (rule.qtab != nullptr) {
    const int4 g = __ldg(rule.qtab + static_cast<size_t>(z) * rule.qtiles + tile);
    s = KeySpan{g.x, min(g.y, nk), g.z, min(g.w, nk)};
  }
  if (CAUSAL) {
    s.hi = min(s.hi, i1 + off + 1);
    s.all_hi = min(s.all_hi, i0 + off + 1);
    if (rule.window > 0) {
      s.lo = max(s.lo, i0 + off - rule.window + 1);
      s.all_lo = max(s.all_lo, i1 + off - rule.window + 1);
    }
  }
  return s;
}

// Key tiles [j0, j0 + return) of BN keys that cover [lo, hi); at least one
// tile (all of it hidden) where no key is seen, so that every work item has
// one.
template <int BN>
__device__ __forceinline__ int score_key_tiles(const KeySpan& s, int& j0) {
  j0 = 0;
  if (s.hi <= s.lo) return 1;
  j0 = s.lo / BN;
  return (s.hi + BN - 1) / BN - j0;
}

template <int BN>
__device__ __forceinline__ bool score_masked(const KeySpan& s, int j) {
  return j * BN < s.all_lo || (j + 1) * BN > s.all_hi;
}

// Query tiles [i0, i0 + return) of BM rows that hold every row which sees a
// key of key tile j (128 keys), at least one.
template <bool CAUSAL, int BM>
__device__ __forceinline__ int score_query_tiles(const ScoreRule& rule, int z, int j, int Nq, int off, int& i0) {
  int a = 0, e = Nq;
  if (rule.ktab != nullptr) {
    const int2 g = __ldg(rule.ktab + static_cast<size_t>(z) * rule.ktiles + j);
    a = g.x;
    e = min(g.y, Nq);
  }
  if (CAUSAL) {
    a = max(a, j * 128 - off);
    if (rule.window > 0) e = min(e, (j + 1) * 128 - 1 + rule.window - off);
  }
  if (e <= a) {  // no row: one tile, hidden
    i0 = 0;
    return 1;
  }
  i0 = a / BM;
  return (e + BM - 1) / BM - i0;
}

// Bits [lo, hi) of a 32-bit word.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  const uint32_t below_hi = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
  const uint32_t below_lo = lo == 32 ? 0xffffffffu : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

// Mask of a packed 16-bit pair from its two columns' bits (bits 0 and 1).
__device__ __forceinline__ uint32_t pair_mask(uint32_t bits) {
  return ((bits & 1u) ? 0x0000ffffu : 0u) | ((bits & 2u) ? 0xffff0000u : 0u);
}

// N raw products S (fp32 bits) -> base-2 scores y, before bias and mask.
template <int N>
__device__ __forceinline__ void score_cap(const ScoreRule& rule, float scale_log2, uint32_t* s) {
  if (rule.cap2 != 0.f) {
    const uint64_t kin = f2_pack(rule.cap_in, rule.cap_in), one = f2_pack(1.f, 1.f);
    const uint64_t C = f2_pack(rule.cap2, rule.cap2), m2C = f2_pack(-2.f * rule.cap2, -2.f * rule.cap2);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float a, b;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), kin), a, b);
      f2_unpack(f2_add(f2_pack(ex2_approx(a), ex2_approx(b)), one), a, b);
      f2_unpack(f2_fma(f2_pack(rcp_approx(a), rcp_approx(b)), m2C, C), a, b);
      s[c] = __float_as_uint(a);
      s[c + 1] = __float_as_uint(b);
    }
  } else {
    const uint64_t k = f2_pack(scale_log2, scale_log2);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float a, b;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), k), a, b);
      s[c] = __float_as_uint(a);
      s[c + 1] = __float_as_uint(b);
    }
  }
}

// y -= slope2 * |first + c|, first = the first column's key minus the row's
// position.  ONE_SIDE (causal): columns that count have first + c <= 0, so
// the bias is slope2 * (first + c), without the absolute value (columns on
// the other side are hidden).
template <int N, bool ONE_SIDE>
__device__ __forceinline__ void score_bias(float slope2, float first, uint32_t* s) {
  if constexpr (ONE_SIDE) {
    const uint64_t k2 = f2_pack(slope2, slope2), f2 = f2_pack(first, first);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float a, b;
      const uint64_t d = f2_add(f2, f2_pack(static_cast<float>(c), static_cast<float>(c + 1)));
      f2_unpack(f2_fma(d, k2, f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]))), a, b);
      s[c] = __float_as_uint(a);
      s[c + 1] = __float_as_uint(b);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c)
      s[c] = __float_as_uint(fmaf(-slope2, fabsf(first + static_cast<float>(c)), __uint_as_float(s[c])));
  }
}

// Constants of a backward call's scores, packed for the f32x2 arithmetic.
struct ScoreConsts {
  uint64_t nsl2, kin, nC, p2C;
  __device__ __forceinline__ ScoreConsts(const ScoreRule& rule, float scale_log2)
      : nsl2(f2_pack(-scale_log2, -scale_log2)),
        kin(f2_pack(rule.cap_in, rule.cap_in)),
        nC(f2_pack(-rule.cap2, -rule.cap2)),
        p2C(f2_pack(2.f * rule.cap2, 2.f * rule.cap2)) {}
};

// Recomputed probabilities of two columns, p = exp2(y - lse2), before the
// mask, and the factor 1 - tanh^2 that the cap puts on dS (`fac`, CAP only).
// `lse2`: of the two columns' rows; `dist`: position minus key (or key minus
// position) of the two; `kb`: what lse2 - y gains per unit of it (ONE_SIDE:
// signed; else per unit of its absolute value).
template <bool CAP, bool BIAS, bool ONE_SIDE>
__device__ __forceinline__ void score_prob(const ScoreConsts& k, uint64_t s, uint64_t lse2, uint64_t dist, uint64_t kb,
                                           float& p0, float& p1, uint64_t& fac) {
  uint64_t x;  // lse2 - y
  if constexpr (CAP) {
    float a, b;
    f2_unpack(f2_mul(s, k.kin), a, b);
    f2_unpack(f2_add(f2_pack(ex2_approx(a), ex2_approx(b)), f2_pack(1.f, 1.f)), a, b);
    const uint64_t r = f2_pack(rcp_approx(a), rcp_approx(b));
    fac = f2_mul(r, f2_fma(r, f2_pack(-4.f, -4.f), f2_pack(4.f, 4.f)));
    x = f2_fma(r, k.p2C, f2_add(k.nC, lse2));
  } else {
    x = f2_fma(s, k.nsl2, lse2);
  }
  if constexpr (BIAS) {
    if constexpr (!ONE_SIDE) {
      float a, b;
      f2_unpack(dist, a, b);
      dist = f2_pack(fabsf(a), fabsf(b));
    }
    x = f2_fma(dist, kb, x);
  }
  float a, b;
  f2_unpack(x, a, b);
  p0 = ex2_approx(-a);
  p1 = ex2_approx(-b);
}

// The columns of a transposed tile (rows keys, columns queries) that key `key`
// is visible to, one bit per column: W words from query row q0 of sequence z.
template <bool CAUSAL, int W>
__device__ __forceinline__ void score_column_bits(const ScoreRule& rule, int z, int key, int q0, int Nk, int off,
                                                  uint32_t* keep) {
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int c0 = q0 + 32 * w;
    uint32_t bits = key < Nk ? 0xffffffffu : 0u;
    if (CAUSAL) bits &= bit_range(key - off - c0, rule.window > 0 ? key + rule.window - off - c0 : 32);
    if (rule.rows != nullptr) {
      const int2* rows = rule.rows + static_cast<size_t>(z) * rule.row_count;
      uint32_t seen = 0u;
#pragma unroll 8
      for (int c = 0; c < 32; ++c) {
        const int2 g = __ldg(rows + min(c0 + c, rule.row_count - 1));
        seen |= (key >= g.x && key < g.y ? 1u : 0u) << c;
      }
      bits &= seen;
    }
    keep[w] = bits;
  }
}

// Zero the 16-bit rows [a, b) of a tile of DSUB 128-byte-swizzled sub-tiles
// of `sub` bytes each (a row's 128 bytes are the same set under the swizzle).
// Called by a whole warp; the caller fences before the async proxy reads.
template <int DSUB>
__device__ __forceinline__ void zero_tile_rows(uint32_t tile, int sub, int a, int b, int lane) {
  for (int idx = lane; idx < (b - a) * 8 * DSUB; idx += 32) {
    const int row = a + idx / (8 * DSUB), rem = idx % (8 * DSUB);
    st_shared_v4(tile + (rem / 8) * sub + row * 128 + (rem % 8) * 16, 0u, 0u, 0u, 0u);
  }
}

// Query rows [q0, q0 + BM) of sequence z that see no key: their rows of a
// 16-bit tile in shared memory (DSUB sub-tiles of `sub` bytes) are zeroed, so
// that a probability of 0 is not multiplied by what such a row may hold.
// Called by a whole warp.  Returns whether any row was.
template <bool CAUSAL, int BM, int DSUB>
__device__ __forceinline__ bool zero_blind_rows(const ScoreRule& rule, int z, int q0, int Nq, int Nk, int off,
                                                uint32_t tile, int sub, int lane) {
  bool any = false;
#pragma unroll 1
  for (int g = 0; g < BM; g += 32) {
    const int q = q0 + g + lane;
    bool blind = false;
    if (q < Nq) {
      const KeyRange r = score_row<CAUSAL>(rule, z, q, Nk, off);
      blind = r.lo >= r.hi;
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, blind); m != 0u; m &= m - 1u) {
      const int row = g + __ffs(static_cast<int>(m)) - 1;
      zero_tile_rows<DSUB>(tile, sub, row, row + 1, lane);
      any = true;
    }
  }
  return any;
}

// Runs f(cap, bias) with the two as compile-time flags.
template <typename F>
__device__ __forceinline__ void score_variants(bool cap, bool bias, F&& f) {
  using Yes = std::true_type;
  using No = std::false_type;
  if (cap) {
    if (bias) f(Yes{}, Yes{}); else f(Yes{}, No{});
  } else {
    if (bias) f(No{}, Yes{}); else f(No{}, No{});
  }
}

}  // namespace fa
