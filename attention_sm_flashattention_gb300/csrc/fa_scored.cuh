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
//          1 - tanh^2 = 4 r (1 - r) is taken as 4 r (e r) with e = exp(2 x /
//          cap), which keeps its relative precision at both ends (1 - r would
//          cancel where scores are near -cap).
//   bias   y -= slope * log2(e) * |position - key|: positions and keys are
//          whole numbers below 2^24, exact in fp32 (further ones round to
//          2^-24 of the distance).
//   range  hidden scores are replaced (never added to), so that a NaN or an
//          infinity in a hidden key's score does not spread.
//
// Roundings to 16 bits.  P and dS are operands of f16-kind MMAs, whose two
// operands have one type, that of V, dO, K and Q: in 32 bits they would take
// tf32 products at half the rate, with V, dO, K and Q converted and twice
// their shared memory.  Each rounds by half a step (2^-11 of the value in
// fp16, 2^-8 in bf16); row sums, lse, 1 - tanh^2 and every accumulator are in
// fp32, from P before it is rounded.  Delta is a sum in fp32 of dO times the
// 16-bit O that the caller has: an exact one would take S and dP, two of the
// dQ kernel's three products, a second time (kinds with sinks, whose few tiles
// need it most, have a cheaper one: fa_bwd_dq_kernel).  Against the exact result o and
// dV are as close as rounding them alone allows, within a third; dQ and dK
// are off by 1.3 to 2.5 times as much (relative: fp16 0.0003 to 0.0005 against
// 0.0002, bf16 0.0024 to 0.0044 against 0.0017), most with capped scores.
#pragma once

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

// Query tiles [i0, i0 + return) of BM rows that hold every row which sees a
// key of key tile j (128 keys), at least one.
template <bool CAUSAL, int BM>
__device__ __forceinline__ int score_query_tiles(const ScoreRule& rule, int z, int j, int Nq, int off, int& i0) {
  int a = 0, e = Nq;
  if (rule.ktab != nullptr) {
    const int4 g = __ldg(rule.ktab + static_cast<size_t>(z) * rule.ktiles + j);
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

// Kinds with sinks: the key tiles that cover the sinks below s.hi and [s.lo,
// s.hi), as virtual tiles [j0, j0 + return): virtual tile v is key tile
// sink_key_tile(v, skip), which leaves out the tiles between the two ranges.
template <int BN>
__host__ __device__ __forceinline__ int sink_key_tiles(int sinks, const KeySpan& s, int& j0, int& skip) {
  j0 = skip = 0;
  if (s.hi <= 0) return 1;
  const int head = (min(sinks, s.hi) + BN - 1) / BN, end = (s.hi + BN - 1) / BN, first = max(s.lo, 0) / BN;
  if (first > head) skip = first - head;
  return end - skip;
}
template <int BN>
__host__ __device__ __forceinline__ int sink_key_tile(int sinks, int v, int skip) {
  return v < (sinks + BN - 1) / BN ? v : v + skip;  // (skip > 0 only where all sinks are below the last key)
}

// Bits [lo, hi) of a 32-bit word.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  const uint32_t below_hi = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
  const uint32_t below_lo = lo == 32 ? 0xffffffffu : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

// The columns from key k0 on that a row sees, one bit each.
template <bool SINK>
__device__ __forceinline__ uint32_t row_bits(const KeyRange& see, int sinks, int k0) {
  uint32_t bits = bit_range(see.lo - k0, see.hi - k0);
  if constexpr (SINK) bits |= bit_range(-k0, min(sinks, see.hi) - k0);
  return bits;
}

// Mask of a packed 16-bit pair from its two columns' bits (bits 0 and 1).
__device__ __forceinline__ uint32_t pair_mask(uint32_t bits) {
  return ((bits & 1u) ? 0x0000ffffu : 0u) | ((bits & 2u) ? 0xffff0000u : 0u);
}

// r = 1 / (1 + exp(2 x / cap)) of two products.  (One reciprocal for four,
// 1 / abcd times the other three, halves the reciprocals and measured slower:
// forward 141 -> 166 us, dQ 213 -> 264 us at Z32 H8 N1024 D128 causal, for the
// moves that regrouping packed pairs takes.)
__device__ __forceinline__ uint64_t cap_ratio(uint64_t kin, uint64_t s) {
  float a, b;
  f2_unpack(f2_mul(s, kin), a, b);
  f2_unpack(f2_add(f2_pack(ex2_approx(a), ex2_approx(b)), f2_pack(1.f, 1.f)), a, b);
  return f2_pack(rcp_approx(a), rcp_approx(b));
}

// 4 r of two products, and `slope` = 1 - tanh^2 = 4 r (1 - r), as 4 r (e r):
// with e / 4 (2 taken from the exponent) and 4 r = 1 / (1/4 + e / 4) no factor
// is left over.  e r is at most 1; where e is infinite r is 0, and the
// saturated product 0 as well.  (1 - r itself would cancel: off by 13% at x =
// -7.7 cap, by all of it at -8.7.)
__device__ __forceinline__ uint64_t cap_ratio4(uint64_t kin, uint64_t s, uint64_t& slope) {
  float a, b, r, t;
  f2_unpack(f2_fma(s, kin, f2_pack(-2.f, -2.f)), a, b);
  a = ex2_approx(a);
  b = ex2_approx(b);
  f2_unpack(f2_add(f2_pack(a, b), f2_pack(0.25f, 0.25f)), r, t);
  r = rcp_approx(r);
  t = rcp_approx(t);
  const uint64_t r4 = f2_pack(r, t);
  slope = f2_mul(r4, f2_pack(__saturatef(a * r), __saturatef(b * t)));
  return r4;
}

// N raw products S (fp32 bits) -> base-2 scores y, before bias and mask.
template <int N, bool CAP>
__device__ __forceinline__ void score_cap(const ScoreRule& rule, float scale_log2, uint32_t* s) {
  if constexpr (CAP) {
    const uint64_t kin = f2_pack(rule.cap_in, rule.cap_in);
    const uint64_t C = f2_pack(rule.cap2, rule.cap2), m2C = f2_pack(-2.f * rule.cap2, -2.f * rule.cap2);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float a, b;
      f2_unpack(f2_fma(cap_ratio(kin, f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]))), m2C, C), a, b);
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
  uint64_t nsl2, kin, nC, hC;
  __device__ __forceinline__ ScoreConsts(const ScoreRule& rule, float scale_log2)
      : nsl2(f2_pack(-scale_log2, -scale_log2)),
        kin(f2_pack(rule.cap_in, rule.cap_in)),
        nC(f2_pack(-rule.cap2, -rule.cap2)),
        hC(f2_pack(0.5f * rule.cap2, 0.5f * rule.cap2)) {}
};

// Recomputed probabilities of four columns where the bits of `keep` are set,
// 0 elsewhere: p = exp2(y - lse2) (P only), and pf = p (1 - tanh^2), what dP -
// Delta is multiplied by.  `lse2`: of the columns' rows; `dist`: position
// minus key (or key minus position) of the first two, the others two further;
// `kb`: what lse2 - y gains per unit of it (ONE_SIDE: signed; else per unit
// of its absolute value).
template <bool CAP, bool BIAS, bool ONE_SIDE, bool P>
__device__ __forceinline__ void score_prob4(const ScoreConsts& k, const uint32_t* s, uint64_t l01, uint64_t l23,
                                            uint64_t dist, uint64_t kb, uint32_t keep, float* p, uint64_t* pf) {
  const uint64_t s01 = f2_pack(__uint_as_float(s[0]), __uint_as_float(s[1]));
  const uint64_t s23 = f2_pack(__uint_as_float(s[2]), __uint_as_float(s[3]));
  uint64_t x[2], fac[2];  // lse2 - y, 1 - tanh^2
  if constexpr (CAP) {
    x[0] = f2_fma(cap_ratio4(k.kin, s01, fac[0]), k.hC, f2_add(k.nC, l01));
    x[1] = f2_fma(cap_ratio4(k.kin, s23, fac[1]), k.hC, f2_add(k.nC, l23));
  } else {
    x[0] = f2_fma(s01, k.nsl2, l01);
    x[1] = f2_fma(s23, k.nsl2, l23);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (BIAS) {
      uint64_t d = h == 0 ? dist : f2_add(dist, f2_pack(2.f, 2.f));
      if constexpr (!ONE_SIDE) {
        float a, b;
        f2_unpack(d, a, b);
        d = f2_pack(fabsf(a), fabsf(b));
      }
      x[h] = f2_fma(d, kb, x[h]);
    }
    float a, b;
    f2_unpack(x[h], a, b);
    const bool k0 = (keep >> (2 * h)) & 1u, k1 = (keep >> (2 * h + 1)) & 1u;
    float p0 = ex2_approx(-a), p1 = ex2_approx(-b);
    if constexpr (P) {
      p[2 * h] = p0 = k0 ? p0 : 0.f;
      p[2 * h + 1] = p1 = k1 ? p1 : 0.f;
    }
    if constexpr (CAP) {  // (the factor of a hidden score may be NaN)
      f2_unpack(f2_mul(f2_pack(p0, p1), fac[h]), p0, p1);
      p0 = k0 ? p0 : 0.f;
      p1 = k1 ? p1 : 0.f;
    } else if constexpr (!P) {
      p0 = k0 ? p0 : 0.f;
      p1 = k1 ? p1 : 0.f;
    }
    pf[h] = f2_pack(p0, p1);
  }
}

// A key's side of the rules, for transposed tiles (rows keys, columns
// queries): the query rows [lo, hi) that see it where those are without gaps.
// `gaps` (given ranges): the rows' own ranges have to be asked, and there may
// be rows that see nothing.
struct QueryRange {
  int lo, hi;
  bool gaps;
};
template <bool CAUSAL, bool SINK = false>
__device__ __forceinline__ QueryRange score_column(const ScoreRule& rule, int z, int key, int Nq, int Nk, int off) {
  QueryRange r{0, Nq, false};
  if (rule.ktab != nullptr) r.gaps = __ldg(rule.ktab + static_cast<size_t>(z) * rule.ktiles + min(key / 128, rule.ktiles - 1)).z == 0;
  if (key >= Nk) return r;  // (no key: its row of the gradients is dropped)
  if (rule.ktab != nullptr && !r.gaps) {
    const int2 g = __ldg(rule.cols + static_cast<size_t>(z) * Nk + key);
    r.lo = g.x;
    r.hi = g.y;
  }
  if (CAUSAL) {
    r.lo = max(r.lo, key - off);
    if (rule.window > 0 && !(SINK && key < rule.sinks)) r.hi = min(r.hi, key + rule.window - off);
  }
  return r;
}

// The columns (W words of 32, from query row q0) that this lane's key is
// visible to, one bit each.  The masks are applied to every tile, as selects
// inside the unrolled loops: code that only masked tiles run is code that the
// instruction cache has dropped since (a masked tile then took 10900 cycles
// against 3200, dK/dV kernel at D = 128).  Called by a whole warp.
template <int W>
__device__ __forceinline__ void score_column_bits(const ScoreRule& rule, int z, int key, const QueryRange& see, int q0,
                                                  uint32_t* keep) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int c0 = q0 + 32 * w;
    keep[w] = bit_range(see.lo - c0, see.hi - c0);
    if (see.gaps) {
      // lane c asks column c's range about every key of the warp in turn
      const int2 g = __ldg(rule.rows + static_cast<size_t>(z) * rule.row_count + min(c0 + lane, rule.row_count - 1));
      const int key0 = key - lane;
      uint32_t seen = 0u;
#pragma unroll 1
      for (int r = 0; r < 32; ++r) {
        const uint32_t b = __ballot_sync(0xffffffffu, key0 + r >= g.x && key0 + r < g.y);
        if (lane == r) seen = b;
      }
      keep[w] &= seen;
    }
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

// Whether the ranges of a query tile's rows may leave out keys between them:
// ranges given by the caller may, unless one key lies in all of them.
__device__ __forceinline__ bool span_gaps(const ScoreRule& rule, int z, const KeySpan& s) {
  return rule.ktab != nullptr && s.all_lo >= s.all_hi && __ldg(rule.ktab + static_cast<size_t>(z) * rule.ktiles).z == 0;
}

// K or V rows of keys that no row of a query tile sees may hold anything; what
// they are multiplied by is 0, but 0 * NaN is NaN.  So they are zeroed in the
// 16-bit tile in shared memory (keys k0 .. k0 + BN - 1, DSUB 128-byte-swizzled
// sub-tiles of `sub` bytes) before an MMA reads it: keys outside [lo, hi), or
// with gaps (span_gaps) those that none of the query rows [i0, i1] (at most
// 128) sees, `rows` being those of their sequence.  Called by a whole warp.
template <bool CAUSAL, int BN, int DSUB>
__device__ __forceinline__ void clear_keys(const int2* rows, int window, int i0, int i1, int nk, int off, int lo, int hi,
                                           bool gaps, int k0, uint32_t tile, int sub) {
  const int lane = threadIdx.x & 31;
  if (gaps) {
    ScoreRule rule{};  // (of which score_row reads three)
    rule.rows = rows;
    rule.window = window;
    KeyRange r[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int i = i0 + 32 * n + lane;
      r[n] = i <= i1 ? score_row<CAUSAL>(rule, 0, i, nk, off) : KeyRange{0, 0};
    }
#pragma unroll 1
    for (int w = 0; w < BN; w += 32) {  // one word of 32 keys after the other
      uint32_t seen = 0u;
#pragma unroll
      for (int n = 0; n < 4; ++n) seen |= bit_range(r[n].lo - k0 - w, r[n].hi - k0 - w);
      seen = __reduce_or_sync(0xffffffffu, seen);
      if (seen == 0xffffffffu) continue;
#pragma unroll 4
      for (int idx = lane; idx < 32 * 8 * DSUB; idx += 32) {
        const int row = idx / (8 * DSUB), rem = idx % (8 * DSUB);
        if (!((seen >> row) & 1u)) st_shared_v4(tile + (rem / 8) * sub + (w + row) * 128 + (rem % 8) * 16, 0u, 0u, 0u, 0u);
      }
    }
  } else {
    const int a = min(max(lo - k0, 0), BN), e = max(min(hi - k0, BN), a);
#pragma unroll 2
    for (int idx = lane; idx < (a + BN - e) * 8 * DSUB; idx += 32) {
      const int r = idx / (8 * DSUB), rem = idx % (8 * DSUB);
      st_shared_v4(tile + (rem / 8) * sub + (r < a ? r : r - a + e) * 128 + (rem % 8) * 16, 0u, 0u, 0u, 0u);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}
template <bool CAUSAL, int BN, int DSUB>
__device__ __noinline__ void clear_keys_call(const int2* rows, int window, int i0, int i1, int nk, int off, int lo, int hi,
                                             bool gaps, int k0, uint32_t tile, int sub) {
  clear_keys<CAUSAL, BN, DSUB>(rows, window, i0, i1, nk, off, lo, hi, gaps, k0, tile, sub);
}

// Nothing to do for most tiles.  CALL, the backward's kernels: a call, because
// in line its length in their loops cost the tiles that have nothing to clear
// (the gaps alone in line up to 6%, Z8 H8 N1024 D128 causal 128 -> 136 us;
// called 130).  The forward's warps change their register counts, which rules
// calls out; in line it cost nothing there.  Two ranges with 1200 keys between
// them, Z2 H8 N2048, forward and backward, without clearing the gap and with:
// D = 128 191 and 251 us, D = 256 308 and 412 us.
template <bool CAUSAL, int BN, int DSUB, bool CALL>
__device__ __forceinline__ void clear_unseen_keys(const ScoreRule& rule, int z, int i0, int i1, int nk, int off, int lo,
                                                  int hi, bool gaps, int k0, uint32_t tile, int sub) {
  if (!gaps && lo <= k0 && hi >= k0 + BN) return;
  const int2* rows = rule.rows + static_cast<size_t>(z) * rule.row_count;
  if constexpr (CALL) {
    clear_keys_call<CAUSAL, BN, DSUB>(rows, rule.window, i0, i1, nk, off, lo, hi, gaps, k0, tile, sub);
  } else {
    clear_keys<CAUSAL, BN, DSUB>(rows, rule.window, i0, i1, nk, off, lo, hi, gaps, k0, tile, sub);
  }
}

// The same for kinds with sinks, where a query tile sees the keys [lo, hi) and
// the first `sinks` below hi: of a tile's 16-key blocks (an MMA's depth each)
// those with a key that is seen, one bit each.  The others take no part in
// products over keys, so that only rows beside seen ones in a block have to be
// cleared, at most 45 of a tile; the first tile mostly has one block of 8 that
// counts (clearing its other 124 rows took a warp 1700 cycles, and kept the
// product waiting).  Where nothing is seen, block 0 counts, cleared: the product
// has to write its result all the same.
template <int BN>
__host__ __device__ __forceinline__ uint32_t sink_blocks(int sinks, int lo, int hi, int k0) {
  const int a = min(max(min(sinks, hi) - k0, 0), BN), b = min(max(lo - k0, 0), BN), e = min(max(hi - k0, b), BN);
  const uint32_t blocks =
      ((1u << ((a + 15) / 16)) - 1u) | (e > b ? ((1u << ((e + 15) / 16)) - 1u) & ~((1u << (b / 16)) - 1u) : 0u);
  return blocks != 0u ? blocks : 1u;
}
template <int BN, int DSUB>
__device__ __forceinline__ void clear_beside_sinks(int sinks, int lo, int hi, int k0, uint32_t tile, int sub) {
  const int a = min(max(min(sinks, hi) - k0, 0), BN), b = min(max(lo - k0, a), BN), e = min(max(hi - k0, b), BN);
  const int lane = threadIdx.x & 31;
  // behind the sinks, before the window and behind it, each up to its block's end (windows that begin among the sinks,
  // or end there, leave empty ranges)
  zero_tile_rows<DSUB>(tile, sub, a, min(b, (a + 15) / 16 * 16), lane);
  zero_tile_rows<DSUB>(tile, sub, max(b / 16 * 16, a), b, lane);
  zero_tile_rows<DSUB>(tile, sub, e, (e + 15) / 16 * 16, lane);
  if (a == 0 && e == b) zero_tile_rows<DSUB>(tile, sub, 0, 16, lane);
  fence_proxy_async_smem();
  __syncwarp();
}
// All of a tile's unseen rows, four at a time, in few instructions.
template <int BN, int DSUB>
__device__ __noinline__ void clear_all_beside_sinks(int sinks, int lo, int hi, int k0, uint32_t tile, int sub) {
  const int a = min(max(min(sinks, hi) - k0, 0), BN), b = min(max(lo - k0, a), BN), e = min(max(hi - k0, b), BN);
  const int lane = threadIdx.x & 31;
  // lane: 16 bytes of row r + lane / 8, sub-tile by sub-tile
  const uint32_t at = tile + lane * 16;
#pragma unroll 1
  for (int r = 0; r < BN; r += 4) {
    const int row = r + lane / 8;
    if ((row >= a && row < b) || row >= e) {
#pragma unroll
      for (int s = 0; s < DSUB; ++s) st_shared_v4(at + s * sub + r * 128, 0u, 0u, 0u, 0u);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}
template <int BN, int DSUB>
__device__ __noinline__ void clear_beside_sinks_call(int sinks, int lo, int hi, int k0, uint32_t tile, int sub) {
  clear_beside_sinks<BN, DSUB>(sinks, lo, hi, k0, tile, sub);
}

// Keys of key tile j that no query sees, where their query ranges tell (no
// gaps): their rows of a 16-bit tile in shared memory are zeroed.  Called by a
// whole warp.  Returns whether any was.
template <bool CAUSAL, int DSUB, bool SINK = false>
__device__ __forceinline__ bool zero_blind_keys(const ScoreRule& rule, int z, int j, int Nq, int Nk, int off,
                                                uint32_t tile, int sub, int lane) {
  bool any = false;
#pragma unroll 1
  for (int g = 0; g < 128; g += 32) {
    const QueryRange r = score_column<CAUSAL, SINK>(rule, z, j * 128 + g + lane, Nq, Nk, off);
    for (uint32_t m = __ballot_sync(0xffffffffu, !r.gaps && r.lo >= r.hi); m != 0u; m &= m - 1u) {
      const int row = g + __ffs(static_cast<int>(m)) - 1;
      zero_tile_rows<DSUB>(tile, sub, row, row + 1, lane);
      any = true;
    }
  }
  return any;
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

}  // namespace fa
