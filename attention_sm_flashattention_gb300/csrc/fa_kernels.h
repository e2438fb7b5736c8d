// Kernel parameter blocks and the per-instantiation launchers shared between
// the C-ABI translation unit and the kernel translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_once.h"

namespace fa {

// Rules of a scored call (fa_fwd_scored, fa_bwd_scored, fa_fwd_paged_scored):
// the score of query position i (of a sequence whose queries end its nk keys:
// absolute position i + off) and key j is
//   x = scale * q_i . k_j;  x = cap * tanh(x / cap) if capped;
//   x -= slope * |i + off - j| if biased;  hidden unless j is in the row's range
// [lo, hi): the row's entry of `rows`, below nk, up to its own position
// (causal) and at most window - 1 positions before it (window > 0).
struct ScoreRule {
  float cap2;           // cap * log2(e); 0 = scores not capped
  float cap_in;         // 2 * log2(e) * scale / cap: exp2(S * cap_in) = exp(2 x / cap)
  const float* slopes;  // [H] by query head, or null
  int H;                // query heads per sequence
  int heads_per_seq;    // the kernel's heads per sequence (packed grouped heads: K/V heads)
  int window;           // 0 = none
  // key ranges (null = none), as key_ranges.cu lays them out: per query row
  // (lo, hi); per 128-row query tile (min lo, max hi over rows that see a key,
  // max lo, min hi over all its rows); per 128-key tile the rows [first, last)
  // that see one of its keys, and 1 if `cols` holds for its keys and every row
  // sees some key; per key the rows [first, last) that see it, where those are
  // without gaps (documents, prefix)
  const int2* rows;
  const int4* qtab;
  const int4* ktab;
  const int2* cols;
  int row_count, qtiles, ktiles;  // per sequence: query rows, query tiles, key tiles
  const int* q_lens;    // paged: new tokens of each sequence, or null (all Nq)
  // kinds with sinks (score_sinks; causal, window > 0, no key ranges): the
  // first `sinks` keys are not hidden by the window
  int sinks;
};

// Shapes: queries (and O, dO, dQ) are [heads, Nq, D]; keys and values (and
// dK, dV) are [heads / group, Nk, D]; query head h reads K/V head h / group.
// Causal: query i sees key j iff j <= i + causal_off, causal_off = Nk - Nq
// (the queries are the last Nq positions of the sequence; Nq <= Nk).
struct FwdParams {
  __half* o;         // [heads, Nq, D] (written through the O tensor map)
  float* lse;        // [heads, Nq]
  int heads;         // query heads, Z * H
  int group;         // query heads per K/V head
  int Nq, Nk;        // query and key lengths (any >= 1)
  int causal_off;    // Nk - Nq
  float scale_log2;  // scale * log2(e)
  int* status;       // device status word
  // Paged K/V cache (paged launchers only).  K and V are [num_pages,
  // page_size, Hkv, D]; query head h of sequence b = head / H reads K/V head
  // (head % H) / group of its cache pages; sequence b's key p lives in page
  // block_table[b * max_pages + p / page_size] at row p % page_size, and its
  // key count is context_lens[b], clamped to [causal ? Nq : 1, max_pages *
  // page_size].
  const int* block_table;
  const int* context_lens;
  int H;             // query heads per sequence
  int num_pages, page_size, max_pages;
  // Selected blocks (sparse launchers): for sequence b and K/V head kvh, list
  // entries e < sel_count[b * Hkv + kvh] (at most max_pages) name physical
  // page sel_pages[(b * Hkv + kvh) * max_pages + e] holding logical block
  // sel_blocks[...]; row r of it is the token at logical position block *
  // page_size + r, visible iff below context_lens[b] (and, causal, at most
  // the query's own position, the queries being the context's last Nq).
  const int* sel_pages;
  const int* sel_blocks;
  const int* sel_count;
  int Hkv;
  // Packed grouped heads (0 = off): the G query heads that share a K/V head
  // run as one head of G * q_period rows (they are consecutive in memory);
  // row r is query position r % q_period, and `heads`, `group`, `Nq` and `H`
  // describe the packed problem (group 1).
  int q_period;
  // Split key range (paged split launchers): each work item's key tiles are
  // cut into `splits` contiguous slices, one work unit each.  A unit writes
  // its rows' partial result to part_o ([splits, heads * Nq, D] fp32, O
  // normalised by the slice's own row sum) and part_lse ([splits, heads *
  // Nq] fp32, natural log; -inf for a slice with no visible key), and the
  // combine kernel merges the slices into o and lse.
  int splits;
  float* part_o;
  float* part_lse;
  ScoreRule rule;  // scored launchers
  int token;       // scored paged launcher: heads of at most 32 rows, four slices per unit
};

struct BwdParams {
  const __half* v;     // [heads / group, Nk, D] (read directly by the D = 256 dK/dV kernel)
  const __half* o;     // [heads, Nq, D] forward output
  const __half* dout;  // [heads, Nq, D]
  const float* lse;    // [heads, Nq] natural-log lse from the forward
  __half* dq;          // [heads, Nq, D]
  __half* dk;          // [heads / group, Nk, D]
  __half* dv;
  float* delta;        // workspace [heads, Nq_pad]: rowsum(O * dO), 0 in the padding
  float* lse2;         // workspace [heads, Nq_pad]: lse * log2(e), +inf in the padding
  int heads;           // query heads
  int group;           // query heads per K/V head
  int Nq, Nk;
  int Nq_pad;          // Nq rounded up to the 128-row query tile
  int causal_off;      // Nk - Nq
  float scale;         // softmax scale
  float scale_log2;    // scale * log2(e)
  int* status;
  ScoreRule rule;      // scored launchers
  // kinds with sinks: the dK/dV kernel's units over far query tiles and their
  // partial results (sink_parts)
  int far_tiles;       // query tiles of a far unit, at most
  int far_units;       // far units of one K/V head
  float* part;         // [K/V heads][part_floats]
  long long part_floats;
};

// dK and dV of a window with sinks.  Key tile j's own unit takes the query
// tiles whose windows reach it, [first, near_end); where it holds sinks, all
// later query tiles see those too.  One unit for them would be the longest by
// far (at 8192 queries and a window of 1024: 64 tiles against 9, times the
// group), so they are cut into far units of far_tiles query tiles, and the
// units of such a key tile write fp32 partial sums, which a join adds in a
// fixed order: [near: 128 rows][far 1: sink rows][far 2: sink rows]..., a row
// being dV then dK.  Key tiles without sinks, or whose windows reach the last
// query, have one unit, which writes dK and dV as elsewhere.
struct SinkTile {
  int first, near_end;  // query tiles of the near unit
  int far;              // far units
  int rows;             // sink keys in this key tile
};
// BM: query rows per tile of the dK/dV kernel; window > 0, off = Nk - Nq.
template <int BM>
__host__ __device__ inline SinkTile sink_tile(int j, int sinks, int window, int Nq, int off, int far_tiles) {
  const int nqt = (Nq + BM - 1) / BM;
  const int a = j * 128 - off > 0 ? j * 128 - off : 0;
  const int e = (j + 1) * 128 - 1 + window - off;  // (the window is below Nk: no overflow)
  SinkTile t;
  t.first = a / BM;
  t.near_end = ((e < Nq ? (e > 0 ? e : 0) : Nq) + BM - 1) / BM;
  if (t.near_end <= t.first) t.near_end = t.first + 1;  // at least one tile, whatever it sees
  t.rows = sinks - j * 128 < 0 ? 0 : sinks - j * 128 < 128 ? sinks - j * 128 : 128;
  t.far = t.rows > 0 ? (nqt - t.near_end + far_tiles - 1) / far_tiles : 0;
  return t;
}

// Far units of the key tiles before j, j at most the number of those with sinks:
// the sum of SinkTile's `far` in closed form, for the host and the join, each of
// whose warps asks for it (a loop over the tiles: 482 us of a backward of 2.9 ms with
// 30000 sinks, D = 128, now 29; in the units of the dK/dV kernel, which are few and
// walk the tiles, it is 1% at most).  Tile x's near unit ends with query
// tile c x + K (c = 128 / BM), clamped to [1, nqt], so that the far query tiles are
// nqt - 1 up to some x and go down by c from there to 0; a unit takes F of them.
// Int: 32 bits are enough where F is what sink_parts chooses, so that no tile has
// more than 65 far units (nqt * 65 < 2^31); long long for any F.
template <int BM, class Int>
__host__ __device__ inline Int sink_far_before(int j, int window, int Nq, int off, int F) {
  constexpr int c = 128 / BM;
  static_assert(c == 1 || c == 2, "query tiles of 128 or 64 rows");
  const int nqt = (Nq + BM - 1) / BM, e = 127 + window - off;
  const int K = e > 0 ? (e + BM - 1) / BM : -(-e / BM);
  // the sum of ceil(y / F) over y = n, n - c, ..., as that of the terms' numbers above 0, F, 2 F, ...
  auto falling = [&](int n) -> Int {
    if (n <= 0) return 0;
    const Int q = static_cast<Int>((static_cast<unsigned>(n) + F - 1) / static_cast<unsigned>(F));
    const Int tri = F * (q * (q - 1) / 2), p = n & 1;
    if (c == 1) return n * q - tri;
    const Int odd = F % 2 != 0 ? (q + p) / 2 : p * q;  // of floor((i F + p) / 2), i < q: those rounded down
    return (n + p) / 2 * q - (tri + p * q - odd) / 2;
  };
  const int flat = K < 1 ? -K / c + 1 : 0;  // tiles with nqt - 1
  Int units = static_cast<Int>(j < flat ? j : flat) * ((nqt - 1 + F - 1) / F);
  if (j > flat) units += falling(nqt - (c * flat + K)) - falling(nqt - (c * j + K));
  return units;
}

// One launcher per head dimension; `causal` and `bf16` (bf16 instead of
// fp16 inputs and outputs) select the instantiation.  Return 0 on success.
// For the backward, `grid` caps each persistent grid (the SM count).  The
// tensor maps carry the element type.
// Dense forward maps: q, k, v, o (D = 256: v with 64-row boxes; o unused).
#define FA_DECLARE_LAUNCHERS(D)                                                                      \
  int launch_fwd_d##D(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm,       \
                      int num_sms, cudaStream_t stream);                                              \
  /* bwd maps: q, k, v, dout, dq, dk, dv, q and k with the D = 256 dQ kernel's boxes, o */                     \
  int launch_bwd_d##D(bool causal, bool bf16, const CUtensorMap* maps, const BwdParams& prm,       \
                      int grid, cudaStream_t stream);

FA_DECLARE_LAUNCHERS(64)
FA_DECLARE_LAUNCHERS(128)
FA_DECLARE_LAUNCHERS(256)
#undef FA_DECLARE_LAUNCHERS

// What a scored kernel instantiation does with its scores.  Compile-time: with
// the four forms beside each other in one kernel, the loops of its roles no
// longer fitted the instruction cache (dK/dV kernel, no rule at all: 222 us,
// against 122 us for the kernel without them, at Z32 H8 N1024 D128 causal).
// kSink, kSinkCap: a causal window whose rows also see the first keys of their
// sequence, in plain and in capped scores.  A kind of its own because a row
// then sees two ranges of keys, and a tile list with a gap.
enum ScoreKind : int { kNoScore = 0, kRanged = 1, kCap = 2, kBias = 3, kCapBias = 4, kSink = 5, kSinkCap = 6 };
constexpr bool score_caps(int kind) { return kind == kCap || kind == kCapBias || kind == kSinkCap; }
constexpr bool score_biases(int kind) { return kind == kBias || kind == kCapBias; }
constexpr bool score_sinks(int kind) { return kind == kSink || kind == kSinkCap; }

// Scored forward (dense; paged; paged with split key ranges and the merge) and
// backward, SCORE a ScoreKind but kNoScore: maps as for the launchers without
// a rule, except that the dense forward's K boxes have fwd_scored_block_n rows
// (V boxes too, but 64 at D = 256).  Instantiated in scored_*.cu.
template <int D, int SCORE>
int launch_fwd_scored(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                      cudaStream_t stream);
template <int D, int SCORE>
int launch_fwd_paged_scored(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                            cudaStream_t stream);
template <int D, int SCORE>
int launch_bwd_scored(bool causal, bool bf16, const CUtensorMap* maps, const BwdParams& prm, int grid,
                      cudaStream_t stream);

// Key ranges of every query row, and their tile tables (ScoreRule), from one
// of: documents (runs of equal ids), prefix lengths, or given (lo, hi) pairs.
struct KeyRangeLayout {  // int32 offsets into the mask buffer
  size_t rows, qtab, ktab, cols, total;
  int qtiles, ktiles;
};
inline KeyRangeLayout key_range_layout(int Z, int Nq, int Nk) {
  KeyRangeLayout l{};
  l.qtiles = static_cast<int>((Nq + 127LL) / 128);
  l.ktiles = static_cast<int>((Nk + 127LL) / 128);
  l.rows = 0;
  l.qtab = (static_cast<size_t>(Z) * Nq * 2 + 3) / 4 * 4;
  l.ktab = l.qtab + static_cast<size_t>(Z) * l.qtiles * 4;
  l.cols = l.ktab + static_cast<size_t>(Z) * l.ktiles * 4;
  l.total = l.cols + static_cast<size_t>(Z) * Nk * 2;
  return l;
}
// What the far units of a backward call need: query tiles each takes, their
// number and the partial results' floats per K/V head.  far_tiles is a near
// unit's length, so that no unit is much longer than the others, but not below
// 8 tiles (a unit's start and its partial rows cost about two), and with many
// sinks as long as leaves at most 64 far units and one more per key tile:
// those bound the partial results, and key tiles are units enough then.
struct SinkParts {
  int far_tiles, far_units;
  long long floats;
};
template <int BM>
inline SinkParts sink_parts(int sinks, int window, int Nq, int Nk, int D) {
  SinkParts p{};
  p.far_tiles = static_cast<int>((127LL + window + BM - 1) / BM + 1);
  if (p.far_tiles < 8) p.far_tiles = 8;
  const int tiles = (sinks + 127) / 128, off = Nk - Nq;
  const long long far = sink_far_before<BM, long long>(tiles, window, Nq, off, 1);  // far query tiles of all key tiles
  if (p.far_tiles < (far + 63) / 64) p.far_tiles = static_cast<int>((far + 63) / 64);
  p.far_units = sink_far_before<BM, int>(tiles, window, Nq, off, p.far_tiles);
  // the key tiles that have far units come first; the last one with sinks may hold less than 128 of them
  int with = 0;
  for (int step = 1 << 23; step > 0; step /= 2)
    if (with + step <= tiles && sink_tile<BM>(with + step - 1, sinks, window, Nq, off, p.far_tiles).far > 0) with += step;
  const SinkTile last = sink_tile<BM>(tiles - 1, sinks, window, Nq, off, p.far_tiles);
  p.floats = (128LL * (with + p.far_units) - static_cast<long long>(last.far) * (128 - last.rows)) * 2 * D;
  return p;
}
// The join: dk and dv rows of the key tiles that have far units.
int launch_sink_join(const BwdParams& prm, int D, bool bf16, cudaStream_t stream);

int launch_key_ranges(const int* doc_ids, const int* prefix_lens, const int* ranges, int* mask, int Z, int Nq, int Nk,
                      cudaStream_t stream);

// Rotary positions (rotary.cu): one of q, k, v, turned or copied from strided
// rows to strided rows or to cache rows.
struct RotarySide {
  const uint16_t* in;
  uint16_t* out;
  long long in_z, in_h, in_n;     // strides in elements
  long long out_z, out_h, out_n;
  int heads;
  int mode;  // 0 plain output rows, 1 cache rows (out_n = row pitch, out_h = head pitch)
  int turn;  // 0: copied
};

struct RotaryParams {
  RotarySide side[3];             // q, k, v; heads = 0 for one that is not there
  const long long* positions;
  long long pos_z;                // 0: the same positions for every sequence
  const int* axes;                // [rot / 2]: each pair's axis, or null (one axis)
  int num_axes;
  long long pos_axis;             // stride of positions from axis to axis
  const double* freqs;
  const long long* slots;         // cache row of each token, or null
  long long cache_rows;
  int Z, N, D, rot;
  float sign, mscale;
  int heads;                      // of all sides
  int heads_per_block;
};
// `wide`: rot a multiple of 16 and every row 16-byte aligned.
int launch_rotary(const RotaryParams& prm, bool bf16, bool interleaved, bool wide, int num_sms, cudaStream_t stream);

// Page tables (page_tables.cu); as fa_cache_step and fa_cache_release take them.
struct PageStepParams {
  const int* free_pages;
  const int* free_count;
  int* block_table;
  const int* cached_lens;
  const int* q_lens;  // or null: N new tokens each
  long long* slot_mapping;
  long long* positions;
  int* context_lens;
  int* free_count_out;
  int B, N, num_pages, page_size, max_pages;
  int page_shift;  // log2(page_size), or -1
  bool wide;  // slot_mapping and positions are 16-byte aligned
};
int launch_page_step(const PageStepParams& prm, cudaStream_t stream);

struct PageReleaseParams {
  int* free_pages;
  const int* free_count;
  const int* block_table;
  const int* context_lens;
  const unsigned char* finished;
  int* context_lens_out;
  int* free_count_out;
  int* counts;  // workspace, B + 1
  int B, num_pages, page_size, max_pages;
};
int launch_page_release(const PageReleaseParams& prm, cudaStream_t stream);

// Paged cache write: token t's K and V rows ([Hkv, D] 16-bit values each) to
// cache row slots[t] of [cache_rows, Hkv, D] caches; negative slots and slots
// >= cache_rows are skipped.
int launch_cache_write(const void* k_new, const void* v_new, const long long* slots, void* k_cache, void* v_cache,
                       int tokens, int Hkv, int D, long long cache_rows, int num_sms, cudaStream_t stream);

// Forward over a paged K/V cache; maps: q, k cache, v cache (4-D, one page
// row block per box), o.
int launch_fwd_paged_d64(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                         cudaStream_t stream);
int launch_fwd_paged_d128(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                          cudaStream_t stream);
int launch_fwd_paged_d256(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                          cudaStream_t stream);
// Forward over selected blocks of a paged cache; maps as for the paged launchers.
int launch_fwd_sparse_d64(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                          cudaStream_t stream);
int launch_fwd_sparse_d128(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                           cudaStream_t stream);
int launch_fwd_sparse_d256(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                           cudaStream_t stream);

// Forward over a paged K/V cache with the key range of every work item split
// into prm.splits slices (partial results into prm.part_o / part_lse), then
// the combine kernel (o, lse); maps as for the paged launchers.
int launch_fwd_paged_split_d64(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                               cudaStream_t stream);
int launch_fwd_paged_split_d128(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                                cudaStream_t stream);
int launch_fwd_paged_split_d256(bool causal, bool bf16, const CUtensorMap* maps, const FwdParams& prm, int num_sms,
                                cudaStream_t stream);
// Merge `splits` partial results per row: rows = heads * Nq, O and lse as
// described for FwdParams::part_o / part_lse.
int launch_split_combine(const float* part_o, const float* part_lse, void* o, float* lse, long long rows, int D,
                         int splits, bool bf16, int num_sms, cudaStream_t stream);

// The same with a block per row (the scored forward's merge).
int launch_split_merge(const float* part_o, const float* part_lse, void* o, float* lse, long long rows, int D,
                       int splits, bool bf16, cudaStream_t stream);

// Index of the current device, or -1 if the runtime cannot tell.
inline int current_device_index() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

// Tile sizes the host needs to build tensor maps and size grids: keys per
// tile of the paged, selected-block and split forward, and of the dense one
// (which at D = 256 moves each 128-key tile as two halves: K by halves of
// the contraction, 128-row boxes; V by halves of the keys, 64-row boxes).
constexpr int fwd_block_n(int D) { return D == 256 ? 64 : 128; }
// scored, over dense K/V: D = 256 has 128-key tiles where no bias is added
constexpr int fwd_scored_block_n(int D, bool biased) { return biased ? fwd_block_n(D) : 128; }
inline int fwd_dense_block_n(int) { return 128; }

}  // namespace fa
