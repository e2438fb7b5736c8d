// Key ranges of scored attention: for every query row the keys [lo, hi) it may
// see, with the tile tables that the attention kernels go by (ScoreRule).
//
//   documents  a document is a run of equal ids along the sequence; a query
//              sees its own run: lo = the run's first position, hi = one past
//              its last.
//   prefix     hi = max(position + 1, prefix): causal behind a prefix that
//              every query sees whole.
//   given      the caller's (lo, hi), clamped to the keys.
//
// One launch: a block of 128 threads per 128-row query tile, then one per
// 128-key tile.  A run that leaves its tile is followed outwards 1024 ids at
// a time, so a block reads about the length of the documents it touches; the
// tables are a few bytes per row and the launch is bound by its latency.
#include "fa_kernels.h"

namespace fa {

constexpr int kRangeThreads = 128;
constexpr int kNone = 0x7fffffff;

// min and max over the block, broadcast to all threads.
__device__ __forceinline__ int block_min(int v, int* sh) {
  v = __reduce_min_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  return min(min(sh[0], sh[1]), min(sh[2], sh[3]));
}
__device__ __forceinline__ int block_max(int v, int* sh) { return -block_min(-v, sh); }

// First position of the run of equal ids that holds position p.
__device__ int run_start(const int* ids, int p, int* sh) {
  const int id = __ldg(ids + p);
  for (int top = p; top > 0; top -= 8 * kRangeThreads) {  // positions below top still to be looked at
    int q = -1;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int x = top - 1 - k * kRangeThreads - static_cast<int>(threadIdx.x);
      if (x >= 0 && __ldg(ids + x) != id) q = max(q, x);
    }
    q = block_max(q, sh);
    if (q >= 0) return q + 1;
  }
  return 0;
}

// One past the last position of the run that holds position p.
__device__ int run_end(const int* ids, int p, int n, int* sh) {
  const int id = __ldg(ids + p);
  for (int bottom = p + 1; bottom < n; bottom += 8 * kRangeThreads) {
    int q = kNone;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int x = bottom + k * kRangeThreads + static_cast<int>(threadIdx.x);
      if (x < n && __ldg(ids + x) != id) q = min(q, x);
    }
    q = block_min(q, sh);
    if (q != kNone) return q;
  }
  return n;
}

// The run that holds position p0 + tid, for the n <= 128 positions from p0.
__device__ void tile_runs(const int* ids, int p0, int n, int Nk, int* sh, unsigned* starts, int& lo, int& hi) {
  const int tid = threadIdx.x, p = p0 + tid;
  // a run starts at thread t: bit t of `starts`
  const bool start = tid > 0 && tid < n && __ldg(ids + p) != __ldg(ids + p - 1);
  const unsigned word = __ballot_sync(0xffffffffu, start);
  if ((tid & 31) == 0) starts[tid / 32] = word;
  lo = run_start(ids, p0, sh);
  hi = run_end(ids, p0 + n - 1, Nk, sh);
  __syncthreads();
  bool found = false;
#pragma unroll
  for (int w = 3; w >= 0; --w) {  // the last start at or before this thread
    const int top = tid - 32 * w;
    const unsigned m = top < 0 ? 0u : starts[w] & (top >= 31 ? 0xffffffffu : (2u << top) - 1u);
    if (!found && m != 0u) {
      lo = p0 + 32 * w + 31 - __clz(static_cast<int>(m));
      found = true;
    }
  }
  found = false;
#pragma unroll
  for (int w = 0; w < 4; ++w) {  // the first start after this thread
    const int top = tid - 32 * w;
    const unsigned m = top >= 31 ? 0u : starts[w] & (top < 0 ? 0xffffffffu : ~((2u << top) - 1u));
    if (!found && m != 0u) {
      hi = p0 + 32 * w + __ffs(static_cast<int>(m)) - 1;
      found = true;
    }
  }
}

__global__ void __launch_bounds__(kRangeThreads) fa_key_ranges_kernel(const int* __restrict__ doc_ids,
                                                                      const int* __restrict__ prefix_lens,
                                                                      const int2* __restrict__ given, int2* rows,
                                                                      int4* qtab, int4* ktab, int2* cols, int Nq,
                                                                      int Nk, int qtiles, int ktiles) {
  __shared__ int sh[4];
  __shared__ unsigned starts[4];
  const int per = qtiles + ktiles;
  const int z = blockIdx.x / per, b = blockIdx.x - z * per;
  const int tid = threadIdx.x, off = Nk - Nq;
  const int* ids = doc_ids != nullptr ? doc_ids + static_cast<size_t>(z) * Nk : nullptr;
  const int prefix = prefix_lens != nullptr ? min(max(__ldg(prefix_lens + z), 0), Nk) : 0;
  const int2* in = given != nullptr ? given + static_cast<size_t>(z) * Nq : nullptr;
  if (b < qtiles) {
    const int i0 = b * 128, i = i0 + tid, n = min(128, Nq - i0);
    int lo = 0, hi = 0;
    if (ids != nullptr) {
      tile_runs(ids, off + i0, n, Nk, sh, starts, lo, hi);
    } else if (in != nullptr) {
      if (tid < n) {
        const int2 g = __ldg(in + i);
        lo = max(g.x, 0);
        hi = min(g.y, Nk);
      }
    } else {
      hi = max(off + i + 1, prefix);
    }
    const bool live = tid < n, sees = live && lo < hi;
    if (live) rows[static_cast<size_t>(z) * Nq + i] = sees ? make_int2(lo, hi) : make_int2(0, 0);
    const int min_lo = block_min(sees ? lo : kNone, sh), max_hi = block_max(sees ? hi : 0, sh);
    const int max_lo = block_max(live ? (sees ? lo : kNone) : 0, sh);
    const int min_hi = block_min(live ? (sees ? hi : 0) : kNone, sh);
    if (tid == 0)
      qtab[static_cast<size_t>(z) * qtiles + b] = make_int4(min_lo == kNone ? 0 : min_lo, max_hi, max_lo, min_hi);
  } else {
    const int j = b - qtiles, k0 = j * 128, n = min(128, Nk - k0);
    int first = kNone, last = 0;  // rows that see this thread's key, then a key of the tile
    if (ids != nullptr) {
      tile_runs(ids, k0, n, Nk, sh, starts, first, last);
      first -= off;
      last -= off;
    } else if (in != nullptr) {
      for (int i = tid; i < Nq; i += kRangeThreads) {
        const int2 g = __ldg(in + i);
        if (g.x < k0 + n && g.y > k0 && g.x < g.y) {
          first = min(first, i);
          last = i + 1;
        }
      }
    } else {
      first = k0 + tid < prefix ? 0 : k0 + tid - off;
      last = Nq;
    }
    first = max(first, 0);
    last = min(last, Nq);
    const bool some = first < last && (in != nullptr || tid < n);
    if (in == nullptr && tid < n) cols[static_cast<size_t>(z) * Nk + k0 + tid] = some ? make_int2(first, last) : make_int2(0, 0);
    first = block_min(some ? first : kNone, sh);
    last = block_max(some ? last : 0, sh);
    if (tid == 0)
      ktab[static_cast<size_t>(z) * ktiles + j] =
          first < last ? make_int4(first, last, in == nullptr, 0) : make_int4(0, 0, in == nullptr, 0);
  }
}

int launch_key_ranges(const int* doc_ids, const int* prefix_lens, const int* ranges, int* mask, int Z, int Nq, int Nk,
                      cudaStream_t stream) {
  const KeyRangeLayout l = key_range_layout(Z, Nq, Nk);
  const long long blocks = static_cast<long long>(Z) * (l.qtiles + l.ktiles);
  fa_key_ranges_kernel<<<static_cast<unsigned>(blocks), kRangeThreads, 0, stream>>>(
      doc_ids, prefix_lens, reinterpret_cast<const int2*>(ranges), reinterpret_cast<int2*>(mask + l.rows),
      reinterpret_cast<int4*>(mask + l.qtab), reinterpret_cast<int4*>(mask + l.ktab),
      reinterpret_cast<int2*>(mask + l.cols), Nq, Nk, l.qtiles, l.ktiles);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace fa
