// Page tables of the paged cache, kept on the GPU: pages for a step's new
// tokens, their slots and positions, and pages given back.
//
// Step.  With h_b cached tokens, q_b new ones and pages of s,
//   first_b = ceil(h_b / s), need_b = ceil((h_b + q_b) / s) - first_b,
//   start_b = need_0 + ... + need_(b-1),
// new page i of sequence b is entry F - 1 - (start_b + i) of the free stack of
// height F; the slot of the token at position p is page(p / s) * s + p % s.
// All that a token needs besides start_b is local, so one kernel does it: each
// block sums need over the sequences before its first one by itself (two loads
// per sequence, from L2), takes the prefix over its own in shared memory, and
// writes its tokens.  A page's first new token writes the table's entry; pages
// that were there are read from it.  No block waits for another.  What bounds
// it: the 16 bytes written per token, and in small calls the launch (a block's
// chain of loads, sum and stores is about 3 us).
//
// Release.  The stack's new entries are in the order of sequences and pages,
// and invalid entries of a row are left out, so a row's place needs the number
// of valid entries before it: a count per sequence (one block each, rows read
// once), then each row's block sums the counts before it and writes.
#include <cstdint>

#include "fa_kernels.h"

namespace fa {

namespace {

constexpr int kStepThreads = 256;
constexpr int kStepTokens = 2048;  // per block: 8 per thread

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the block's threads, to all of them; `scratch`: 32 ints.
__device__ __forceinline__ int block_sum(int x, int* scratch) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  x = warp_sum(x);
  __syncthreads();  // (the scratch may still be read)
  if (lane == 0) scratch[warp] = x;
  __syncthreads();
  return warp_sum(lane < warps ? scratch[lane] : 0);
}

// Sum over the threads before this one; `total`: over all.
__device__ __forceinline__ int block_prefix(int x, int* scratch, int& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  int up = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = up;
  __syncthreads();
  const int mine = lane < warps ? scratch[lane] : 0;
  total = warp_sum(mine);
  return warp_sum(lane < warp ? mine : 0) + up - x;
}

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return min(max(x, lo), hi); }

// Pages of `tokens` tokens (up to 2^32 - 1 of them), at most max_pages.
__device__ __forceinline__ int pages_of(unsigned tokens, unsigned page, int max_pages) {
  return static_cast<int>(min(tokens / page + (tokens % page != 0u), static_cast<unsigned>(max_pages)));
}

struct StepSeq {
  int have, fresh, first, need;  // cached and new tokens, first new page and their number
};
__device__ __forceinline__ StepSeq step_seq(const PageStepParams& p, int b) {
  StepSeq s;
  s.have = max(p.cached_lens[b], 0);
  s.fresh = p.q_lens != nullptr ? clamp_int(p.q_lens[b], 0, p.N) : p.N;
  s.first = pages_of(static_cast<unsigned>(s.have), p.page_size, p.max_pages);
  s.need = pages_of(static_cast<unsigned>(s.have) + static_cast<unsigned>(s.fresh), p.page_size, p.max_pages) - s.first;
  return s;
}
__device__ __forceinline__ int step_len(const StepSeq& s) {
  return static_cast<int>(min(static_cast<unsigned>(s.have) + static_cast<unsigned>(s.fresh), 0x7fffffffu));
}

}  // namespace

// `apart`: each block writes the new lengths of the sequences that begin in it,
// and the last one the stack's height.  Where those are written in place, other
// blocks may still have to read the old ones: a kernel of one block follows
// (3 us more; with one block alone, its threads have read theirs by then).
__global__ void __launch_bounds__(kStepThreads) fa_page_step_kernel(const PageStepParams p, bool apart) {
  __shared__ int scratch[32];
  __shared__ int have[kStepTokens + 1], fresh[kStepTokens + 1], first[kStepTokens + 1], start[kStepTokens + 1];
  const int tid = threadIdx.x;
  const long long total = static_cast<long long>(p.B) * p.N, t0 = static_cast<long long>(blockIdx.x) * kStepTokens;
  const int count = static_cast<int>(min(total - t0, static_cast<long long>(kStepTokens)));
  const int b0 = static_cast<int>(t0 / p.N), n0 = static_cast<int>(t0 - static_cast<long long>(b0) * p.N);
  const int seqs = static_cast<int>((static_cast<long long>(n0) + count - 1) / p.N) + 1;  // that the block's tokens are of
  const int F = clamp_int(*p.free_count, 0, p.num_pages);
  int before = 0;
  for (int b = tid; b < b0; b += kStepThreads) before += step_seq(p, b).need;
  if (b0 > 0) before = block_sum(before, scratch);
  const bool many = seqs > 1;
  if (!many) __syncthreads();  // (as block_prefix does: every thread has read the height)
  for (int x = 0; x < seqs; x += kStepThreads) {
    StepSeq s{};
    if (x + tid < seqs) s = step_seq(p, b0 + x + tid);
    int sum = 0, mine = before;
    if (many) mine += block_prefix(s.need, scratch, sum);
    if (x + tid < seqs) {
      have[x + tid] = s.have;
      fresh[x + tid] = s.fresh;
      first[x + tid] = s.first;
      start[x + tid] = mine;
      const int b = b0 + x + tid;
      if (apart && (x + tid > 0 || n0 == 0)) p.context_lens[b] = step_len(s);
      if (apart && b == p.B - 1 && t0 + count == total) *p.free_count_out = F - mine - s.need;
    }
    before += sum;
  }
  __syncthreads();
  const unsigned N = static_cast<unsigned>(p.N), page = static_cast<unsigned>(p.page_size);
  // Two tokens per thread and turn, 16 bytes a store; all turns' loads before
  // any store.
  constexpr int kTurns = kStepTokens / (2 * kStepThreads);
  long long slot[kTurns][2];
  unsigned pos[kTurns][2];
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    if (2 * u * kStepThreads >= count) break;
    const int x = 2 * (tid + u * kStepThreads);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const unsigned at = static_cast<unsigned>(n0) + static_cast<unsigned>(x + e);
      const int l = many ? static_cast<int>(min(at / N, static_cast<unsigned>(seqs - 1))) : 0;
      const unsigned n = at - static_cast<unsigned>(l) * N;
      const unsigned ps = static_cast<unsigned>(have[l]) + n;
      const unsigned pg = p.page_shift >= 0 ? ps >> p.page_shift : ps / page;
      pos[u][e] = ps;
      slot[u][e] = -1;
      if (x + e < count && n < static_cast<unsigned>(fresh[l]) && pg < static_cast<unsigned>(p.max_pages)) {
        int* entry = p.block_table + static_cast<size_t>(b0 + l) * p.max_pages + pg;
        int id;
        if (static_cast<int>(pg) < first[l]) {
          id = *entry;
        } else {
          const int nth = start[l] + static_cast<int>(pg) - first[l];
          id = nth < F ? p.free_pages[F - 1 - nth] : -1;
          if (ps == pg * page) *entry = id;
        }
        if (id >= 0 && id < p.num_pages) slot[u][e] = static_cast<long long>(id) * p.page_size + (ps - pg * page);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    if (2 * u * kStepThreads >= count) break;
    const int x = 2 * (tid + u * kStepThreads);
    if (p.wide && x + 1 < count) {
      *reinterpret_cast<longlong2*>(p.slot_mapping + t0 + x) = make_longlong2(slot[u][0], slot[u][1]);
      *reinterpret_cast<longlong2*>(p.positions + t0 + x) = make_longlong2(pos[u][0], pos[u][1]);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (x + e >= count) break;
        p.slot_mapping[t0 + x + e] = slot[u][e];
        p.positions[t0 + x + e] = pos[u][e];
      }
    }
  }
}

// Lengths and the stack's height after the step, in place.
__global__ void __launch_bounds__(1024) fa_page_step_finish_kernel(const PageStepParams p) {
  __shared__ int scratch[32];
  const int F = clamp_int(*p.free_count, 0, p.num_pages);
  int need = 0;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const StepSeq s = step_seq(p, b);
    need += s.need;
    p.context_lens[b] = step_len(s);
  }
  need = block_sum(need, scratch);  // (every thread has read the height)
  if (threadIdx.x == 0) *p.free_count_out = F - need;
}

int launch_page_step(const PageStepParams& p, cudaStream_t stream) {
  const long long blocks = (static_cast<long long>(p.B) * p.N + kStepTokens - 1) / kStepTokens;
  if (blocks > 0x7fffffffLL) return -1;
  const bool in_place = p.context_lens == p.cached_lens || p.free_count_out == p.free_count;
  const bool apart = !in_place || blocks == 1;
  fa_page_step_kernel<<<static_cast<unsigned>(blocks), kStepThreads, 0, stream>>>(p, apart);
  if (cudaGetLastError() != cudaSuccess) return -1;
  if (apart) return 0;
  fa_page_step_finish_kernel<<<1, 1024, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

namespace {

// Valid pages among a row's entries that hold its tokens.
__device__ __forceinline__ int held_pages(const PageReleaseParams& p, int b) {
  return p.finished[b] ? pages_of(static_cast<unsigned>(max(p.context_lens[b], 0)), p.page_size, p.max_pages) : 0;
}
__device__ __forceinline__ bool valid_page(const PageReleaseParams& p, int id) { return id >= 0 && id < p.num_pages; }

}  // namespace

constexpr int kReleaseThreads = 256;
constexpr int kReleaseLoads = 8;  // per thread and turn, all in flight

// counts[b]: pages that sequence b gives back; counts[B]: the stack's height
// (the next kernel may write over the one it was read from).
__global__ void __launch_bounds__(kReleaseThreads) fa_page_count_kernel(const PageReleaseParams p) {
  __shared__ int scratch[32];
  const int b = blockIdx.x;
  const int* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
  const int held = held_pages(p, b);
  int n = 0;
#pragma unroll kReleaseLoads
  for (int i = threadIdx.x; i < held; i += kReleaseThreads) n += valid_page(p, row[i]);
  if (held > 0) n = block_sum(n, scratch);
  if (threadIdx.x == 0) {
    p.counts[b] = n;
    if (b == 0) p.counts[p.B] = clamp_int(*p.free_count, 0, p.num_pages);
  }
}

__global__ void __launch_bounds__(kReleaseThreads) fa_page_release_kernel(const PageReleaseParams p) {
  __shared__ int scratch[32];
  const int b = blockIdx.x, tid = threadIdx.x;
  const bool last = b == p.B - 1;
  const int held = held_pages(p, b), len = p.context_lens[b];
  const bool done = p.finished[b] != 0;
  if (held > 0 || last) {
    int at = 0;
#pragma unroll 4
    for (int x = tid; x < b; x += kReleaseThreads) at += p.counts[x];
    const int mine = p.counts[b];
    at = block_sum(at, scratch) + p.counts[p.B];
    if (last && tid == 0) *p.free_count_out = min(at + mine, p.num_pages);
    const int* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
    // (a page given back twice could overfill the stack: what is past it is dropped)
    if (mine == held) {  // all valid, as they mostly are: a copy
#pragma unroll kReleaseLoads
      for (int i = tid; i < held; i += kReleaseThreads)
        if (at + i < p.num_pages) p.free_pages[at + i] = row[i];
    } else {
      for (int i = 0; i < held; i += kReleaseThreads) {
        const int id = i + tid < held ? row[i + tid] : -1;
        const bool valid = valid_page(p, id);
        int sum;
        const int to = at + block_prefix(valid, scratch, sum);
        if (valid && to < p.num_pages) p.free_pages[to] = id;
        at += sum;
      }
    }
  }
  __syncthreads();  // every thread has read the length
  if (tid == 0) p.context_lens_out[b] = done ? 0 : len;
}

// Small calls in one block, a warp per sequence: its entries are read once, into
// registers, and written behind the sum of the counts of the warps before it.
constexpr int kSmallSeqs = 32;
constexpr int kSmallLoads = 8;  // per lane
__global__ void __launch_bounds__(32 * kSmallSeqs) fa_page_release_small_kernel(const PageReleaseParams p) {
  __shared__ int counts[kSmallSeqs];
  const int b = threadIdx.x / 32, lane = threadIdx.x % 32;  // (the block has 32 * B threads)
  const int F = clamp_int(*p.free_count, 0, p.num_pages);
  const int held = held_pages(p, b), len = p.context_lens[b];
  const bool done = p.finished[b] != 0;
  const int* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
  int id[kSmallLoads], n = 0;
#pragma unroll
  for (int u = 0; u < kSmallLoads; ++u) id[u] = 32 * u + lane < held ? row[32 * u + lane] : -1;
#pragma unroll
  for (int u = 0; u < kSmallLoads; ++u) n += __popc(__ballot_sync(0xffffffffu, valid_page(p, id[u])));
  if (lane == 0) counts[b] = n;
  __syncthreads();  // every thread has read the height and its length
  int to = F + warp_sum(lane < b ? counts[lane] : 0);
  if (b == p.B - 1 && lane == 0) *p.free_count_out = min(to + n, p.num_pages);
  if (lane == 0) p.context_lens_out[b] = done ? 0 : len;
#pragma unroll
  for (int u = 0; u < kSmallLoads; ++u) {
    const unsigned valid = __ballot_sync(0xffffffffu, valid_page(p, id[u]));
    const int mine = to + __popc(valid & ((1u << lane) - 1u));
    if (valid_page(p, id[u]) && mine < p.num_pages) p.free_pages[mine] = id[u];
    to += __popc(valid);
  }
}

int launch_page_release(const PageReleaseParams& p, cudaStream_t stream) {
  // (16 sequences of up to 256 pages: 2.0 us in a graph against 3.8 with two
  // launches; a block for more of them, which walks the rows: 256 of 32 8.3 against 4.4)
  if (p.B <= kSmallSeqs && p.max_pages <= 32 * kSmallLoads) {
    fa_page_release_small_kernel<<<1, 32 * p.B, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  }
  fa_page_count_kernel<<<p.B, kReleaseThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  fa_page_release_kernel<<<p.B, kReleaseThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace fa
