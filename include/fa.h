/*
 * fa.h -- C ABI of libfa.so: exact FlashAttention forward and backward for
 * one NVIDIA GB300 (sm_103a): fp16 inputs and outputs (fa_fwd, fa_bwd; bf16
 * through fa_fwd_bf16, fa_bwd_bf16 and the _ex calls), fp32 accumulation.
 *
 * What is computed (source: «把 FlashAttention 搬上昇腾：Triton-Ascend CV
 * Pipeline 优化实战»):
 *   forward  (§一)  S = Q K^T * scale,  P = softmax(S),  O = P V, computed
 *                   tile by tile with the online softmax (running row max m,
 *                   denominator l, unnormalised fp32 accumulator), exp2 with
 *                   log2(e) folded into the scale; causal mode visits only
 *                   key tiles at or below the diagonal and masks exactly only
 *                   inside diagonal tiles (§一, §八).
 *   backward (§二)  Delta = rowsum(O * dO), P recomputed from the saved
 *                   log-sum-exp, dP = dO V^T, dS = scale * P * (dP - Delta),
 *                   dQ = dS K, dK = dS^T Q, dV = P^T dO, with every gradient
 *                   tile written by exactly one CTA and a workspace that does
 *                   not grow with the number of heads times N^2 (§二's three
 *                   rules).
 *
 * Layout and types (all calls):
 *   q, k, v, o, dout, dq, dk, dv : fp16 (IEEE binary16), contiguous
 *                                  [Z, H, N, D] row-major, 16-byte aligned.
 *   lse                          : fp32 [Z, H, N]; lse[z,h,i] is the natural
 *                                  log of sum_j exp(S_ij) over the visible
 *                                  keys j (j <= i when causal).
 *   Every (z, h) pair is an independent head; queries and keys have the same
 *   length N (any N >= 1; a last partial 128-row tile is masked).  Causal
 *   means key j is visible to query i iff j <= i.  fa_fwd_ex / fa_bwd_ex
 *   below add grouped K/V heads and different query and key lengths.
 *
 * Ownership: every pointer is device memory owned by the caller; the library
 * keeps no pointer after a call returns and allocates no device memory on
 * these paths.  The only library state is one device status word per device.
 *
 * Asynchrony: fa_fwd / fa_bwd validate their arguments on the host, enqueue
 * kernels on `stream` and return.  A return of FA_OK means "enqueued".
 * Results are ready when the stream reaches that point.
 *
 * Errors: argument problems are reported synchronously, before anything is
 * enqueued, with a negative code (below).  A device-side wait that gives up
 * (bounded by about one second; it never hangs the GPU) is reported through
 * fa_device_status().  Not thread-safe with respect to concurrent first calls
 * on the same device from several host threads.
 */
#ifndef FA_GB300_FA_H
#define FA_GB300_FA_H

#include <stddef.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define FA_OK 0
#define FA_ERR_INVALID_ARG (-1) /* null pointer, a size <= 0, H not a multiple of Hkv, bad causal flag or
                                   dtype, non-finite or <= 0 scale, misaligned pointer */
#define FA_ERR_UNSUPPORTED (-2) /* D not in {64, 128, 256}, causal with Nq > Nk, or sizes past 32-bit indexing */
#define FA_ERR_WORKSPACE (-3)   /* workspace null, misaligned or smaller than its size query
                                   (fa_bwd_workspace_size, fa_fwd_paged_split_workspace_size) */
#define FA_ERR_CUDA (-4)        /* a CUDA runtime call or kernel launch failed */
#define FA_ERR_DEVICE (-5)      /* current device is not a compute capability 10.3 GPU */
#define FA_ERR_TIMEOUT (-6)     /* (fa_device_status) a kernel wait gave up; results invalid */
#define FA_ERR_SCRATCH_LIMIT (-7) /* (fa_bwd_noalloc) problem needs more than the built-in scratch buffer */

/*
 * Forward pass.  Source: «把 FlashAttention 搬上昇腾» §一 (tiled online
 * softmax, exp2, fp32 m/l/acc, fp16 P into the matrix unit, causal loop
 * bound + diagonal-only mask), §七 (D256: the key and value tiles move in
 * halves; the 256-column accumulator fits whole).
 *   q, k, v : inputs [Z,H,N,D] fp16.
 *   o       : output [Z,H,N,D] fp16, O = softmax(Q K^T scale) V, rounded to
 *             nearest from the fp32 accumulator divided by l.
 *   lse     : output [Z,H,N] fp32 (natural-log log-sum-exp of each row of S).
 *   Z, H, N : batch, heads, sequence length (N >= 1).
 *   D       : head dimension, 64, 128 or 256.
 *   causal  : 0 or 1.
 *   scale   : softmax scale applied to Q K^T (usually 1/sqrt(D)); finite, > 0.
 *   stream  : CUDA stream the kernel is enqueued on (0 = legacy default).
 * Returns FA_OK or a negative FA_ERR_* code.
 */
FA_API int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int Z, int H, int N, int D,
           int causal, float scale, cudaStream_t stream);

/*
 * Bytes of device workspace fa_bwd (or fa_bwd_bf16) needs: Delta and the
 * log2-scaled lse (2 x Z*H*N' fp32, N' = N rounded up to a multiple of 128,
 * each vector rounded up to 256 bytes).  It grows with Z*H*N, never with N^2
 * over all heads (§二, third rule): every dQ, dK and dV tile is accumulated
 * on chip by the one CTA that writes it.  Returns 0 for unsupported
 * arguments.
 */
FA_API size_t fa_bwd_workspace_size(int Z, int H, int N, int D, int causal);

/*
 * Backward pass.  Source: «把 FlashAttention 搬上昇腾» §二 (equations and
 * the three rules), §五 (persistent programs: here one per SM, each taking
 * (head, tile) work units in turn, and every dQ/dK/dV tile has one writer),
 * §七 (D256: the accumulators split so that they fit; here one gradient at a
 * time).
 *   q, k, v, o, dout : inputs [Z,H,N,D] fp16; o must be fa_fwd's output for
 *                      the same q, k, v, causal and scale.
 *   lse              : input [Z,H,N] fp32 from the same fa_fwd call.
 *   dq, dk, dv       : outputs [Z,H,N,D] fp16, overwritten (not accumulated).
 *   workspace        : device scratch of at least workspace_bytes >=
 *                      fa_bwd_workspace_size(Z,H,N,D,causal) bytes, 256-byte
 *                      aligned; contents on entry are ignored, on exit
 *                      undefined.  Must not be used by another call that runs
 *                      concurrently on the GPU.
 *   other arguments  : as for fa_fwd.
 * Enqueues two persistent kernels on `stream`: first the dQ kernel, which
 * also forms Delta = rowsum(O * dO) and the log2-scaled lse of every query
 * row into the workspace, then the dK/dV kernel, which reads them.
 * Returns FA_OK or a negative FA_ERR_* code.
 */
FA_API int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
           void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int Z, int H, int N, int D,
           int causal, float scale, cudaStream_t stream);

/*
 * bf16 forward and backward.  Source: «把 FlashAttention 搬上昇腾» §九 (every
 * candidate version is checked for correctness in FP16 and in BF16).  Identical to fa_fwd / fa_bwd
 * except that every [Z,H,N,D] tensor (q, k, v, o, dout, dq, dk, dv) is
 * bf16, and P and dS are rounded to bf16 before the matrix unit; lse, Delta,
 * the accumulators and the softmax statistics stay fp32.  Same layout,
 * alignment, ownership, workspace (fa_bwd_workspace_size) and error codes.
 */
FA_API int fa_fwd_bf16(const void* q, const void* k, const void* v, void* o, float* lse, int Z, int H, int N,
                       int D, int causal, float scale, cudaStream_t stream);

FA_API int fa_bwd_bf16(const void* q, const void* k, const void* v, const void* o, const void* dout,
                       const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                       int Z, int H, int N, int D, int causal, float scale, cudaStream_t stream);

/*
 * Grouped K/V heads and different query / key lengths.  Source: «把
 * FlashAttention 搬上昇腾», the GQA Paged Attention part of the contest
 * section: the number of query heads is an integer multiple of the number
 * of K/V heads, several query heads share one K/V head, each sequence has
 * its own context length and the last incomplete block is masked.
 *
 *   q, o, dout, dq : [Z, H, Nq, D]        lse : fp32 [Z, H, Nq]
 *   k, v, dk, dv   : [Z, Hkv, Nk, D]      (H a multiple of Hkv; g = H / Hkv)
 *   Query head h of batch z reads K/V head h / g of batch z (consecutive
 *   query heads share a K/V head).  dk, dv of a shared head are the sums of
 *   the gradients of its g query heads, each written once by one CTA.
 *   Nq, Nk : any lengths >= 1.
 *   causal : the queries are the last Nq positions of an Nk-long sequence:
 *            query i sees key j iff j <= i + (Nk - Nq).  Needs Nq <= Nk
 *            (otherwise some row would see no key): FA_ERR_UNSUPPORTED.
 *   dtype  : FA_DTYPE_F16 or FA_DTYPE_BF16, the element type of every
 *            [.., D] tensor (lse, Delta and accumulation stay fp32).
 * Layout, alignment, ownership, asynchrony and errors as for fa_fwd /
 * fa_bwd; workspace from fa_bwd_ex_workspace_size (0 = unsupported shape).
 * fa_fwd(q, k, v, o, lse, Z, H, N, D, c, s, st) is
 * fa_fwd_ex(q, k, v, o, lse, Z, H, H, N, N, D, c, s, FA_DTYPE_F16, st).
 */
#define FA_DTYPE_F16 0
#define FA_DTYPE_BF16 1
FA_API int fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int Z, int H, int Hkv, int Nq,
                     int Nk, int D, int causal, float scale, int dtype, cudaStream_t stream);

/*
 * Forward over a paged K/V cache.  Source: «把 FlashAttention 搬上昇腾», the
 * contest section's ReshapeAndCache and GQA Paged Attention parts: the cache
 * is kept in physical blocks ("pages") of page_size tokens (token slot s in
 * page s / page_size, row s % page_size); block_tables maps each sequence's
 * logical blocks to physical ones; context_lens gives each sequence's real
 * length and the invalid tokens of its last block are masked; query heads
 * share K/V heads as in fa_fwd_ex.
 *
 *   q, o         : [B, H, Nq, D] (dtype), contiguous, 16-byte aligned.
 *   lse          : fp32 [B, H, Nq].
 *   k_cache,
 *   v_cache      : [num_pages, page_size, Hkv, D] (dtype), 16-byte aligned.
 *   block_table  : int32 [B, max_pages], device memory: sequence b's key p
 *                  is in page block_table[b * max_pages + p / page_size].
 *                  Entries outside [0, num_pages) read as zero keys/values
 *                  (never out of bounds).
 *   context_lens : int32 [B], device memory: sequence b attends to its first
 *                  context_lens[b] keys, clamped to [causal ? Nq : 1,
 *                  max_pages * page_size].
 *   causal       : the Nq queries are the last Nq of the sequence's
 *                  context_lens[b] tokens (query i sees key p iff p <= i +
 *                  context_lens[b] - Nq).
 *   page_size    : 16, 32, 64 or 128, and at most 64 when D = 256.
 * Returns FA_OK (enqueued), FA_ERR_INVALID_ARG (null / misaligned pointer,
 * a size <= 0, H % Hkv != 0, bad dtype / causal / scale),
 * FA_ERR_UNSUPPORTED (D or page_size not supported, sizes past 32-bit
 * indexing), FA_ERR_DEVICE or FA_ERR_CUDA.
 */
/*
 * Paged cache write (ReshapeAndCache).  Source: «把 FlashAttention 搬上昇腾»,
 * the contest section's ReshapeAndCache part: token t's K and V go to block
 * slot_mapping[t] / page_size at offset slot_mapping[t] % page_size of the
 * caches; a negative slot skips the token.
 *   k_new, v_new : [tokens, Hkv, D] 16-bit (fp16 or bf16; copied bit for
 *                  bit), contiguous, 16-byte aligned.
 *   slot_mapping : int64 [tokens], device memory.  Slots >= num_pages *
 *                  page_size are skipped as well (never written out of
 *                  bounds).
 *   k_cache,
 *   v_cache      : [num_pages, page_size, Hkv, D], same element type,
 *                  written in place.
 * tokens == 0 enqueues nothing.  Two tokens with the same slot: one of them
 * wins (unspecified which).  Returns FA_OK, FA_ERR_INVALID_ARG,
 * FA_ERR_UNSUPPORTED (D not 64/128/256), FA_ERR_DEVICE or FA_ERR_CUDA.
 */
FA_API int fa_reshape_and_cache(const void* k_new, const void* v_new, const long long* slot_mapping, void* k_cache,
                                void* v_cache, int tokens, int Hkv, int D, int num_pages, int page_size,
                                cudaStream_t stream);

FA_API int fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                        const int* context_lens, void* o, float* lse, int B, int H, int Hkv, int Nq, int D,
                        int num_pages, int page_size, int max_pages, int causal, float scale, int dtype,
                        cudaStream_t stream);

/*
 * Paged forward with each sequence's key range split into slices, for calls
 * with too few (sequence, head) work items to fill the GPU (decode with a
 * small batch and long contexts).  Source: «把 FlashAttention 搬上昇腾», §一
 * -- the online softmax merges blocks of keys through a running max and sum;
 * whole slices of keys merge the same way: slice s reports lse_s and its own
 * normalised O_s, and lse = log sum_s exp(lse_s), O = sum_s exp(lse_s - lse)
 * O_s.  The result equals fa_fwd_paged's up to rounding.
 *
 *   all arguments as fa_fwd_paged, plus
 *   num_splits      : slices per work item, 1 .. 256; a work item with T key
 *                     tiles (128 keys, 64 at D = 256) uses min(num_splits, T)
 *                     balanced slices.  1 runs fa_fwd_paged's path.
 *   workspace       : device memory of at least
 *                     fa_fwd_paged_split_workspace_size(B, H, Nq, D,
 *                     num_splits) bytes, 16-byte aligned, caller-owned, only
 *                     used by this call on `stream` (fp32 per-slice lse and O).
 *
 * Launches the paged kernel over (work item, slice) units, then a merge
 * kernel that writes o and lse.  Errors as fa_fwd_paged, plus
 * FA_ERR_INVALID_ARG for num_splits out of range and FA_ERR_WORKSPACE for a
 * missing, misaligned or short workspace.
 */
FA_API int fa_fwd_paged_split(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                              const int* context_lens, void* o, float* lse, void* workspace, size_t workspace_bytes,
                              int B, int H, int Hkv, int Nq, int D, int num_pages, int page_size, int max_pages,
                              int num_splits, int causal, float scale, int dtype, cudaStream_t stream);

/* Bytes of workspace fa_fwd_paged_split needs (0 for invalid arguments). */
FA_API size_t fa_fwd_paged_split_workspace_size(int B, int H, int Nq, int D, int num_splits);

/*
 * A slice count for fa_fwd_paged_split on the current device: the largest
 * that keeps every (work item, slice) unit in one wave of the SM count (1
 * when the work items alone fill the GPU), at most the key tiles of the
 * longest context (max_pages * page_size keys) and 256.  Returns 1 for
 * invalid arguments.
 */
FA_API int fa_fwd_paged_split_count(int B, int H, int Hkv, int Nq, int D, int page_size, int max_pages, int causal);

/*
 * Forward over selected blocks of a paged cache.  Source: «把 FlashAttention
 * 搬上昇腾», the contest section's Quest Sparse Attention part: only the
 * chosen (Top-K) blocks of a sequence get exact attention, read through the
 * paged mapping, with per-sequence context lengths and grouped heads.  The
 * choice itself (block scoring, Top-K) is an input of this call.
 *
 *   q, o, lse, k_cache, v_cache, page_size, causal, dtype : as fa_fwd_paged.
 *   sel_pages    : int32 [B, Hkv, max_sel], device: physical pages of the
 *                  selected blocks of sequence b for K/V head kvh.
 *   sel_blocks   : int32 [B, Hkv, max_sel], device: the logical block each
 *                  of them holds (row r is the token at position block *
 *                  page_size + r).
 *   sel_count    : int32 [B, Hkv], device: entries in use (clamped to
 *                  [0, max_sel]).
 *   context_lens : int32 [B], device: tokens at positions >= context_lens[b]
 *                  never take part (the last block's invalid tokens); with
 *                  causal, the queries are the last Nq tokens of the context
 *                  and see positions up to their own.
 * Selected blocks may come in any order.  A query row that sees no selected
 * token gets O = 0 and lse = -inf.  Errors as for fa_fwd_paged.
 */
FA_API int fa_fwd_sparse(const void* q, const void* k_cache, const void* v_cache, const int* sel_pages,
                         const int* sel_blocks, const int* sel_count, const int* context_lens, void* o, float* lse,
                         int B, int H, int Hkv, int Nq, int D, int num_pages, int page_size, int max_sel, int causal,
                         float scale, int dtype, cudaStream_t stream);

FA_API size_t fa_bwd_ex_workspace_size(int Z, int H, int Hkv, int Nq, int Nk, int D, int causal);

FA_API int fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int Z,
                     int H, int Hkv, int Nq, int Nk, int D, int causal, float scale, int dtype, cudaStream_t stream);

/*
 * Scored attention: scores that are capped, biased by distance and restricted
 * to a range of keys per query.  With x = scale * q_i . k_j and the queries
 * the last Nq of the Nk key positions (query i at position i + Nk - Nq):
 *   softcap > 0 : x = softcap * tanh(x / softcap)      (0: not capped)
 *   slopes      : x -= slopes[h] * |i + Nk - Nq - j|, slopes fp32 [H] in
 *                 device memory, by query head          (NULL: no bias)
 *   visible     : key j takes part for query i iff it lies in the row's range
 *                 of `key_ranges` (NULL: 0 <= j < Nk), j <= i + Nk - Nq
 *                 when causal, and j > i + Nk - Nq - window when window > 0
 *                 (needs causal).
 * Then o = softmax(x) v and lse as for fa_fwd_ex; a query that sees no key
 * gets o = 0 and lse = -inf.  Values in keys that no query of a 128-row tile
 * sees may be anything, NaN included, also between given ranges; a NaN or
 * infinity in the V of a key that some query of the tile sees reaches the
 * tile's other rows that see any key.  The arithmetic is fa_fwd_ex's; x is
 * computed in fp32 with an absolute error of a few 2^-24 of softcap.
 *
 * fa_key_ranges fills the buffer `mask` (fa_key_ranges_size bytes, 16-byte
 * aligned, device memory) from exactly one of
 *   doc_ids     : int32 [Z, Nk]: a query sees the run of equal ids that its
 *                 position lies in (packed documents; combine with causal);
 *   prefix_lens : int32 [Z]: a query sees keys up to its own position, and
 *                 the first prefix_lens[z] keys (bidirectional prefix);
 *   ranges      : int32 [Z, Nq, 2]: keys lo <= j < hi (lo >= hi: none), 8-byte
 *                 aligned.
 * The buffer serves any number of forward and backward calls of the same Z,
 * Nq and Nk.  doc_ids and prefix_lens need Nq <= Nk.
 * Errors as for fa_fwd_ex, plus FA_ERR_INVALID_ARG for a negative or not
 * finite softcap, a negative window or a window without causal,
 * FA_ERR_UNSUPPORTED for a softcap above 4096 (whose scores would be off by as
 * much as P is rounded) or so small that scale / softcap overflows, and
 * FA_ERR_WORKSPACE for a mask buffer that is missing or too small.
 */
FA_API size_t fa_key_ranges_size(int Z, int Nq, int Nk);
FA_API int fa_key_ranges(const int* doc_ids, const int* prefix_lens, const int* ranges, void* mask, size_t mask_bytes,
                         int Z, int Nq, int Nk, cudaStream_t stream);

FA_API int fa_fwd_scored(const void* q, const void* k, const void* v, void* o, float* lse, int Z, int H, int Hkv, int Nq,
                         int Nk, int D, int causal, float scale, float softcap, const float* slopes, int window,
                         const void* key_ranges, size_t key_ranges_bytes, int dtype, cudaStream_t stream);

/*
 * Backward of fa_fwd_scored, with the same rules: p = exp(x - lse), dx = p
 * (do . v - rowsum(o do)) (1 - tanh^2(scale q . k / softcap)), dq = scale dx
 * k, dk = scale dx^T q, dv = p^T do.  Rows and keys that take part nowhere get
 * zeros, and whatever their inputs hold stays out of the others' gradients; a
 * NaN or infinity in one that takes part reaches the gradients of the 128-row
 * tiles that it meets.  slopes have no gradient.  Workspace, layout and errors as for
 * fa_bwd_ex (fa_bwd_ex_workspace_size).
 */
FA_API int fa_bwd_scored(const void* q, const void* k, const void* v, const void* o, const void* dout,
                         const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int Z,
                         int H, int Hkv, int Nq, int Nk, int D, int causal, float scale, float softcap,
                         const float* slopes, int window, const void* key_ranges, size_t key_ranges_bytes, int dtype,
                         cudaStream_t stream);

/*
 * Scored attention of a chunk of new tokens over a paged cache.  Cache, block
 * table, page sizes, D and dtype as for fa_fwd_paged, splits and workspace as
 * for fa_fwd_paged_split (num_splits == 1: none needed), softcap, slopes and
 * window as for fa_fwd_scored, and
 *   context_lens : int32 [B]: keys of each sequence, clamped to [0, max_pages
 *                  * page_size] (0: its rows see nothing).
 *   q_lens       : int32 [B] or NULL: sequence b has q_lens[b] new tokens (NULL:
 *                  Nq), clamped to [0, Nq]; they are the first q_lens[b] of its
 *                  Nq rows and the last of its context (row i at position
 *                  context_lens[b] - q_lens[b] + i).  Rows behind them, and rows
 *                  before position 0, get o = 0 and lse = -inf.
 */
FA_API int fa_fwd_paged_scored(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                               const int* context_lens, const int* q_lens, void* o, float* lse, void* workspace,
                               size_t workspace_bytes, int B, int H, int Hkv, int Nq, int D, int num_pages,
                               int page_size, int max_pages, int num_splits, int causal, float scale, float softcap,
                               const float* slopes, int window, int dtype, cudaStream_t stream);

/*
 * A slice count for fa_fwd_paged_scored on the current device (1 for invalid
 * arguments): slices in whole waves of the SM count, of at least a few key
 * tiles each.  Heads of at most 32 rows (H / Hkv * Nq, D <= 128) run four
 * slices per work unit where num_splits is 4 or more (num_splits / 4 units per
 * head), and should.
 */
FA_API int fa_fwd_paged_scored_split_count(int B, int H, int Hkv, int Nq, int D, int page_size, int max_pages,
                                           int causal);

/*
 * Attention within a causal window that also sees the first tokens (sinks):
 * fa_fwd_scored, fa_bwd_scored and fa_fwd_paged_scored with causal 1, and
 *   visible : key j takes part for the query at position p iff j <= p, and
 *             j > p - window or j < sinks.
 * sinks 0 is the window alone; sinks > 0 needs window > 0
 * (FA_ERR_INVALID_ARG).  Capped scores (softcap) as there; a distance bias or
 * key ranges do not go with sinks and are no arguments of these calls.
 * Keys between the sinks and the windows of a 128-row query tile are not read
 * (whole key tiles; paged: whole pages), and may hold anything.
 *
 * fa_bwd_sinks: the dK and dV of sinks, which all later queries see, are summed
 * over parts of the queries in fp32, in the workspace, and joined in a fixed
 * order; hence a workspace of fa_bwd_sinks_workspace_size bytes (0: invalid
 * arguments), 256-byte aligned.  o and lse are fa_fwd_sinks's own for the same
 * arguments: for the sinks, rowsum(o do) is taken from sum_j p_j (do . v_j), in fp32,
 * which an o over other keys than this call's is not.
 * fa_fwd_paged_sinks_split_count: as fa_fwd_paged_scored_split_count, for the
 * keys that such a call reads.
 */
FA_API int fa_fwd_sinks(const void* q, const void* k, const void* v, void* o, float* lse, int Z, int H, int Hkv, int Nq,
                        int Nk, int D, float scale, float softcap, int window, int sinks, int dtype,
                        cudaStream_t stream);

FA_API size_t fa_bwd_sinks_workspace_size(int Z, int H, int Hkv, int Nq, int Nk, int D, int window, int sinks);

FA_API int fa_bwd_sinks(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                        void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int Z, int H, int Hkv,
                        int Nq, int Nk, int D, float scale, float softcap, int window, int sinks, int dtype,
                        cudaStream_t stream);

FA_API int fa_fwd_paged_sinks(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                              const int* context_lens, const int* q_lens, void* o, float* lse, void* workspace,
                              size_t workspace_bytes, int B, int H, int Hkv, int Nq, int D, int num_pages,
                              int page_size, int max_pages, int num_splits, float scale, float softcap, int window,
                              int sinks, int dtype, cudaStream_t stream);

FA_API int fa_fwd_paged_sinks_split_count(int B, int H, int Hkv, int Nq, int D, int page_size, int max_pages,
                                          int window, int sinks);

/*
 * Rotary positions of q [Z, H, N, D] and k [Z, Hkv, N, D] (Hkv = 0: q alone).
 * Pair j of a head's first `rot` values is turned by the angle positions[z, n]
 * * freqs[j] (radians, the product taken in at least 64 bits) and scaled by
 * mscale:
 *   y0 = mscale (x0 cos a - x1 sin a),  y1 = mscale (x1 cos a + x0 sin a);
 * interleaved 0: pairs (j, j + rot / 2); 1: pairs (2 j, 2 j + 1).  Values past
 * rot are copied.  inverse 1 turns by -a: the gradient of the turn.
 *   *_strides : host arrays of three strides, in elements, of (sequence, head,
 *               token); the D values of a row are contiguous.  Rows whose
 *               addresses are multiples of 16 bytes, with rot a multiple of
 *               16, move 16 bytes at a time.  Outputs may be the inputs
 *               themselves (same strides) but overlap them, or themselves, in no
 *               other way.
 *   positions : int64, device: token n of sequence z at z * positions_stride +
 *               n (stride 0: shared by all sequences); any value.
 *   freqs     : fp64 [rot / 2], device: radians per position, finite.
 *   D 64, 128 or 256; rot even, at most D.
 *
 * fa_rotary_and_cache turns q into q_out, and writes the turned k_new and
 * v_new (as they are) [Z, Hkv, N, D] to the cache rows slot_mapping[z * N + n]
 * as fa_reshape_and_cache does (negative slots and slots past the cache are
 * skipped; q rows are written all the same).  Two tokens with the same slot: each
 * 16 bytes of the row (each value, where rows do not move 16 bytes at a time)
 * are one of theirs, unspecified whose.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (D, rot, sizes),
 * FA_ERR_DEVICE, FA_ERR_CUDA.
 */
FA_API int fa_rotary(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
                     const void* k, const long long* k_strides, void* k_out, const long long* k_out_strides,
                     const long long* positions, long long positions_stride, const double* freqs, int Z, int H,
                     int Hkv, int N, int D, int rot, int interleaved, int inverse, float mscale, int dtype,
                     cudaStream_t stream);

FA_API int fa_rotary_and_cache(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
                               const void* k_new, const long long* k_strides, const void* v_new,
                               const long long* v_strides, const long long* positions, long long positions_stride,
                               const double* freqs, const long long* slot_mapping, void* k_cache, void* v_cache, int Z,
                               int H, int Hkv, int N, int D, int rot, int interleaved, float mscale, int num_pages,
                               int page_size, int dtype, cudaStream_t stream);

/*
 * The same with several axes (time, height and width of image and video
 * tokens, say): pair j is turned by the angle position_a * freqs[j], a =
 * axes[j], where position_a is the token's position on axis a.
 *   positions : int64, device: that of token n of sequence z on axis a at a *
 *               axis_stride + z * positions_stride + n.
 *   axes      : int32 [rot / 2], device: the axis of each pair; one outside
 *               [0, num_axes) is not turned (it is scaled by mscale).
 *   num_axes  : >= 1.
 * Everything else as for fa_rotary and fa_rotary_and_cache.
 */
FA_API int fa_rotary_axes(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
                          const void* k, const long long* k_strides, void* k_out, const long long* k_out_strides,
                          const long long* positions, long long positions_stride, long long axis_stride,
                          const int* axes, int num_axes, const double* freqs, int Z, int H, int Hkv, int N, int D,
                          int rot, int interleaved, int inverse, float mscale, int dtype, cudaStream_t stream);

FA_API int fa_rotary_and_cache_axes(const void* q, const long long* q_strides, void* q_out,
                                    const long long* q_out_strides, const void* k_new, const long long* k_strides,
                                    const void* v_new, const long long* v_strides, const long long* positions,
                                    long long positions_stride, long long axis_stride, const int* axes, int num_axes,
                                    const double* freqs, const long long* slot_mapping, void* k_cache, void* v_cache,
                                    int Z, int H, int Hkv, int N, int D, int rot, int interleaved, float mscale,
                                    int num_pages, int page_size, int dtype, cudaStream_t stream);

/*
 * The paged cache's tables, kept on the GPU (nothing here reads them back), so
 * that a serving loop's steps can be captured in a graph.  Pages that nobody
 * holds are a stack: free_pages int32 [num_pages], of which the first *free_count
 * (int32, clamped to [0, num_pages]) are free, the last of them the next to go.
 *
 * fa_cache_step takes pages for a step's new tokens and says where they go:
 *   cached_lens  : int32 [B]: tokens that each sequence has (negative: 0).
 *   q_lens       : int32 [B] or NULL (N): new tokens, clamped to [0, N].
 *   block_table  : int32 [B, max_pages], as for fa_fwd_paged: the entries of the
 *                  pages that the new tokens begin are written, in the order of
 *                  sequences and pages; others are left as they are.
 *   slot_mapping : int64 [B, N], as for fa_reshape_and_cache: the cache row of
 *                  new token n of sequence b; -1 for rows behind the new tokens,
 *                  for tokens past max_pages pages and for those whose page is
 *                  not in [0, num_pages).
 *   positions    : int64 [B, N], as for fa_rotary: cached_lens[b] + n, all rows.
 *   context_lens : int32 [B]: cached and new tokens, for fa_fwd_paged (may be
 *                  cached_lens itself).
 *   free_count_out : int32: the stack's height after the step (may be free_count
 *                  itself).  Negative: so many pages were missing; their table
 *                  entries are -1, and their tokens have no slot.
 * The lengths count tokens without a slot too.  A sequence that outgrows its
 * max_pages pages has to end before: fa_fwd_paged and its like clamp lengths to
 * the table, and would take its last rows for earlier positions.
 *
 * fa_cache_release gives back the pages of the sequences b with finished[b] != 0
 * (bytes [B]): the entries of their first context_lens[b] tokens that lie in [0,
 * num_pages) go onto the stack in the order of sequences and pages (past
 * num_pages: dropped).  Pages of other sequences stay theirs, also those that a
 * window has passed.  A page belongs to one sequence: one that two rows name is
 * pushed twice, and would be handed out twice.  context_lens_out is 0 for them and
 * context_lens for the others; the block table is left as it is.  Outputs may be
 * context_lens and free_count themselves.  workspace:
 * fa_cache_release_workspace_size(B) bytes, 4-byte aligned, used by this call alone
 * while it runs.
 * Outputs overlap no input but as said.  Errors: FA_ERR_INVALID_ARG,
 * FA_ERR_UNSUPPORTED (B * max_pages + num_pages past 32 bits),
 * FA_ERR_WORKSPACE, FA_ERR_DEVICE, FA_ERR_CUDA.
 */
FA_API int fa_cache_step(const int* free_pages, const int* free_count, int* block_table, const int* cached_lens,
                         const int* q_lens, long long* slot_mapping, long long* positions, int* context_lens,
                         int* free_count_out, int B, int N, int num_pages, int page_size, int max_pages,
                         cudaStream_t stream);

FA_API size_t fa_cache_release_workspace_size(int B);

FA_API int fa_cache_release(int* free_pages, const int* free_count, const int* block_table, const int* context_lens,
                            const unsigned char* finished, int* context_lens_out, int* free_count_out, void* workspace,
                            size_t workspace_bytes, int B, int num_pages, int page_size, int max_pages,
                            cudaStream_t stream);

/*
 * Backward pass that allocates nothing and takes no workspace.
 *
 * The attention pages have no counterpart to this call; it exists for
 * callers that cannot allocate device memory when they run the backward --
 * for example code that runs inside a fixed memory pool or arena it does not
 * own, or an embedding host whose allocator must not be re-entered.
 *
 * It computes exactly what fa_bwd computes (same kernels, same arguments
 * without workspace/workspace_bytes, same outputs bit for bit), but the
 * scratch that fa_bwd takes from the caller (Delta and the log2-scaled
 * lse) lives in one static device buffer of FA_NOALLOC_SCRATCH_BYTES (64 MiB)
 * compiled into libfa.so.  Every GPU on which the library is used holds that
 * buffer until the process exits.
 *
 *   Limit  : fa_bwd_workspace_size(Z,H,N,D,causal) (about 8*Z*H*N bytes) must
 *            fit in the buffer; otherwise FA_ERR_SCRATCH_LIMIT is returned
 *            before anything is enqueued.
 *   Set-up : the first call on a device (with that device current) looks up
 *            the buffer's device address; make that first call before any
 *            stream capture.
 *   Sharing: all calls share the one buffer and it keeps the last call's
 *            contents.  Nothing in it needs clearing -- each call writes
 *            every scratch element it reads -- but calls whose kernels may
 *            overlap on the GPU (different streams, other host threads)
 *            race on it: serialise them.
 * Returns FA_OK or a negative FA_ERR_* code.
 */
#define FA_NOALLOC_SCRATCH_BYTES (64ull << 20)
FA_API int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dout,
                          const float* lse, void* dq, void* dk, void* dv, int Z, int H, int N, int D, int causal,
                          float scale, cudaStream_t stream);

/*
 * Synchronises `stream`, then returns and clears the device status word of
 * the current device: FA_OK, FA_ERR_TIMEOUT (a kernel wait gave up; the
 * outputs of the calls since the last check are invalid) or FA_ERR_CUDA.
 */
FA_API int fa_device_status(cudaStream_t stream);

/*
 * Like fa_device_status but also returns the raw status word (timeout site in
 * bits 8 and up) through *raw when raw is not NULL.
 */
FA_API int fa_device_status_raw(cudaStream_t stream, int* raw);

/*
 * Self-test of the failure-detection path: enqueues one tiny kernel on
 * `stream` that waits on a shared-memory barrier nothing ever signals, using
 * the same bounded wait as every kernel of the library.  The wait gives up
 * after about one second, records FA_ERR_TIMEOUT with site code 200 in the
 * device status word and the kernel returns normally, so the context stays
 * usable.  Callers then see FA_ERR_TIMEOUT from fa_device_status().
 * Returns FA_OK once enqueued, FA_ERR_CUDA or FA_ERR_DEVICE otherwise.
 */
FA_API int fa_selftest_wait_timeout(cudaStream_t stream);

/* Static, human-readable description of an FA_* code. */
FA_API const char* fa_error_string(int code);

/*
 * Number of (query tile, key tile) pairs one head's pass visits with the
 * dense forward's tiling (128-row query tiles and 128-key tiles for every D,
 * the last of each possibly partial): the causal loop bound of §八 (T*T tiles
 * non-causal, 1+2+...+T causal for square tiles).  Host-only helper used
 * for the FLOP model; -1 on bad arguments.
 */
FA_API long long fa_fwd_tile_count(int N, int D, int causal);

/*
 * Algorithmic FLOPs of one call over all heads (the work the method must do,
 * not counting what it avoids): forward 4*N*N*D non-causal, 2*N*(N+1)*D
 * causal, per head; backward 2.5x that (five GEMMs incl. the recompute of P).
 */
FA_API double fa_fwd_flops(int Z, int H, int N, int D, int causal);
FA_API double fa_bwd_flops(int Z, int H, int N, int D, int causal);

/*
 * The same for the fa_fwd_ex / fa_bwd_ex shapes: 4*D per visible (query,
 * key) pair per query head, Nq*Nk pairs non-causal, Nq*(Nq+1)/2 +
 * Nq*(Nk-Nq) causal; backward 2.5x.
 */
FA_API double fa_fwd_ex_flops(int Z, int H, int Nq, int Nk, int D, int causal);
FA_API double fa_bwd_ex_flops(int Z, int H, int Nq, int Nk, int D, int causal);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_H */
