/*
 * pagedattn.h -- C ABI of the GB300 (sm_103a) paged KV-cache attention library
 * (libpagedattn.so).
 *
 * What it computes: O = softmax(scale * Q K^T) V per query head, optionally
 * causal (bottom-right aligned: query row i of Lq sees keys t <= i + Lk - Lq),
 * for MHA and GQA (query head h reads kv head h / (Hq/Hkv)).  K and V are read
 * through a per-sequence block table of pages of 16 to 256 tokens (or from a
 * contiguous cache), with per-sequence lengths taken from device arrays -- the flash_attn_with_kvcache /
 * flash_attn_varlen_func interface discussed on
 *   flash-attention #824 "Add support for small page sizes" (reproduction
 *     snippet; page size 16; k=/v= append through block_table),
 *   vLLM #6052 "Unify the kernel used in flash attention backend" (one varlen
 *     launch for prefill and decode; CUDA-graph padding rules),
 *   flash-attention #1000 "Inappropriate Number of Splits Predicted by
 *     determine_num_splits" (split-KV on a preallocated contiguous cache;
 *     cache_seqlens lives on the GPU and must not be read by the host),
 *   vLLM #3010 "Introduce flash-attn (>= 2.5.0)" (paged decode and
 *     prefill-with-cache-write benchmarks, MHA and GQA).
 *
 * Conventions shared by every entry point
 *   - All pointers are DEVICE pointers owned by the caller, except where a
 *     comment says otherwise.  The library allocates nothing and never
 *     synchronises; every call is ordered on `stream` (a cudaStream_t; 0 is
 *     the legacy default stream) and reads lengths only on the GPU.
 *   - Element types: PA_F16 or PA_BF16; q, caches, new k/v and out share it.
 *     Softmax statistics, partial outputs and LSE are fp32.  LSE is the
 *     natural-log log-sum-exp of the scaled scores; rows with no visible key
 *     produce O = 0 and LSE = -inf.
 *   - head_dim D must be 64 or 128; a paged cache's page size is 16, 32, 64,
 *     128 or 256 tokens (page_size argument); Hq must be a multiple of Hkv.
 *   - Cache tensors are described by pa_tensor4 (element strides; the D axis
 *     is contiguous).  Base pointers must be 16-byte aligned and all three
 *     strides multiples of 8 elements (16 bytes), because K/V tiles are
 *     fetched with the Tensor Memory Accelerator.
 *   - Return value: PA_OK (0) or a negative PA_ERR_* code for a rejected
 *     argument or a failed launch.  Errors the GPU finds while running
 *     (block-table entries outside the pool, lengths beyond the table or the
 *     cache, a pipeline wait that timed out) are written to `err_word`
 *     (int32[4] in device memory, zeroed by the caller; may be NULL):
 *     err_word[0] = first PA_DEVERR_* code, [1] = sequence index, [2] = the
 *     offending value.  The kernels never fault on such input: an out-of-range
 *     page is replaced by page 0 for reading and is never written.
 *   - pa_last_error_string() describes the last non-OK return on the calling
 *     thread.
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

typedef struct CUstream_st* pa_stream_t; /* same type as cudaStream_t */

enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = -1, /* null pointer, negative size, bad stride or alignment */
  PA_ERR_UNSUPPORTED = -2, /* dtype, head_dim, Hq % Hkv, or shape outside the kernels */
  PA_ERR_CUDA = -3,        /* a CUDA runtime call or kernel launch failed */
  PA_ERR_WORKSPACE = -4    /* workspace pointer NULL or smaller than required */
};

/* PA_E4M3: 8-bit cache values (four exponent, three mantissa bits, largest 448), each
 * standing for itself times its kv head's fp32 scale; only where a call says so.
 * PA_F32: rotary tables of pa_rotary_append_varlen, logits of pa_beam_select. */
enum { PA_F16 = 0, PA_BF16 = 1, PA_E4M3 = 2, PA_F32 = 3 };

/* Codes written to err_word[0] by the kernels. */
enum {
  PA_DEVERR_PAGE_OOB = 1,    /* block_table entry < 0 or >= num_pages            */
  PA_DEVERR_LENGTH = 2,      /* length < 0, beyond the table, cache or max_seqlen_k */
  PA_DEVERR_TIMEOUT = 3,     /* a pipeline wait exceeded its time limit          */
  PA_DEVERR_CAPACITY = 4,    /* the page pool or the packed rows do not suffice  */
  PA_DEVERR_VALUE = 5        /* a beam's logits or parent that stand for nothing */
};

/* A 4-D cache view.  Paged: [num_pages, page_size, Hkv, D] with stride_b =
 * elements between pages, stride_t between the token slots of a page,
 * stride_h between kv heads.  Contiguous (block_table == NULL):
 * [B, capacity, Hkv, D] with stride_b between sequences.
 *
 * page_size (the paged calls' argument): tokens per page, one of 16, 32, 64,
 * 128, 256 -- vLLM's 16-token blocks and the 256-token pages flash-attention
 * required, which vLLM #3010 "Introduce flash-attn" compares (cache-write cost
 * at context 512 / 1024).  Ignored when block_table == NULL; any other value
 * with a block table returns PA_ERR_UNSUPPORTED.  Position pos of sequence b
 * is in page block_table[b * bt_stride + pos / page_size], slot
 * pos % page_size. */
typedef struct {
  void* ptr;
  int64_t stride_b;
  int64_t stride_t;
  int64_t stride_h;
} pa_tensor4;

/*
 * pa_append_kv -- write new tokens' k/v into the cache (a bit copy).
 *
 * For every b < B, i < Lnew, kv head g: position pos = cache_seqlens[b] + i
 * receives k_new[b, i, g, :] (and v_new likewise) at page
 * block_table[b * bt_stride + pos / page_size], slot pos % page_size; or, with
 * block_table == NULL, at row [b, pos] of a contiguous cache.  The k=/v=
 * append of flash_attn_with_kvcache (flash-attention #824, reproduction
 * snippet and the reply noting that the call allocates nothing and writes
 * through block_table).  cache_seqlens is input only and is not updated.
 *
 *   k_new, v_new  [B, Lnew, Hkv, D] contiguous.
 *   block_table   int32 [B, >= max_pages] rows of stride bt_stride, or NULL.
 *   cache_extent  paged: number of pages in the pool; contiguous: capacity
 *                 (tokens) of each sequence.
 * Positions outside the table (pos / page_size >= max_pages) or the capacity, and
 * out-of-pool pages, are skipped and reported in err_word.  Appends of two
 * sequences that share a physical page race (the caller's responsibility).
 */
PA_API int pa_append_kv(pa_tensor4 k_cache, pa_tensor4 v_cache, const void* k_new,
                        const void* v_new, const int32_t* cache_seqlens,
                        const int32_t* block_table, int64_t bt_stride, int max_pages,
                        int page_size, int B, int Lnew, int Hkv, int D, int64_t cache_extent,
                        int dtype, int32_t* err_word, pa_stream_t stream);

/*
 * pa_fwd_kvcache -- flash_attn_with_kvcache forward: decode, multi-query
 * decode and causal prefill over a paged (or contiguous) cache, with optional
 * in-kernel append and split-KV.
 *
 * Sequence b attends over Lk_b = cache_seqlens[b] + Lnew keys: positions
 * below cache_seqlens[b] come from the cache, positions at or above it are
 * the Lnew new tokens, which are also written into the cache (as
 * pa_append_kv) in the same call.  (flash-attention #824: reproduction
 * snippet; flash-attention #1000: split-KV and the host-side num_splits
 * problem; vLLM #3010: paged decode table.)
 *
 *   q            [B, Lq, Hq, D], element strides q_sb, q_st, q_sh (multiples
 *                of 8); D contiguous.
 *   k_new/v_new  [B, Lnew, Hkv, D] contiguous, or NULL with Lnew == 0.
 *   cache_seqlens int32 [B] (device): tokens already cached.
 *   block_table  int32 [B, >= max_pages] (row stride bt_stride) or NULL for a
 *                contiguous cache; entries past ceil(Lk_b/page_size) are never
 *                read.  page_size: see pa_tensor4.
 *   cache_extent paged: pages in the pool; contiguous: tokens per sequence.
 *   max_seqlen_k host-known upper bound of Lk_b (a capacity, never read back).
 *   scale        softmax scale (e.g. 1/sqrt(D)).
 *   num_splits   0: split-KV count chosen on the GPU from cache_seqlens;
 *                >= 1: at most that many splits per sequence.
 *   out          [B, Lq, Hq, D] contiguous; lse fp32 [B, Hq, Lq] or NULL.
 *   workspace    device scratch of pa_fwd_kvcache_workspace_size(...) bytes
 *                (may be NULL when that size is 0).  Its contents on entry do
 *                not matter.
 * Which kernel runs depends on the query rows per kv head, Lq * (Hq / Hkv):
 *   <= 2     the split-KV decode kernel, CUDA-core consumers;
 *   3 - 16   the split-KV decode kernel, warp-level tensor-core consumer;
 *   17 - 128 the tcgen05 engine, all query heads of a kv head packed in one
 *            tile, split-KV, followed by the combine kernel when it splits;
 *   > 128    the tcgen05 prefill kernel, two 128-row query tiles per CTA.
 * The decode kernel appends k_new / v_new in the same launch and merges its
 * splits in the same launch (one launch per call); the engine and prefill
 * paths run the append kernel first.
 */
PA_API int pa_fwd_kvcache(const void* q, int64_t q_sb, int64_t q_st, int64_t q_sh,
                          pa_tensor4 k_cache, pa_tensor4 v_cache, const void* k_new,
                          const void* v_new, int Lnew, const int32_t* cache_seqlens,
                          const int32_t* block_table, int64_t bt_stride, int max_pages,
                          int page_size, int B, int Lq, int Hq, int Hkv, int D,
                          int64_t cache_extent, int max_seqlen_k,
                          float scale, int causal, int num_splits, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, int32_t* err_word, int dtype,
                          pa_stream_t stream);

/* Bytes of workspace pa_fwd_kvcache needs for these sizes (0 if none). */
PA_API size_t pa_fwd_kvcache_workspace_size(int B, int Lq, int Hq, int Hkv, int D,
                                            int max_seqlen_k, int num_splits);

/*
 * pa_fwd_kvcache_rotary -- pa_fwd_kvcache with rotary position embedding of
 * the new tokens.  flash-attention #824 "Add support for small page sizes"
 * names the feature (a fix to fused RoPE embeddings in this forward) without
 * defining it; the rotation is the published RoFormer one:
 *
 *   - features [0, rotary_dim) are rotated, the rest pass through;
 *   - rotary_interleaved == 0: feature p pairs with p + rotary_dim / 2;
 *     otherwise feature 2p pairs with 2p + 1;
 *   - a pair (x1, x2) of a token at position pos becomes
 *     (x1 c - x2 s, x1 s + x2 c), c = rotary_cos[pos][p], s = rotary_sin[pos][p].
 *
 * Positions: new token i of sequence b is at cache_seqlens[b] + i (the slot the
 * append writes it to); query row i of Lq is at cache_seqlens[b] + Lnew - Lq + i.
 * The rotated k is what the append stores in the cache; the rotated q is what
 * attends.  The rotation is computed in fp32 and rounded once to the dtype.
 *
 * Arguments are those of pa_fwd_kvcache plus
 *   rotary_cos, rotary_sin  [rotary_len, rotary_dim / 2], row-major, dtype of q;
 *                           device memory owned by the caller.
 *   rotary_len              rows of the tables; a position >= rotary_len
 *                           leaves the token unrotated and records
 *                           PA_DEVERR_LENGTH (sequence, position) in err_word.
 *   rotary_dim              even, 2 <= rotary_dim <= D.
 * Requires Lnew >= 1 (the rotation applies to appended tokens).  workspace:
 * pa_fwd_kvcache_rotary_workspace_size bytes, 256-byte aligned.
 * Query blocks of up to 16 rows per kv head (Lq * Hq / Hkv <= 16: decode,
 * GQA decode, short multi-query decode) are rotated inside the attention
 * launch: q as it is staged for the kernel, k_new where the fused append
 * stores it; the workspace is then pa_fwd_kvcache's own.  Longer query
 * blocks run one extra kernel (the rotation into the workspace, ahead of
 * pa_fwd_kvcache's own scratch) before the attention launches.  Same return
 * codes as pa_fwd_kvcache.
 */
PA_API int pa_fwd_kvcache_rotary(const void* q, int64_t q_sb, int64_t q_st, int64_t q_sh,
                                 pa_tensor4 k_cache, pa_tensor4 v_cache, const void* k_new,
                                 const void* v_new, int Lnew, const int32_t* cache_seqlens,
                                 const int32_t* block_table, int64_t bt_stride, int max_pages,
                                 int page_size, int B, int Lq, int Hq, int Hkv, int D,
                                 int64_t cache_extent, int max_seqlen_k, const void* rotary_cos,
                                 const void* rotary_sin,
                                 int rotary_len, int rotary_dim, int rotary_interleaved,
                                 float scale, int causal, int num_splits, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, int32_t* err_word,
                                 int dtype, pa_stream_t stream);

/* Bytes of workspace pa_fwd_kvcache_rotary needs for these sizes. */
PA_API size_t pa_fwd_kvcache_rotary_workspace_size(int B, int Lq, int Hq, int Hkv, int D, int Lnew,
                                                   int max_seqlen_k, int num_splits);

/*
 * pa_fwd_kvcache_noalloc -- pa_fwd_kvcache for callers that cannot allocate
 * device memory.  (No counterpart on the pages: this is a library-usage entry
 * point, not part of the attention method.)
 *
 * Some callers cannot call cudaMalloc: code running inside another library's
 * allocator or stream callback, serving processes whose device memory pool is
 * owned and capped by the framework, or latency paths that must never reach
 * the driver's allocator.  They can pass inputs and outputs but not the
 * split-KV scratch that pa_fwd_kvcache takes as `workspace`.  This variant
 * takes the same arguments minus the workspace and uses a fixed scratch array
 * of PA_NOALLOC_SCRATCH_BYTES that every GPU using the library holds until the
 * process exits.  It calls no allocating routine.
 *
 *   - Sizes whose split scratch (pa_fwd_kvcache_workspace_size) exceeds
 *     PA_NOALLOC_SCRATCH_BYTES are rejected with PA_ERR_WORKSPACE.
 *   - The first call on a device looks up the array's device address (once
 *     per device, with that device current).  Under CUDA's lazy module
 *     loading that lookup may load the library's device code on that device,
 *     which allocates in the driver (the array included): make the first call
 *     during set-up -- outside allocator hooks and before any stream capture.
 *   - All calls share the array, which keeps the last call's contents; no
 *     entry needs to start at zero.  Calls whose kernels overlap on the GPU
 *     (other streams, other threads) race on it: serialise them.
 */
#define PA_NOALLOC_SCRATCH_BYTES (8 << 20)
PA_API int pa_fwd_kvcache_noalloc(const void* q, int64_t q_sb, int64_t q_st, int64_t q_sh,
                                  pa_tensor4 k_cache, pa_tensor4 v_cache, const void* k_new,
                                  const void* v_new, int Lnew, const int32_t* cache_seqlens,
                                  const int32_t* block_table, int64_t bt_stride, int max_pages,
                                  int page_size,
                                  int B, int Lq, int Hq, int Hkv, int D, int64_t cache_extent,
                                  int max_seqlen_k, float scale, int causal, int num_splits,
                                  void* out, float* lse, int32_t* err_word, int dtype,
                                  pa_stream_t stream);

/*
 * pa_fwd_varlen_unified -- one launch for a mixed batch of chunked-prefill
 * and decode sequences over a paged cache (vLLM #6052 "Unify the kernel used
 * in flash attention backend": a single varlen kernel for prefill, decode and
 * chunked prefill; cumulative query lengths padded with repeated entries).
 *
 *   q             [total_q, Hq, D], element strides q_st, q_sh; packed by
 *                 cu_seqlens_q.
 *   cu_seqlens_q  int32 [B+1], non-decreasing, cu_seqlens_q[0] == 0.  A
 *                 sequence with no query rows (a padding entry) writes nothing.
 *   seqlens_k     int32 [B]: keys of sequence b, INCLUDING its new chunk,
 *                 which must already be in the cache (pa_append_kv).
 *   max_seqlen_q, max_seqlen_k  host-known capacities (grid sizing only).
 *   out [total_q, Hq, D] contiguous; lse fp32 [Hq, total_q] or NULL.
 *   workspace     pa_fwd_varlen_workspace_size(...) bytes.
 * The tcgen05 engine runs the whole batch in one launch: sequences of up to
 * 128 query rows per kv head as packed (split-KV) items, longer chunks as
 * pairs of 128-row query tiles, each CTA taking a contiguous run of work
 * units of equal estimated cost; when a decode sequence is split, the combine
 * kernel follows as a programmatic dependent launch.  At most 4096 entries
 * (B, padding entries included); more return PA_ERR_UNSUPPORTED.
 */
PA_API int pa_fwd_varlen_unified(const void* q, int64_t q_st, int64_t q_sh, pa_tensor4 k_cache,
                                 pa_tensor4 v_cache, const int32_t* cu_seqlens_q,
                                 const int32_t* seqlens_k, const int32_t* block_table,
                                 int64_t bt_stride, int max_pages, int page_size, int B,
                                 int total_q,
                                 int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int D,
                                 int64_t num_pages, float scale, int causal, void* out,
                                 float* lse, void* workspace, size_t workspace_bytes,
                                 int32_t* err_word, int dtype, pa_stream_t stream);

PA_API size_t pa_fwd_varlen_workspace_size(int B, int total_q, int max_seqlen_q, int Hq,
                                           int Hkv, int D, int max_seqlen_k);

/*
 * pa_split_combine -- merge split-KV partial results (the combine step that
 * follows flash_fwd_splitkv_kernel, vLLM #6052 comment on num_splits == 0 with
 * a page table; flash-attention #1000).
 *
 * For each b < B, query row i < Lq, head h < Hq with n = splits_per_seq[b]
 * (or S when splits_per_seq == NULL):
 *   LSE = ln sum_{s<n} exp(LSE_s),  O = sum_{s<n} exp(LSE_s - LSE) O_s,
 * where O_s = o_partial[s, b, i, h, :] is the NORMALISED output of split s
 * and LSE_s = lse_partial[s, b, i, h] (-inf for an empty split, whose O_s is
 * then never read).  Rows whose n is 0 are left untouched; n is clamped to S.
 *   o_partial fp32 [S, B, Lq, Hq, D]; lse_partial fp32 [S, B, Lq, Hq];
 *   out [B, Lq, Hq, D] (dtype); lse fp32 [B, Hq, Lq] or NULL.
 */
PA_API int pa_split_combine(const float* o_partial, const float* lse_partial,
                            const int32_t* splits_per_seq, int S, int B, int Lq, int Hq, int D,
                            void* out, float* lse, int dtype, pa_stream_t stream);

/*
 * pa_plan_step -- pages, block tables, slots and positions of a step's new
 * tokens, from the lengths alone, on the GPU (one launch).  The metadata that
 * vLLM #6052 builds on the host for its single varlen launch: block tables,
 * cumulative query lengths with repeated entries for padding, and the slots of
 * the cache write.
 *
 * Request b has cache_seqlens[b] tokens in the cache and brings q_lens[b] >= 0
 * new ones (0: it rests, or is a padding entry).  It needs
 *   ceil((cached + new) / page_size) - ceil(cached / page_size)
 * pages of the pool.  Requests are admitted in order while the free pages and
 * token_capacity suffice; the first one that does not fit and every later one
 * get no rows in this step and keep their lengths (PA_DEVERR_CAPACITY with the
 * first one's index and its needed pages).  A request with a negative length,
 * or more tokens than its table row holds, is left out the same way, its length
 * kept as it is (PA_DEVERR_LENGTH), and does not stop those behind it.
 *
 *   cache_seqlens, q_lens  int32 [B].
 *   block_table   int32 [B, >= max_pages] rows of stride bt_stride; the new
 *                 pages are written behind each request's own, nothing else.
 *   free_pages    int32 [num_pages], of which the first *free_count are the
 *                 free pages, a stack: the step's k-th new page (by request,
 *                 then by position) is free_pages[*free_count - 1 - k].  Not
 *                 written.
 *   cu_seqlens_q  int32 [B+1] out: first packed row of each request.
 *   seqlens_k     int32 [B] out: tokens in the cache after the step's append
 *                 (pa_fwd_varlen_unified's argument); may be cache_seqlens.
 *   slot_mapping  int64 [token_capacity] out: page * page_size + place in it
 *                 of each packed row's token; -1 behind the last row, and for a
 *                 token whose table entry lies outside the pool
 *                 (PA_DEVERR_PAGE_OOB with the request and the entry's column).
 *   positions     int32 [token_capacity] out: the token's position in its
 *                 sequence; 0 behind the last row.
 *   free_count_out  int32 [1] out: free pages left; may be free_count.
 * At most 4096 requests, 2^31 - 4096 tokens a table row, and 2^31 - 2^16 pages
 * and rows; more are refused.  A *free_count outside
 * [0, num_pages] is reported (PA_DEVERR_CAPACITY, index -1) and clamped.
 * err_word[1] is the request, [2] the offending value.  Pages belong to one
 * request each; two calls on the same pool must be ordered by the caller.
 */
PA_API int pa_plan_step(const int32_t* cache_seqlens, const int32_t* q_lens, int B,
                        int32_t* block_table, int64_t bt_stride, int max_pages, int page_size,
                        const int32_t* free_pages, const int32_t* free_count, int64_t num_pages,
                        int32_t* cu_seqlens_q, int32_t* seqlens_k, int64_t* slot_mapping,
                        int32_t* positions, int token_capacity, int32_t* free_count_out,
                        int32_t* err_word, pa_stream_t stream);

/*
 * pa_release_pages -- gives pages back to pa_plan_step's pool (one launch):
 * those of finished requests (keep_lens[b] == 0) and of requests that take
 * tokens back, such as rejected speculative ones.
 *
 * Request b keeps min(keep_lens[b], cache_seqlens[b]) tokens; its table entries
 * from ceil(keep / page_size) up to ceil(cached / page_size) are pushed onto
 * free_pages behind the first *free_count, by request, then by position.
 *   seqlens_out     int32 [B] out: tokens kept; may be cache_seqlens.
 *   free_count_out  int32 [1] out; may be free_count.
 * block_table is not written: entries behind a sequence's pages mean nothing.
 * A negative or too long cached length and a negative keep_lens[b] leave the
 * request as it is (PA_DEVERR_LENGTH).  An entry outside the pool is not given
 * back (PA_DEVERR_PAGE_OOB).  Where the list would hold more than num_pages
 * pages, the first request that does not fit and every later one stay as they
 * are (PA_DEVERR_CAPACITY).  Limits as pa_plan_step.
 */
PA_API int pa_release_pages(const int32_t* cache_seqlens, const int32_t* keep_lens, int B,
                            const int32_t* block_table, int64_t bt_stride, int max_pages,
                            int page_size, int32_t* free_pages, const int32_t* free_count,
                            int64_t num_pages, int32_t* seqlens_out, int32_t* free_count_out,
                            int32_t* err_word, pa_stream_t stream);

/*
 * pa_rotary_append_varlen -- rotary embedding of a ragged batch's new tokens
 * by positions with one or several axes, and the write of their k and v into
 * the slots of a paged cache, in 16 bits or as e4m3 (one launch).  The step
 * before pa_fwd_varlen_unified and pa_fwd_varlen_e4m3, whose chunks must
 * already be in the cache.
 *
 * Token t's pair p (paired as in pa_fwd_kvcache_rotary) turns by row
 * positions[pair_axis[p]][t] of the tables: c = rotary_cos[row][p].  Images and
 * video have a position on each axis (time, height, width); text has one.
 *
 *   q, k, v       [T, H, D] views, element strides *_st, *_sh (multiples of
 *                 8), D contiguous, 16-byte aligned; slices of one projection
 *                 will do.  q may be NULL (k and v only).
 *   q_out         the rotated q, with its own strides; may be q.
 *   k_cache, v_cache  paged, of `dtype` or PA_E4M3 (cache_dtype); for PA_E4M3
 *                 strides are multiples of 16 elements.  Stored is
 *                 e4m3(x / s), s the kv head's scale: the fp32 quotient, to
 *                 the nearest e4m3 value, saturating at +-448; NaN stays NaN.
 *   k_scale, v_scale  fp32 [Hkv] on the device (PA_E4M3 only); NULL: 1.
 *   slot_mapping  int64 [T]: page * page_size + place; negative: the token's k
 *                 and v are not stored.  A slot outside the pool is skipped
 *                 and reported (PA_DEVERR_PAGE_OOB, token, page).  Two tokens
 *                 with one slot race.
 *   positions     int32 [n_axes, T], rows of stride pos_stride; n_axes 1 to 4.
 *                 A token with a position outside [0, rotary_len) on any axis
 *                 is not rotated (PA_DEVERR_LENGTH, token, position).
 *   pair_axis     HOST array of rotary_dim / 2 axis numbers, read before the
 *                 call returns; NULL: axis 0 for every pair.
 *   rotary_cos, rotary_sin  [rotary_len, rotary_dim / 2] of `dtype` or PA_F32
 *                 (rotary_dtype); rotary_cos NULL: nothing is rotated, q is
 *                 copied.
 * The rotation is computed in fp32 and rounded once to what is stored.
 */
PA_API int pa_rotary_append_varlen(
    const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
    const void* v, int64_t v_st, int64_t v_sh, void* q_out, int64_t qo_st, int64_t qo_sh,
    pa_tensor4 k_cache, pa_tensor4 v_cache, const float* k_scale, const float* v_scale,
    const int64_t* slot_mapping, int page_size, int64_t num_pages, const int32_t* positions,
    int64_t pos_stride, int n_axes, const uint8_t* pair_axis, const void* rotary_cos,
    const void* rotary_sin, int rotary_len, int rotary_dim, int rotary_interleaved,
    int rotary_dtype, int T, int Hq, int Hkv, int D, int dtype, int cache_dtype,
    int32_t* err_word, pa_stream_t stream);

/*
 * pa_fwd_varlen_e4m3 -- pa_fwd_varlen_unified over an e4m3 cache: attention of
 * a ragged batch of prompt chunks and single tokens over paged 8-bit K and V,
 * with half the cache's bytes to read.
 *
 * Arguments as pa_fwd_varlen_unified, with k_cache and v_cache of e4m3 values
 * (strides multiples of 16 elements) and
 *   k_scale, v_scale  fp32 [Hkv] on the device: what a stored value of the kv
 *                     head is multiplied by; NULL: 1.
 *   workspace         pa_fwd_varlen_e4m3_workspace_size bytes, 256-byte
 *                     aligned, always; its contents on entry do not matter.
 *                     A size for some B and max_seqlen_q holds for smaller ones.
 *                     Calls that may overlap on the GPU need one each.
 * q and out are fp16 or bf16; both products are computed in fp16 with fp32
 * accumulation (e4m3 is exact in fp16; a bf16 row of q is scaled by a power of
 * two first), so the result is that of the dequantised cache up to the rounding
 * of the probabilities to fp16.  Keys that a row does not see have no effect on
 * it, whatever they hold.  Rows behind cu_seqlens_q[B] are not written.  At most
 * 4096 entries and 2^31 - 4096 tokens a table row, and at most 2^31 - 1 tiles of
 * 256 rows per kv head by 128 keys; more return PA_ERR_UNSUPPORTED.
 */
PA_API int pa_fwd_varlen_e4m3(const void* q, int64_t q_st, int64_t q_sh, pa_tensor4 k_cache,
                              pa_tensor4 v_cache, const float* k_scale, const float* v_scale,
                              const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                              const int32_t* block_table, int64_t bt_stride, int max_pages,
                              int page_size, int B, int total_q, int max_seqlen_q,
                              int max_seqlen_k, int Hq, int Hkv, int D, int64_t num_pages,
                              float scale, int causal, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, int32_t* err_word, int dtype,
                              pa_stream_t stream);

PA_API size_t pa_fwd_varlen_e4m3_workspace_size(int B, int total_q, int max_seqlen_q, int Hq,
                                                int Hkv, int D, int max_seqlen_k);

/*
 * pa_beam_select -- the best continuations of each request over its beams and
 * the vocabulary (one launch): a beam search's step from logits to scores,
 * parents and tokens.  pa_beam_reorder then moves the beams' pages.
 *
 * Beam k of request b has the score s = scores[b, k] and the logits x:
 *   score(k, v) = s + (x[v] - ln sum_w exp(x[w])), in 64 bits,
 * and the N largest are returned in descending order, the lowest k * V + v first
 * among equal ones.
 *
 *   logits       [B, K, V] of `dtype` (PA_F16, PA_BF16 or PA_F32), element
 *                strides stride_b, stride_k; any alignment of the rows.  -inf:
 *                a token that may not be chosen.
 *   scores       fp32 [B, K]; a beam whose score is not finite is dead: it has
 *                no candidates and its logits are not read.
 *   finished     uint8 [B, K] or NULL; not 0: the beam's only candidate is
 *                end_token with its score as it is, and its logits are not read.
 *   end_token    in [0, V), or negative for none (finished must be NULL then).
 *   scores_out   fp32 [B, N]; parents, tokens int32 [B, N]: k and v.  Where there
 *                are fewer candidates: -inf, -1 and -1 (pa_beam_reorder drops
 *                such a beam, and the next call takes it for dead).
 *   finished_out uint8 [B, N] or NULL: the parent was finished, or the token is
 *                end_token.  None of the outputs may be an input.
 * A beam whose logits hold a NaN or +inf has no candidates and is reported
 * (PA_DEVERR_VALUE, b * K + k); one with nothing but -inf has none.  Any finite
 * logits will do (a row of the type's lowest value is one of equal logits); a token
 * whose score is below fp32's range is no candidate.  ln sum exp is good to 2^-17,
 * so the order of two beams' candidates is sure where their scores are 2^-16 apart;
 * within a beam, and between beams of equal logits, it is that of 64 bits.
 * K <= 32, N <= 64, V <= 2^24, B <= 2^20.  N above 32 is right but may be slow: where
 * a CTA has a small part of each row, thousands of elements are compared one by one
 * (one request of 32 beams of 32000 bf16 logits: 36 us with N = 32, 5 ms with 33).
 */
PA_API int pa_beam_select(const void* logits, int64_t stride_b, int64_t stride_k,
                          const float* scores, const uint8_t* finished, int end_token, int B,
                          int K, int V, int N, float* scores_out, int32_t* parents,
                          int32_t* tokens, uint8_t* finished_out, int32_t* err_word, int dtype,
                          pa_stream_t stream);

/*
 * pa_beam_reorder -- block tables, lengths and page pool after the beams of each
 * request have been replaced by their continuations (one launch).  Beams share
 * the pages of their common past: what is moved is table entries, and only a
 * page that would be written by several beams is copied (pa_copy_pages).
 *
 * Row b * K + i of the tables becomes child i of request b: the tokens and
 * pages of row b * K + parents[b, i].  Beams of a request share pages only at
 * the same column of their tables.  No page is in the tables of two requests, a
 * common prompt's neither: nothing counts references, so the request that ends
 * first would give back what the other still reads and writes.
 *   - A page of a column that no child holds there goes back to the pool: pushed
 *     onto free_pages behind the first *free_count, by request, column, beam.
 *   - A child's last page that is partly filled will be written to.  Where an
 *     earlier child holds it too, or another child holds it whole, the child
 *     gets a fresh page and an entry in `copies`.  Fresh pages come from the top
 *     of the pool as it stands after the pushes, by request, column, child.
 * The step after a prompt has parents all 0: one row becomes K.  A request that
 * ends has parents all -1: its pages go back, each once (pa_release_pages would
 * push the pages that rows share once a row).
 *
 *   parents       int32 [B, K]: a beam of the request, or -1: the child has no
 *                 tokens and holds no page.
 *   seqlens       int32 [B * K]: tokens in the cache of each row, each beam its own.
 *   block_table   int32 [B * K, >= max_pages], rows of stride bt_stride.
 *   block_table_out  with its own stride bto_stride; may be block_table (with the
 *                 same stride).  A child's entries up to its last page are written.
 *   seqlens_out   int32 [B * K]; may be seqlens.
 *   free_pages    int32 [num_pages], free_count, free_count_out as in
 *                 pa_plan_step and pa_release_pages.
 *   copies        int32 [B * K, 3]: for each child the page to be copied, the
 *                 fresh page and the number of tokens; -1, -1, 0: none.
 * Requests are taken in order while the pool holds their fresh pages; the first
 * that does not fit and every later one stay as they are, without copies
 * (PA_DEVERR_CAPACITY, the request and its fresh pages).  An entry of the pool that is
 * no page of it counts as the pool's end (PA_DEVERR_PAGE_OOB, the first row that wants
 * a fresh page, the column, where that stops a request).  A request with a parent
 * outside [-1, K) (PA_DEVERR_VALUE, the row, the parent), a length outside its
 * table row (PA_DEVERR_LENGTH, the row, the length) or an entry outside the pool
 * (PA_DEVERR_PAGE_OOB, the row, the column) stays as it is, too, and does not
 * stop those behind it.  K <= 32 and B * K <= 4096; other limits as pa_plan_step.
 */
PA_API int pa_beam_reorder(const int32_t* parents, const int32_t* seqlens, int B, int K,
                           const int32_t* block_table, int64_t bt_stride, int max_pages,
                           int page_size, int32_t* free_pages, const int32_t* free_count,
                           int64_t num_pages, int32_t* block_table_out, int64_t bto_stride,
                           int32_t* seqlens_out, int32_t* copies, int32_t* free_count_out,
                           int32_t* err_word, pa_stream_t stream);

/*
 * pa_copy_pages -- copies the first tokens of pages to other pages, in the
 * caches of all layers (one launch per 256 caches): what pa_beam_reorder asks for.
 *
 *   copies     int32 [n, 3] on the device: source page, target page, tokens; an
 *              entry with a negative source or target, or no tokens, is skipped.
 *              A page outside the pool, or more tokens than a page has, is
 *              skipped and reported (PA_DEVERR_PAGE_OOB, the entry, the page;
 *              PA_DEVERR_LENGTH, the entry, the tokens).  No target may be
 *              another entry's source or target.
 *   caches     HOST array of n_caches device pointers, read before the call
 *              returns: [num_pages, page_size, H, D] each, k and v alike, with the
 *              same BYTE strides stride_b, stride_t, stride_h (multiples of 16) and
 *              head_bytes = D * element size (a multiple of 16) contiguous bytes.
 */
PA_API int pa_copy_pages(const int32_t* copies, int n, void* const* caches, int n_caches,
                         int64_t stride_b, int64_t stride_t, int64_t stride_h, int head_bytes,
                         int H, int page_size, int64_t num_pages, int32_t* err_word,
                         pa_stream_t stream);

/*
 * pa_fwd_cross -- attention of a ragged batch's rows to the keys of their entry,
 * of another length (cross attention to an encoder's states): no mask by
 * position, no cache and no pages.  All rows of an entry read one copy of its
 * keys and values: the beams of a request, and several tokens of each, are
 * rows of one entry.
 *
 *   q             [total_q, Hq, D], element strides q_st, q_sh (multiples of 8),
 *                 packed by cu_seqlens_q int32 [B+1], as in pa_fwd_varlen_unified.
 *   k, v          [total_k, Hkv, D], element strides *_st, *_sh (multiples of 8),
 *                 16-byte aligned: slices of one projection will do.
 *   cu_seqlens_k  int32 [B+1]: entry b's keys begin at row cu_seqlens_k[b] and end
 *                 at cu_seqlens_k[b+1], or, with seqlens_k, after its first
 *                 seqlens_k[b] rows (a padded batch).
 *   seqlens_k     int32 [B] or NULL.
 *   key_mask      uint8 [total_k] or NULL: 0: no row sees the key, whatever k and v
 *                 hold there (NaN and infinities too).
 *   max_seqlen_q, max_seqlen_k  host-known bounds of an entry's rows and keys.
 *   out [total_q, Hq, D] contiguous; lse fp32 [Hq, total_q] or NULL.
 *   workspace     pa_fwd_cross_workspace_size bytes, 256-byte aligned (NULL where
 *                 that is 0); its contents on entry do not matter.  Calls that may
 *                 overlap on the GPU need one each.
 *   scale         positive, and finite times log2(e).
 * Sums of p v are fp32, with p up to 2^40 (bf16) or 2^15 (fp16): bf16 values of v above
 * 2^60 may overflow.  Rows without a key: O = 0, LSE = -inf.  Rows behind
 * cu_seqlens_q[B] are not written.  An entry with rows or keys outside q and k, or more
 * than the bounds, is reported (PA_DEVERR_LENGTH, the entry, the length): its rows that
 * lie in q and within max_seqlen_q have no keys then.  At most 2^30 tiles of 256 rows per
 * kv head by 128 keys, by the bounds; more return PA_ERR_UNSUPPORTED.
 */
PA_API int pa_fwd_cross(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st,
                        int64_t k_sh, const void* v, int64_t v_st, int64_t v_sh,
                        const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                        const int32_t* seqlens_k, const uint8_t* key_mask, int B, int total_q,
                        int total_k, int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int D,
                        float scale, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int32_t* err_word, int dtype, pa_stream_t stream);

PA_API size_t pa_fwd_cross_workspace_size(int total_q, int max_seqlen_q, int Hq, int Hkv, int D);

/* Human-readable text of the last non-OK return on the calling thread. */
PA_API const char* pa_last_error_string(void);

/* Library version, major * 10000 + minor * 100 + patch. */
PA_API int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
