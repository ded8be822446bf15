/*
 * libroutedmoe, 4-bit K/V cache: what a speculative-decode step does next to the routed-MoE
 * layer.  A paged cache of keys and values in the experts' own 4-bit format, the attention
 * that reads it, and the calls that allocate, share, copy, compact and free its pages.
 *
 * One step of a batch of sequences, everything on one stream and without a host wait:
 *     moe_kv4_reserve   pages for the step's new tokens (shared pages it will write are copied)
 *     per layer:  moe_kv4_append   the step's K and V rows into the pages
 *                 moe_kv4_attend   the step's query rows over each sequence's tokens
 *                 ... moe_layer, moe_route_grouped + moe_plan + moe_forward, ...
 *     moe_kv4_compact   the accepted tokens moved together, the rejected ones' pages freed
 * and, between steps, moe_kv4_fork (sequences that share another's pages) and moe_kv4_trim
 * (cut or free sequences).
 *
 * Values.  A block of 16 consecutive channels x of one token and head is held as E2M1 codes
 * with one E4M3 scale, both rounded to nearest even:
 *     s = E4M3(min(448, max|x| / (6 ts))),   code = E2M1(x / (s ts)),   value = code * s * ts
 * with ts the cache's FP32 tensor scale of K or of V (code 0 where s is 0).  Infinities are
 * held as +-6 * 448 * ts; a NaN is held as 0; both set MOE_KV4_NONFINITE.
 *
 * Page format.  pool is [layers][pages][page bytes]; a page holds page_size tokens of one
 * layer as [kv_heads][page_size / 16] tiles of 18 * head_dim bytes, each 16 tokens of one head:
 *     K codes   [head_dim / 32][16 tokens][16 bytes]  piece j: channels 32j .. 32j+31
 *     V codes   [16 tokens][head_dim / 2 bytes]
 *     K scales  [16 tokens][head_dim / 16]
 *     V scales  [16 tokens][head_dim / 16]
 * (two codes to a byte, the even channel in the low nibble).  Token p of a sequence lies in the
 * page table[seq][p / page_size], slot p % page_size.
 *
 * Steps.  The rows of a step (queries, keys, values, kept flags) are those of sequence 0, then
 * of sequence 1, and so on: sequence s has the rows cu_rows[s] .. cu_rows[s+1] - 1 (cu_rows on
 * the device, [seqs + 1], cu_rows[0] = 0, non-decreasing), which are its LAST tokens: row r of
 * n lies at position lens[s] - n + r.  A sequence without rows takes no part.
 *
 * Conventions are those of moe.h: device pointers owned by the caller, asynchronous calls that
 * can be captured in a CUDA graph, host-detected errors returned before anything is enqueued.
 * Calls on one cache must be ordered on one stream.  Device-detected conditions are OR-ed into
 * the status word of the cache's workspace (moe_kv4_read_status); no condition makes a call
 * read or write outside the caller's arrays.
 */
#ifndef ROUTED_MOE_KV4_H
#define ROUTED_MOE_KV4_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Status bits of a cache's workspace. */
#define MOE_KV4_NO_PAGE 0x1u   /* moe_kv4_reserve ran out of free pages or table entries: this
                                  sequence and (for pages) those after it that needed some are
                                  refused: they keep their length, pages and tokens, and the
                                  step's later calls leave them out (moe_kv4_reserve) */
#define MOE_KV4_BAD_PAGE 0x2u  /* a token in use lies on a page number outside [0, pages), or
                                  before its sequence's start: it was skipped */
#define MOE_KV4_NONFINITE 0x4u /* moe_kv4_append met an infinity or a NaN */
#define MOE_KV4_BAD_SEQ 0x8u   /* a sequence number outside [0, seqs) or forked onto itself: skipped */

#define MOE_KV4_TIMEOUT 0x10u  /* a bounded wait in the attention kernel gave up: its results are not valid */

typedef enum moe_kv4_dtype { MOE_KV4_BF16 = 0, MOE_KV4_FP16 = 1 } moe_kv4_dtype;

/* One cache.  head_dim 64, 128 or 256; page_size a multiple of 16 up to 1024; kv_heads 1 to
 * 1024; seqs and pages up to 65535 and 2^30; pool and workspace 256-byte aligned.
 *   lens  [seqs] int32             tokens of each sequence (0: empty)
 *   table [seqs][max_pages] int32  page numbers of its tokens, -1 past them
 *   refs  [pages] int32            table entries that point at a page; 0: the page is free
 * A caller that keeps a page for itself sets its refs entry to 1 or more. */
typedef struct moe_kv4_cache {
  void* pool;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  void* workspace;
  size_t workspace_bytes;
  int32_t layers, pages, kv_heads, head_dim, page_size, seqs, max_pages;
  float k_scale, v_scale; /* tensor scales, above 0, at most 2^119 */
} moe_kv4_cache;

/* Bytes of one page of one layer, and of the workspace of a cache (0 if the sizes are
 * unsupported): 43 MB for partial results of the attention, whatever the sizes, and 28 a sequence.  Host functions: need no GPU and no pointer of the cache. */
MOE_API size_t moe_kv4_page_bytes(const moe_kv4_cache* cache);
MOE_API size_t moe_kv4_workspace_bytes(const moe_kv4_cache* cache);

/* MOE_OK, MOE_ERR_INVALID_ARG or MOE_ERR_UNSUPPORTED for the sizes of a cache (host only). */
MOE_API int moe_kv4_check(const moe_kv4_cache* cache);

/* Zero the status word, the counters and the refusals of a fresh workspace.  Once after allocation. */
MOE_API int moe_kv4_workspace_init(const moe_kv4_cache* cache, moe_stream_t stream);

/* Quantise the step's K and V rows into `layer`.
 *   k, v  [rows][kv_heads][head_dim] of `dtype`, channels consecutive; row and head strides in
 *         elements, multiples of 8; 16-byte aligned
 *   rows  rows in all (cu_rows[seqs]; entries of cu_rows beyond it are cut to it)
 * The pages must have been reserved, and be the sequence's own. */
MOE_API int moe_kv4_append(const moe_kv4_cache* cache, int layer, const void* k, int64_t k_row_stride,
                           int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride,
                           int dtype, const int32_t* cu_rows, int rows, moe_stream_t stream);

/* The values held for the step's rows (the last cu_rows[s+1] - cu_rows[s] tokens of every
 * sequence) of `layer`: k, v [rows][kv_heads][head_dim] of `dtype`, contiguous, 16-byte aligned
 * (either may be NULL).  Rows that lie before their sequence's start are zeroed, as are those of a
 * refused sequence. */
MOE_API int moe_kv4_read(const moe_kv4_cache* cache, int layer, void* k, void* v, int dtype, const int32_t* cu_rows,
                         int rows, moe_stream_t stream);

/* Attention of the step's query rows over their sequences' tokens in `layer`:
 *     out[r][h] = sum_t p_t v_t,   p = softmax over the tokens t that row r sees of scale q.k_t
 *     lse[r][h] = log sum_t exp(scale q.k_t)
 * with k_t, v_t of the head h / (q_heads / kv_heads).  The row at position x sees the tokens
 * t <= x, with window > 0 only t > x - window.  With `tree` the row sees every token before the
 * step, and token j of the step where bit j of tree[row] is set (a step has at most 64 tokens
 * then; window must be 0).  A row that sees nothing, or whose sequence
 * was refused, gets out 0 and lse -infinity.
 *   q        [rows][q_heads][head_dim] of `dtype`; strides in elements, multiples of 8
 *   max_rows the largest number of rows of a sequence, as far as the host knows: it chooses the
 *            kernel's tile, for the whole call; more rows are computed all the same.  A prompt's
 *            chunk among single rows is faster in a call of its own, with cu_rows that leave the
 *            others out
 *   scale    finite, and times k_scale too
 *   tree     [rows] uint64 or NULL
 *   out      [rows][q_heads][head_dim] of `dtype`, contiguous, 16-byte aligned
 *   lse      [rows][q_heads] float or NULL
 * At most 2^30 tokens a sequence are looked at.  Rows of no sequence are left as they are.  Scores,
 * softmax statistics and sums are FP32; p is rounded to FP16: 11 bits, fewer where it is
 * below 2^-21 of its row's largest, none below 2^-32.
 * Two launches: the attention, and the joining of what it cut over several SMs; the result does
 * not depend on timing. */
MOE_API int moe_kv4_attend(const moe_kv4_cache* cache, int layer, const void* q, int64_t q_row_stride,
                           int64_t q_head_stride, int q_heads, int dtype, const int32_t* cu_rows, int rows,
                           int max_rows, float scale, int window, const uint64_t* tree, void* out, float* lse,
                           moe_stream_t stream);

/* Room for new_tokens[s] >= 0 more tokens of every sequence (device, [seqs]; negative counts as
 * 0): lens grows by it, and free pages, lowest numbers first in the order of the sequences, are
 * added to the tables.  Where a sequence's last page is partly filled and shared (refs above 1
 * before the call), it is first replaced by a free page holding a copy of it on every layer.
 * A sequence that gets no room (MOE_KV4_NO_PAGE) is refused: its lens stays as it was, and until a
 * later reservation for it succeeds, moe_kv4_trim cuts it or moe_kv4_fork replaces it, the calls of
 * a step treat its rows as rows without a place: append and compact skip them (no token or page of
 * it, or of a sequence it shares pages with, changes), read gives zeros, and attend out 0 and lse
 * -infinity.  So a step can go on without asking for the status first. */
MOE_API int moe_kv4_reserve(const moe_kv4_cache* cache, const int32_t* new_tokens, moe_stream_t stream);

/* Sequence dst[i] becomes a copy of sequence src[i], sharing its pages, for i < n (device
 * arrays).  What dst[i] held is freed first.  The dst must differ from one another and from
 * every src. */
MOE_API int moe_kv4_fork(const moe_kv4_cache* cache, const int32_t* src, const int32_t* dst, int n,
                         moe_stream_t stream);

/* Cut every sequence to at most to_tokens[s] tokens (device, [seqs]; negative counts as 0, which
 * frees the sequence): the pages past its end leave its table. */
MOE_API int moe_kv4_trim(const moe_kv4_cache* cache, const int32_t* to_tokens, moe_stream_t stream);

/* Keep the step's rows with keep[r] != 0 ([rows] uint8): on every layer their K and V move
 * together, in order, to the places from the step's first token on; every sequence is cut to
 * what it keeps.  At most 64 rows a sequence (max_rows, the host's bound; rows past it are
 * dropped).  The step's pages must be the sequence's own. */
MOE_API int moe_kv4_compact(const moe_kv4_cache* cache, const uint8_t* keep, const int32_t* cu_rows, int rows,
                            int max_rows, moe_stream_t stream);

/* Copy the status word to *status_bits (blocking on `stream`), clear it when `clear` is
 * non-zero.  MOE_OK if no bit is set, MOE_ERR_DEVICE if any is. */
MOE_API int moe_kv4_read_status(const moe_kv4_cache* cache, int clear, uint32_t* status_bits, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ROUTED_MOE_KV4_H */
