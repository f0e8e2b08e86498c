/*
 * attn_paged.h -- attention over a paged key/value cache, and the cache's pages.
 *
 *   attn_paged_fwd      a batch's newest tokens against their cached keys, with
 *                       a sliding window and first tokens that stay visible
 *   attn_prefix_fwd     the same for groups of sequences that share a prefix,
 *                       read once for the whole group
 *   attn_slices_from_windows  the windowed mask as a slice list, for attn_fwd
 *                       and attn_bwd over packed sequences
 *   attn_cache_*        pages of the cache: grow, write, fork, free, trim,
 *                       compact, copy
 *
 * Conventions are those of attn_slice.h: the caller owns every buffer, calls
 * are enqueued on `stream` of the current device and return ATTN_OK or an
 * ATTN_ERR_* code; what is wrong with the arguments is found on the host
 * before anything is launched, what is wrong with the contents of device
 * arrays (lengths, page indices, lists) is found by the kernels, which then
 * read and write nothing out of range and leave ATTN_ERR_INVALID_ARG or
 * ATTN_ERR_CAPACITY for attn_last_device_error().  A call allocates nothing
 * and keeps nothing from one call to the next; calls may be captured into
 * CUDA graphs (make the first call on a device before a capture).  Calls that
 * may run at the same time need workspaces of their own.
 *
 * The cache
 *   Keys and values live in pages of page_size tokens, [n_pages, page_size,
 *   hk, d] bf16.  Row `slot` of the page table lists the pages of one
 *   sequence: token j is row j % page_size of page table[slot][j / page_size].
 *   Entries behind the last page, and entries of pages given back by
 *   attn_cache_trim, are -1.  seq_lens[slot] counts the tokens.  refs[p]
 *   counts the table rows that hold page p; a page is free when it is 0.
 *   A page that is not full belongs to one sequence only.
 */
#ifndef ATTN_PAGED_H
#define ATTN_PAGED_H

#include "attn_slice.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_PAGED_MAX_SEQS 4096     /* sequences (or groups) of one call      */
#define ATTN_PAGED_MAX_LEN (1 << 30) /* max_pages * page_size                  */
#define ATTN_CACHE_MAX_POOLS 256     /* page arrays of one attn_cache_copy_pages */

/* Keys and values in pages.  Strides are in elements, multiples of 8, alike
 * for keys and values; d is contiguous; both bases 16-byte aligned.  Pages of
 * a power of two of at least 16 tokens. */
typedef struct {
  const void *k, *v;
  int32_t n_pages, page_size, hk, d;
  int64_t page_stride, token_stride, head_stride;
} attn_pages_t;

/* The sequences of a call: sequence b is row seqs[b] of the table and of
 * seq_lens (row b where seqs is null).  Device pointers, int32. */
typedef struct {
  const int32_t *table;    /* [n_slots, max_pages], rows table_stride apart    */
  const int32_t *seq_lens; /* [n_slots]                                        */
  const int32_t *seqs;     /* [n_seqs] or null                                 */
  int64_t table_stride;
  int32_t n_slots, max_pages, n_seqs, reserved;
} attn_seqs_t;

/* Device workspace of attn_paged_fwd and attn_prefix_fwd on the current
 * device (n_tokens, hq, d: of the queries; prefix: 1 for attn_prefix_fwd). */
int attn_paged_workspace_bytes(int n_tokens, int hq, int d, int prefix, size_t *bytes);

/* Attention of each sequence's newest tokens over its cached keys.
 *   q         [n_tokens, hq, d] bf16, 16-byte aligned; sequence b owns tokens
 *             q_ptr[b] .. q_ptr[b+1]
 *   q_ptr     [n_seqs+1] int32, not decreasing, or null: one token each (then
 *             n_tokens == n_seqs).  Rows outside every sequence's range are
 *             not read, and their outputs are left as they were.
 *   max_q     about the largest number of tokens of one sequence; only picks
 *             the kernel, any value >= 1 gives the same result up to rounding
 * With L = seq_lens[slot] and n = q_ptr[b+1] - q_ptr[b], token t of sequence b
 * stands at position i = L - n + t (its own key is cached already) and sees the
 * keys j <= i with j > i - window or j < sinks; window = 0: every j <= i.
 *   out       [n_tokens, hq, d] bf16 or f32: softmax(scale q k^T) v over them
 *   lse       [hq, n_tokens] f32: ln sum exp(scale q.k)
 * A token that sees nothing (L = 0, or i < 0) gets out = 0, lse = -inf.
 * Cached rows at and behind L are never used, whatever they hold.
 * Errors: INVALID_ARG; UNSUPPORTED (d not 64 or 128, page size, strides,
 * alignment, n_seqs > ATTN_PAGED_MAX_SEQS, max_pages * page_size >
 * ATTN_PAGED_MAX_LEN); CAPACITY (ws_bytes); CUDA.  On the device INVALID_ARG:
 * a slot, length, q_ptr entry or needed page index out of range.  A sequence
 * with a bad slot, length or q_ptr is taken as one of length 0 or of no
 * tokens; one with a bad page gets outputs of no meaning; others are served. */
int attn_paged_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                   const attn_pages_t *pages, const attn_seqs_t *seqs, float scale, int window,
                   int sinks, void *out, int out_dtype, float *lse, void *d_ws, size_t ws_bytes,
                   attn_stream_t stream);

/* Attention of sequences whose groups share a prefix.  The sequences
 * group_ptr[g] .. group_ptr[g+1] of `seqs` form group g; `prefix` holds one
 * row per group (prefix->n_seqs groups): the prefix's pages and length, of
 * the same page arrays.  A token sees its group's whole prefix, then its own
 * sequence's keys j <= i as in attn_paged_fwd (seq_lens counts the tokens
 * behind the prefix).  A sequence before the first group or behind the last
 * has no prefix.  Each prefix is read once for its whole group.  Other
 * arguments, outputs and errors as in attn_paged_fwd; with a group_ptr that
 * decreases or leaves the batch (INVALID_ARG on the device) the outputs of the
 * groups' tokens mean nothing. */
int attn_prefix_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                    const attn_pages_t *pages, const attn_seqs_t *prefix, const int32_t *group_ptr,
                    const attn_seqs_t *seqs, float scale, void *out, int out_dtype, float *lse,
                    void *d_ws, size_t ws_bytes, attn_stream_t stream);

/* The windowed causal mask of packed sequences as a slice list (host only):
 * sequence after sequence of h_lengths[i] >= 0 tokens, each token seeing its
 * sequence's keys j <= i with j > i - window or j < sinks (window 0: all).
 * At most three disjoint slices a sequence: its first window + sinks rows
 * causal; behind them the sinks full and the window bi-causal.
 *   h_out  room for `capacity` slices (may be null with capacity 0); *n_out
 *          receives the count
 * Errors: INVALID_ARG (negative length, window or sinks; a total of 2^31 or
 * more), CAPACITY. */
int attn_slices_from_windows(const int32_t *h_lengths, int n, int window, int sinks,
                             attn_slice_t *h_out, int capacity, int *n_out);

#ifdef __cplusplus
}
#endif
#endif /* ATTN_PAGED_H */
