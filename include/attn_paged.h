/*
 * attn_paged.h -- attention over a paged key/value cache, and the cache's pages.
 *
 *   attn_paged_fwd      a batch's newest tokens against their cached keys, with
 *                       a sliding window and first tokens that stay visible
 *   attn_prefix_fwd     the same for groups of sequences that share a prefix,
 *                       read once for the whole group
 *   attn_slices_from_windows  the windowed mask as a slice list, for attn_fwd
 *                       and attn_bwd over packed sequences
 *   attn_cache_*        pages of the cache: grow, write, read, fork, free,
 *                       trim, compact, copy
 *   attn_paged8_fwd, attn_prefix8_fwd, attn_cache8_write, attn_cache8_read
 *                       the same over pages that hold 8 bits a value
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
 *   The attn_cache_* calls keep all of this, and lengths change by them alone.
 *   There is no call that takes single tokens back.  A caller that lowers a
 *   length itself (rejected tokens of a verified batch) may do so only where the
 *   row keeps its number of pages and no other row holds its last one.  A page
 *   that the length leaves behind stays counted for good: attn_cache_free passes
 *   it by, attn_cache_extend writes over its entry.
 */
#ifndef ATTN_PAGED_H
#define ATTN_PAGED_H

#include "attn_slice.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_PAGED_MAX_SEQS 4096     /* sequences (or groups) of one call      */
#define ATTN_PAGED_MAX_LEN (1 << 30) /* max_pages * page_size                  */
#define ATTN_PAGED_MAX_KEYS (INT64_C(1) << 36) /* n_seqs * max_pages * page_size */
#define ATTN_CACHE_MAX_SLOTS 16384   /* rows of a cache's page table           */
#define ATTN_CACHE_MAX_PAGES (1 << 30)
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
 *             the kernel, any value >= 1 gives the same result up to rounding.
 *             Far too large a value costs time: many short sequences then run
 *             on tiles made for long ones
 * With L = seq_lens[slot] and n = q_ptr[b+1] - q_ptr[b], token t of sequence b
 * stands at position i = L - n + t (its own key is cached already) and sees the
 * keys j <= i with j > i - window or j < sinks; window = 0: every j <= i.
 *   out       [n_tokens, hq, d] bf16 or f32: softmax(scale q k^T) v over them
 *   lse       [hq, n_tokens] f32: ln sum exp(scale q.k)
 * q and the memory between the pages' first byte and last must not overlap
 * out (INVALID_ARG); lse and d_ws, which are written too, must not overlap
 * anything else (not looked at).
 * A token that sees nothing (L = 0, or i < 0) gets out = 0, lse = -inf.
 * Cached rows at and behind L, and those that no token of the sequence sees,
 * are never used, whatever they hold.  (A key that some tokens of a sequence
 * see and others do not is masked for those by a weight of zero: a value of it
 * that is not finite can reach them, as in attn_fwd; a token that sees nothing
 * gets its zeros all the same.)
 * Errors: INVALID_ARG; UNSUPPORTED (d not 64 or 128, page size, strides,
 * alignment, n_seqs > ATTN_PAGED_MAX_SEQS, max_pages * page_size >
 * ATTN_PAGED_MAX_LEN, times n_seqs > ATTN_PAGED_MAX_KEYS, n_tokens * hq >=
 * 2^31); CAPACITY (ws_bytes); CUDA.  On the device INVALID_ARG:
 * a slot, length, q_ptr entry or needed page index out of range.  A sequence
 * with a bad slot, length or q_ptr is taken as one of length 0 or of no
 * tokens; one with a bad page gets outputs of no meaning; others are served.
 * TIMEOUT where a bounded wait for a kernel's loads or products ran out
 * (attn_set_wait_limit_ns): outputs are then incomplete. */
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
 * arguments, outputs and errors as in attn_paged_fwd; with a group_ptr or
 * q_ptr that decreases or leaves the batch (INVALID_ARG on the device) the
 * outputs mean nothing. */
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

/* ---- pages of the cache --------------------------------------------------
 * The page table and counts of one cache.  One table serves any number of
 * page arrays (the keys and values of every layer).  Device pointers. */
typedef struct {
  int32_t *table;          /* [n_slots, max_pages], rows table_stride apart    */
  int32_t *seq_lens;       /* [n_slots]                                        */
  int32_t *refs;           /* [n_pages]                                        */
  int64_t table_stride;
  int32_t n_slots, max_pages, n_pages, page_size;
} attn_cache_t;

/* An empty cache has every table entry -1, every length and count 0; the
 * caller makes it so once.  The lists below are int32 device arrays of n <=
 * ATTN_PAGED_MAX_SEQS entries, read when the call runs.  A call whose list
 * names a row out of range, or names twice a row that it changes, whose
 * lengths are out of range (INVALID_ARG), or for which free pages, table
 * columns or `cap` do not suffice (CAPACITY) changes nothing, sets copies[0]
 * = 0, and leaves that code for attn_last_device_error().  Page indices out
 * of range in the table are never followed (INVALID_ARG).  Fresh pages are
 * the free ones of the lowest index, handed out in the list's order; pages
 * that a call frees are not handed out by the same call.
 * Host errors: INVALID_ARG; UNSUPPORTED (page size not a power of two of at
 * least 16, the limits above, alignment); CAPACITY (ws_bytes); CUDA. */

/* Adds counts[i] >= 0 tokens to row seqs[i]: pages are taken for them and the
 * length grows; attn_cache_write fills them. */
int attn_cache_extend(const attn_cache_t *cache, const int32_t *seqs, const int32_t *counts, int n,
                      attn_stream_t stream);

/* Empties the listed rows: their pages lose a holder each, their lengths
 * become 0 and their entries -1. */
int attn_cache_free(const attn_cache_t *cache, const int32_t *seqs, int n, attn_stream_t stream);

/* Gives back, of the listed rows (null: every row, n = n_slots), the pages
 * that a token at position seq_len - 1 or later never sees through a window
 * >= 1 and first tokens `sinks`: their entries become -1.  Lengths and
 * positions stay. */
int attn_cache_trim(const attn_cache_t *cache, const int32_t *seqs, int n, int window, int sinks,
                    attn_stream_t stream);

/* Makes row dst[i] hold what row src[i] held before the call, for all i at
 * once (a source may be named several times, and may itself be replaced; no
 * dst twice); what the dst rows held before is freed.  Full pages are shared.
 * A partial last page stays with its source, or with the source's first child
 * of the list where the source is replaced; every other child gets a fresh
 * page, and the pair enters the copy list:
 *   copies [1 + 2 cap] int32: the count, then the pages to copy from, then at
 *          1 + cap those to copy to; entries behind the count are -1.  n
 *          copies at most.
 *   d_ws   attn_cache_workspace_bytes(cache, n) bytes
 * The pages' contents move with attn_cache_copy_pages, which has to run
 * before anything is written to the rows. */
int attn_cache_fork(const attn_cache_t *cache, const int32_t *src, const int32_t *dst, int n,
                    int32_t *copies, int cap, void *d_ws, size_t ws_bytes, attn_stream_t stream);

/* Moves the pages in use to the lowest indices: with u pages in use, those at
 * u and above, in ascending order, go to the free ones below u, in ascending
 * order.  The table, the counts and the copy list (n_pages / 2 copies at
 * most) say so; attn_cache_copy_pages moves the contents.  Table entries
 * behind a row's last page have to be -1 or are left alone. */
int attn_cache_compact(const attn_cache_t *cache, int32_t *copies, int cap, void *d_ws,
                       size_t ws_bytes, attn_stream_t stream);

/* Workspace of attn_cache_fork with lists of n, and of attn_cache_compact. */
int attn_cache_workspace_bytes(const attn_cache_t *cache, int n, size_t *bytes);

/* Copies whole pages inside every listed array: copies as above (it may also
 * be the caller's own).  h_pools: host array of n_pools device pointers, each
 * to n_pages pages of page_bytes, page_stride_bytes apart (multiples of 16,
 * 16-byte aligned).  Pairs with an index out of range are left out
 * (INVALID_ARG on the device).  No page may be copied to twice, nor copied
 * both to and from: its contents would be either's. */
int attn_cache_copy_pages(void *const *h_pools, int n_pools, size_t page_bytes,
                          size_t page_stride_bytes, int n_pages, const int32_t *copies, int cap,
                          attn_stream_t stream);

/* Writes new keys and values to the ends of their sequences: token t of
 * sequence b (q_ptr and seqs as in attn_paged_fwd) goes to position
 * seq_len - n + t.
 *   k_new, v_new  [n_tokens, hk, d] bf16, 16-byte aligned, strides in elements
 *                 and multiples of 8, d contiguous
 * Tokens of no sequence are not read; a token whose slot, position or page is
 * out of range is not written (INVALID_ARG on the device).  Where `seqs` names a
 * row twice, both write its last positions, which then hold either's tokens.
 * k_new and v_new must not lie where the call writes (not looked at).
 * UNSUPPORTED also: pages with a stride of zero, n_tokens > ATTN_PAGED_MAX_LEN. */
int attn_cache_write(const attn_pages_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr,
                     const void *k_new, const void *v_new, int n_tokens, int64_t new_token_stride,
                     int64_t new_head_stride, attn_stream_t stream);

/* Reads cached keys and values back as rows: token t of sequence b (q_ptr and
 * seqs as above, n = q_ptr[b+1] - q_ptr[b]) is position seq_len - n + t, the
 * places that attn_cache_write fills; n = seq_len reads a whole sequence.
 *   k_out, v_out  [n_tokens, hk, d] bf16 or f32 (out_dtype), 16-byte aligned
 * Rows of no sequence are left as they were; so is a row whose slot, position
 * or page is out of range (INVALID_ARG on the device).  The outputs must not lie
 * where the call reads (not looked at).  UNSUPPORTED also: n_tokens >
 * ATTN_PAGED_MAX_LEN, hk > 1024. */
int attn_cache_read(const attn_pages_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr,
                    int n_tokens, void *k_out, void *v_out, int out_dtype, attn_stream_t stream);

/* ---- pages in 8 bits -------------------------------------------------------
 * k and v of `pages` are codes of one byte, strides in elements (bytes) and
 * multiples of 16; every token and key/value head has one scale for its keys
 * and one for its values, [n_pages, page_size, hk] f32, strides in elements,
 * alike for both and not negative.  A value is code * scale.
 * The table operations above serve these pages as they are: attn_cache_copy_pages
 * moves the codes in one call and the scales in another.  A code of e4m3 that is no
 * number (the calls below write none) counts as some value up to 480 or as NaN. */
enum { ATTN_CODES_INT8 = 0, ATTN_CODES_E4M3 = 1 };
typedef struct {
  attn_pages_t pages;
  const float *k_scales, *v_scales;
  int64_t scale_page_stride, scale_token_stride, scale_head_stride;
  int32_t format, reserved;   /* ATTN_CODES_* */
} attn_pages8_t;

/* attn_paged_fwd and attn_prefix_fwd over such pages.  Scores and weights take
 * the scales in 32 bits; codes enter the products as they are, so that nothing
 * is rounded that the codes had not been.  Scales are expected not to be
 * negative, finite and, but for 0, above 1e-24, and may lie as far apart as that.
 * What is formed in 32 bits has to be finite there: a query's products with codes,
 * its largest magnitude times `scale` and a key's scale, and 2^8 times the sum of a
 * sequence's values (which scales up to 1e24 keep to at any length).  Codes and
 * scales behind a sequence's end, and those that no token of the sequence sees, are never used,
 * whatever they hold; a key that some tokens of a sequence see and others do not
 * has to have a value and scale that are finite, as above.  The outputs of a token
 * that sees a scale that is not finite mean nothing.  The workspace is that of the
 * calls above. */
int attn_paged8_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                    const attn_pages8_t *pages, const attn_seqs_t *seqs, float scale, int window,
                    int sinks, void *out, int out_dtype, float *lse, void *d_ws, size_t ws_bytes,
                    attn_stream_t stream);
int attn_prefix8_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                     const attn_pages8_t *pages, const attn_seqs_t *prefix, const int32_t *group_ptr,
                     const attn_seqs_t *seqs, float scale, void *out, int out_dtype, float *lse,
                     void *d_ws, size_t ws_bytes, attn_stream_t stream);

/* attn_cache_write into such pages.  Of a token's head with the largest
 * magnitude a, M = 127 (int8) or 448 (e4m3): its scale is a / M, and x becomes
 * the code next to x M / a, the even one of two as near (a = 0: scale and codes
 * 0).  Where a value is not finite the scale is NaN and the codes are 0: the
 * head's whole row reads as NaN.  Where `seqs` names a row twice, its last
 * positions may hold codes and scales of different tokens.  UNSUPPORTED also: scales with a stride of zero,
 * hk > 1024. */
int attn_cache8_write(const attn_pages8_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr,
                      const void *k_new, const void *v_new, int n_tokens, int64_t new_token_stride,
                      int64_t new_head_stride, attn_stream_t stream);

/* attn_cache_read from such pages: code * scale, rounded once. */
int attn_cache8_read(const attn_pages8_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr,
                     int n_tokens, void *k_out, void *v_out, int out_dtype, attn_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* ATTN_PAGED_H */
