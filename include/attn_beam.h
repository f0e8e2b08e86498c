/*
 * attn_beam.h -- a beam search's step over the sequences of a paged cache.
 *
 *   attn_beam_select    the best continuations of every prompt, over its beams
 *                       and the vocabulary
 *   attn_beam_reorder   states brought into the chosen order; the cache itself
 *                       is reordered by attn_cache_fork, whose copies
 *                       attn_cache_copy_pages makes (of pages in 8 bits one
 *                       call for the codes and one for the scales)
 *
 * Conventions are those of attn_paged.h.  Row g * beams + b of an array is beam
 * b of prompt (group) g.
 */
#ifndef ATTN_BEAM_H
#define ATTN_BEAM_H

#include "attn_slice.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_BEAM_MAX 64              /* beams of a group, and continuations kept */
#define ATTN_BEAM_MAX_STATES 64       /* arrays of one attn_beam_reorder          */

/* Workspace of attn_beam_select on the current device. */
int attn_beam_workspace_bytes(int groups, int beams, int vocab, int keep, size_t *bytes);

/* Of the beams * vocab continuations of each group, the `keep` best by
 *   score[b] + logit[b][v] - ln sum_w exp(logit[b][w])
 * best first, equal ones by their place b * vocab + v.  The logarithm is that of a
 * sum in 32 bits, good to 2^-19 (measured: 2^-21 up to 2^21 tokens, 2^-20 of 2^24
 * that ascend) and the same for rows of a call that are the same; the rest is
 * added and compared in 64 bits.  So continuations of one beam, or of equal ones,
 * are always in order, those of different beams where they are 2^-18 apart.
 *   logits   [groups * beams, vocab] f32 or bf16 (ATTN_DTYPE_*), rows row_stride
 *            elements apart
 *   scores   [groups, beams] f32
 *   done     [groups, beams] bytes, or null: where one is not 0 the beam has
 *            ended; its one continuation is the token `eos` at its own score,
 *            and its logits are not used
 *   eos      the token that ends a beam, or -1 (then done must be null)
 *   slots    [groups * beams] int32, or null
 *   out_scores, out_parents, out_tokens  [groups, keep] f32, int32, int32: the
 *            score, the parent's row g * beams + b, and the token
 *   out_done [groups, keep] bytes, or null: 1 where the parent has ended or the
 *            token is eos
 *   out_src  [groups, keep] int32, or null: slots[parent] (the parent where
 *            slots is null), the `src` of attn_cache_fork
 * A continuation that cannot be (a logit of -inf; a beam whose score, or whose
 * sum, is not finite: a NaN or +inf among its logits, -inf alone; what an ended
 * beam does not offer) has the score -inf and stands behind all others, by its
 * place as well.  groups = 0 does nothing.  No output may lie on an input, the
 * workspace or another output (not looked at).
 * Errors: INVALID_ARG (keep > beams * vocab, eos >= vocab, null arrays, ..);
 * UNSUPPORTED (beams or keep > ATTN_BEAM_MAX, groups * beams >= 2^24, vocab >
 * 2^30, alignment of an array to its elements, of d_ws to 16); CAPACITY (ws_bytes); CUDA. */
int attn_beam_select(const void *logits, int logits_dtype, int64_t row_stride, int groups, int beams,
                     int vocab, const float *scores, const uint8_t *done, int eos, const int32_t *slots,
                     int keep, float *out_scores, int32_t *out_parents, int32_t *out_tokens,
                     uint8_t *out_done, int32_t *out_src, void *d_ws, size_t ws_bytes,
                     attn_stream_t stream);

/* Row i of every state becomes what row parents[i] was before the call, for all
 * i at once, in place.  parents: [groups * beams] int32, each within its own
 * group, as attn_beam_select leaves them with keep = beams.
 *   h_states, h_row_bytes, h_row_strides  host arrays of n_states: a state's
 *            address, the bytes of a row (>= 0) and from row to row (>= those)
 * Rows of any size and alignment are served; multiples of 16 bytes are fastest.
 * No two states may share memory (of this only two that begin at one address are
 * seen: INVALID_ARG), nor one with the parents.  A group one of whose parents
 * lies outside it is left as it was (INVALID_ARG on the device).
 * Errors: INVALID_ARG; UNSUPPORTED (beams > ATTN_BEAM_MAX, n_states >
 * ATTN_BEAM_MAX_STATES, groups * beams >= 2^24); CUDA. */
int attn_beam_reorder(void *const *h_states, const int64_t *h_row_bytes, const int64_t *h_row_strides,
                      int n_states, const int32_t *parents, int groups, int beams, attn_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* ATTN_BEAM_H */
