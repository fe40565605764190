/*
 * specdecode.h -- C ABI of libspecverify, the operators of a decode loop that
 * stand next to the verify step (specverify.h) on AMD Instinct MI355X
 * (gfx950): beam selection over beams and vocabulary, the reordering of beam
 * states, and the block tables, slot maps and moves of a paged key/value
 * cache whose lengths the verify step decides.
 *
 * Memory, streams, status codes and workspaces are as in specverify.h: every
 * array is a DEVICE pointer owned by the caller unless noted, nothing is
 * allocated, all work is enqueued on `stream`, kernels only (a call can be
 * captured into a graph).  Data errors found on the device set bits of
 * *error_word, which the caller clears; no data makes a kernel access memory
 * outside the arrays that a call describes.  Arrays of a call may not overlap
 * unless noted.
 */
#ifndef SPECDECODE_H
#define SPECDECODE_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device-side error word. */
#define SV_ERR_SCORE 128    /* a beam score is NaN or +inf: the sequence's outputs are -1       */
#define SV_ERR_PARENT 256   /* a beam parent >= W: that beam's state stays as it is             */
#define SV_ERR_LENGTH 512   /* a length outside what its arrays hold (see each call)            */
#define SV_ERR_PAGES 1024   /* the free list ran out of pages, or would hold more than num_pages */
#define SV_ERR_PAGE 2048    /* a page number outside [0, num_pages) where a page is needed      */

#define SV_MAX_BEAMS 32       /* beams per sequence                            */
#define SV_MAX_CANDIDATES 64  /* candidates beam selection returns per sequence */
#define SV_MAX_POOLS 1024     /* caches moved by one call                      */

/*
 * Beam search's selection.  For sequence b, beam w with cumulative score
 * s_w = scores[b, w], logits z_w and temperature T, the candidates are
 *   c(w, v) = s_w + z_w(v) / T - ln sum_u exp(z_w(u) / T)
 * over beams w < W and tokens v < V with z_w(v) > -inf.  A beam with
 * s_w == -inf, or whose logits are all -inf, has no candidate; a finished
 * beam (finished[b, w] != 0) has one, (w, eos) at c = s_w.  The logits of dead
 * and finished beams have no effect, NaN among them.
 * Out come the M candidates of largest c in descending order, equal ones by
 * lower beam, then larger logit, then lower token; where there are fewer, the
 * rest are (-inf, -1, -1).  Order is decided on c in 64 bits, with the sum of
 * exponentials in fp32 per 16-byte vector and fp64 beyond (error of the
 * logarithm ~1e-8); out_score is c rounded to fp32 (to -inf below its range,
 * as for a token masked by the type's lowest value at T < 1: parent and token
 * tell such a candidate from none).
 *   logits       element (b, w, v) at b * seq_stride + w * beam_stride + v,
 *                strides >= 0 in elements (0 shares rows), dtype SV_F32/SV_BF16
 *   temperature  [B] float, > 0 and finite (else SV_ERR_TEMPERATURE), or NULL: 1
 *   finished     [B, W] int32 or NULL;  eos in [0, V), or -1 when finished is NULL
 *   out_score [B, M] float, out_parent [B, M] int32, out_token [B, M] int32
 *   out_finished [B, M] int32 or NULL: 1 where the parent was finished or the
 *                token is eos, else 0
 * A sequence with a bad temperature or score, or a NaN or +inf logit in a
 * beam in the running (SV_ERR_ROW), gets -inf, -1, -1 and 0 throughout.
 * 1 <= W <= SV_MAX_BEAMS, 1 <= M <= SV_MAX_CANDIDATES, W * V < 2^31.
 * Two kernel launches.  out_score may be scores, and out_finished may be
 * finished, when M == W (the loop's own buffers).
 */
size_t spec_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t dtype, int32_t M);

int32_t spec_beam_select(const void *logits, int32_t B, int32_t W, int32_t V, int32_t dtype, int64_t seq_stride,
                         int64_t beam_stride, const float *scores, const float *temperature,
                         const int32_t *finished, int32_t eos, int32_t M, float *out_score, int32_t *out_parent,
                         int32_t *out_token, int32_t *out_finished, int32_t *error_word, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * Reordering of beam states, in place: in each of n_pools arrays
 *   pool[(b * W + w), g, s, :]   [B * W, G, S, row_bytes]
 * beam j of sequence b takes over the rows of beam parent[b, j] at positions
 * s < length[b] (NULL: S), as they were before the call, for all j at once.
 * parent[b, j] < 0 leaves beam j as it is; >= W does too, with SV_ERR_PARENT.
 * Positions from length[b] on are left as they are; a length outside [0, S]
 * moves nothing of the sequence, with SV_ERR_LENGTH.
 *   pools   HOST array of n_pools <= SV_MAX_POOLS device pointers, of any
 *           alignment (multiples of 16, like row_bytes, move in 16-byte vectors)
 *   parent  [B, W] int32,  W <= SV_MAX_BEAMS
 * One kernel launch per 128 pools.
 */
int32_t spec_beam_reorder(void *const *pools, int32_t n_pools, int32_t B, int32_t W, int32_t G, int32_t S,
                          int64_t row_bytes, const int32_t *parent, const int32_t *length, int32_t *error_word,
                          void *stream);

/*
 * The same in a paged cache: in pools [num_pages, G, page_size, row_bytes],
 * position s of beam w of sequence b lies at offset s % page_size of page
 * block_table[b * W + w, s / page_size] ([B * W, max_blocks] int32).  The
 * positions start[b] (NULL: 0) <= s < length[b] move; a beam and its parent
 * that hold the same page there share it and nothing moves.  Any other page
 * of that range belongs to one beam alone (else the outcome is unspecified).
 * A page outside [0, num_pages) sets SV_ERR_PAGE and its rows stay; start and
 * length outside 0 <= start <= length <= max_blocks * page_size move nothing
 * of the sequence, with SV_ERR_LENGTH (start > length alone is no error).
 * max_length, a host bound on length[b], sizes the launch: positions from it
 * on are not moved (SV_ERR_LENGTH).
 */
int32_t spec_beam_reorder_paged(void *const *pools, int32_t n_pools, int32_t B, int32_t W, int32_t G,
                                int32_t page_size, int64_t row_bytes, int32_t num_pages,
                                const int32_t *block_table, int32_t max_blocks, const int32_t *parent,
                                const int32_t *start, const int32_t *length, int32_t max_length,
                                int32_t *error_word, void *stream);

/*
 * Pages and slots for new tokens.  Sequence b holds s = seq_len[b] tokens in
 * the pages block_table[b, 0 .. ceil(s / page_size) - 1] and is to hold
 * n = (new_len ? new_len[b] : 0) + extra more (K + 1 before a verify step:
 * new_len = the draft lengths, extra = 1).  In order of b each sequence takes
 *   need = ceil((s + n) / page_size) - ceil(s / page_size)
 * pages from the end of the free list, page j of the call being
 * free_list[free_count - 1 - j], and its block table grows by them.  Out come
 *   query_start [B + 1]  sum of n over the sequences before b (the total last)
 *   page_start  [B + 1]  the same of the pages taken
 *   granted     [B]      n, or 0 for a sequence that does not get its pages
 *   slots       [max_tokens] int64: page * page_size + offset of each token,
 *               sequence by sequence; -1 for tokens not granted and behind the last
 *   positions   [max_tokens] int32: s + its place among the new; 0 behind the last
 *   seq_ids     [max_tokens] int32: b; -1 behind the last
 *   free_count_out [1]   what is left (may be free_count)
 * From the first sequence on whose pages the free list does not hold, no
 * sequence that needs pages gets any (SV_ERR_PAGES).  A sequence with
 * s < 0, n < 0 or s + n > max_blocks * page_size has no tokens and one whose
 * tokens reach beyond max_tokens is not granted any (SV_ERR_LENGTH).  A free
 * page outside [0, num_pages), or such an entry where a sequence's last page
 * is to be filled, sets SV_ERR_PAGE, and its tokens' slots are -1.
 * seq_len is left as it is: spec_cache_commit says what was kept, before the
 * next extend (which would take pages for the same positions again).
 *   free_list [num_pages] int32;  free_count [1] in [0, num_pages]
 * B <= 2^20.  One kernel launch, two for more than 4096 tokens or 1024 sequences.
 */
int32_t spec_cache_extend(const int32_t *seq_len, const int32_t *new_len, int32_t extra, int32_t B,
                          int32_t *block_table, int32_t max_blocks, int32_t page_size, const int32_t *free_list,
                          int32_t num_pages, const int32_t *free_count, int32_t *free_count_out,
                          int32_t max_tokens, int64_t *slots, int32_t *positions, int32_t *seq_ids,
                          int32_t *query_start, int32_t *granted, int32_t *page_start, int32_t *error_word,
                          void *stream);

/*
 * Lengths after a verify step.  Of the reserved[b] tokens appended behind
 * seq_len[b] (spec_cache_extend's granted), sequence b keeps
 * k = accepted_len[b] + extra (extra = 1: the token the step started from and
 * its accepted drafts; accepted_len = -1 keeps none): seq_len_out[b] =
 * seq_len[b] + k, and the pages behind ceil(seq_len_out / page_size) go back
 * to the free list, the page taken last first, so that giving everything back
 * restores the list.  finished[b] != 0 (NULL: none) ends a sequence: its
 * length becomes 0 and all its pages go back.  Block table entries of pages
 * given back are left as they are and mean nothing any more.
 *   page_start [B + 1] out: sum of the pages given back before b (the total last)
 *   seq_len_out may be seq_len, free_count_out may be free_count
 * k outside [0, reserved] is clamped, with SV_ERR_LENGTH where anything was
 * reserved (a sequence without its pages keeps nothing); seq_len < 0,
 * reserved < 0 or a sum above max_blocks * page_size set it too, give nothing
 * back and leave the length (0 for a finished one).  Pages that would make
 * the list longer than num_pages are not put there (SV_ERR_PAGES); a page
 * outside [0, num_pages) is put there as -1, with SV_ERR_PAGE.
 * B <= 2^20.  One kernel launch, two for more than 1024 sequences, and where
 * B * max_blocks > 65536 and finished is given.
 */
int32_t spec_cache_commit(const int32_t *seq_len, const int32_t *reserved, const int32_t *accepted_len,
                          int32_t extra, const int32_t *finished, int32_t B, const int32_t *block_table,
                          int32_t max_blocks, int32_t page_size, int32_t *free_list, int32_t num_pages,
                          const int32_t *free_count, int32_t *free_count_out, int32_t *seq_len_out,
                          int32_t *page_start, int32_t *error_word, void *stream);

/*
 * The accepted path of a token tree (spec_verify_tree) in a paged cache.  The
 * tree's node i was written behind the `first` tokens it grew from (first = 1:
 * the root context), at position seq_len[b] + first + i; for i <
 * accepted_len[b] the rows of node path[b, i] move to position
 * seq_len[b] + first + i, so that the accepted tokens follow each other.  The
 * path must ascend, 0 <= path[b, 0] < path[b, 1] < ... < N (SV_ERR_TREE
 * otherwise), and its positions must lie below max_blocks * page_size
 * (SV_ERR_LENGTH): a sequence that fails is left as it is.  A page outside
 * [0, num_pages) sets SV_ERR_PAGE and that row does not move.  accepted_len
 * <= 0 moves nothing; above N is SV_ERR_TREE.
 *   pools  HOST array of device pointers, as for spec_beam_reorder_paged;
 *          path [B, N] int32, N <= 128
 * One kernel launch per 128 pools.
 */
int32_t spec_cache_compact(void *const *pools, int32_t n_pools, int32_t B, int32_t G, int32_t page_size,
                           int64_t row_bytes, int32_t num_pages, const int32_t *block_table, int32_t max_blocks,
                           const int32_t *seq_len, int32_t first, const int32_t *path,
                           const int32_t *accepted_len, int32_t N, int32_t *error_word, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECDECODE_H */
