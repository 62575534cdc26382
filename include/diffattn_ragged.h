/*
 * A serving step over a packed ("ragged") batch on the paged cache of
 * diffattn_paged.h: prompts, chunks of prompts and single tokens together (part
 * of libdiffattn; types, status codes and conventions as there).
 *
 * The new tokens of B sequences stand behind one another in tensors of N rows:
 * those of sequence b are rows q_start[b] .. q_start[b + 1] - 1 (q_start: device
 * int32 [B + 1], not falling, q_start[0] >= 0); rows outside q_start[0] ..
 * q_start[B] - 1 belong to none: they are not written, and what they hold has no
 * influence.  A sequence's
 * n tokens are its newest: token i sits at position kv_len[b] - n + i of its
 * cache (kv_len counts them; a negative position is padding).
 *
 * A step: diffragged_step grows the sequences, gives them pages and works out
 * where each token goes; per layer, diffragged_append turns the queries and
 * keys and writes the cache's rows, and diffragged_fwd attends.  All sizes but
 * the tensors' capacities are read on the device, so a captured step replays
 * with new ones.
 *
 * Eviction.  Nothing here adds to a cache's weights (diffpaged_fwd with
 * accumulate does), and diffragged_append sets those of new places to zero:
 * after packed steps alone all weights are equal, and diffpaged_evict keeps the
 * last `recent` keys and the first keep - recent.  It cuts one cache's lengths,
 * so a cache that is evicted from has a book of its own.  Positions count the
 * places of a cache: after an eviction they are lower than the tokens' places in
 * the text, and a caller whose kept keys are turned by those gives
 * diffragged_append positions of its own.
 */
#ifndef DIFFATTN_RAGGED_H
#define DIFFATTN_RAGGED_H

#include "diffattn_paged.h"
#include "diffattn_rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The pages of a cache (or of several of one geometry, such as the layers' of a
 * model) and who has them; all device int32. */
typedef struct diffragged_book {
    int32_t *kv_len;     /* [B] lengths */
    int32_t *held;       /* [B] pages that each sequence has: the first entries of its table */
    int32_t *page_table; /* [B, max_pages] */
    int32_t *free_pages; /* [capacity] a stack of the pages that nobody has */
    int32_t *free_count; /* [1] how many */
    int64_t B;
    int64_t max_pages;   /* >= 1 */
    int64_t capacity;    /* >= 0 */
    int32_t page_size;   /* >= 1; max_pages * page_size < 2^30 */
    int32_t reserved;    /* 0 */
} diffragged_book;

/*
 * diffragged_step — the batch's bookkeeping for one step.
 *
 * new_len: device int32 [B], each sequence's new tokens; -1 ends a sequence (its
 * length becomes 0).  Lengths grow; a sequence then holds ceil(length /
 * page_size) pages: what it has beyond that (it has ended, or diffpaged_evict
 * has cut it) goes back on the stack, by sequence and place in its table, and
 * what it lacks is then taken from the top of the stack, in the same order.
 * Entries of the table that no longer hold a page keep their values, and so do
 * those of free_pages above the new count.  Each page stands once, in one
 * sequence's table or on the stack: one that several sequences share (which
 * diffragged_fwd may read) would be given back by each of them, so tables with
 * shared pages are not for a book.
 *
 * Outputs: q_start [B + 1]; for each packed row positions [N] (int32) and slots
 * [N] (int64, page * page_size + row in it), either NULL when not wanted, -1 in
 * rows behind the last token.
 *
 * Calls on a book are ordered with those that use its lengths and table (same
 * stream, or synchronised).  N and capacity are at most 2^30.
 *
 * A step that does not fit (too few free pages, more than N tokens, a sequence
 * longer than its table, a stack that would outgrow its capacity) or whose
 * numbers are wrong (new_len < -1; a negative length or count; held outside
 * ceil(length / page_size) .. max_pages) changes nothing: q_start is all 0,
 * positions and slots all -1, and DIFFATTN_ERR_PAGE is stored in status (when
 * given).
 */
diffattn_status diffragged_step(const diffragged_book *book, const int32_t *new_len, int64_t N,
                                int32_t *q_start, int32_t *positions, int64_t *slots,
                                int32_t *status, void *stream);

/*
 * diffragged_append — the packed tokens' rows into the cache, turned by their
 * positions.
 *
 * q1, q2: device bf16 [N, H, d]; k1, k2: [N, kv_heads, d]; v: [N, kv_heads, 2d];
 * q1_out, q2_out: [N, H, d], bf16 or, with DIFFATTN_E4M3_QK, e4m3.  q1, q2 and
 * their outputs are all NULL where only the cache is written; a bf16 output may
 * be its input (same strides).  strides[0..6]: those of q1, q2, k1, k2, v,
 * q1_out, q2_out in elements (n: of a token, h: of a head, b not used; positive
 * multiples of 16 bytes below 2^39), or NULL when all are contiguous.
 * slots: device int64 [N]; a token of slot -1 is left out, its query rows too;
 * one outside -1 .. num_pages * page_size - 1 as well, and DIFFATTN_ERR_PAGE is
 * stored.  No slot but -1 stands twice.  table NULL: nothing is turned, else
 * positions (device int32 [N]) has each token's.  Values are rounded once, to
 * bf16 or (saturating at +-448, NaN stays NaN) to e4m3; v is copied.  Weights of
 * the written places become zero where the cache has any.
 * desc: N, H (a multiple of kv_heads; with q1 NULL only checked), d, dtype;
 * B and the rest are checked but not used.
 */
diffattn_status diffragged_append(const diffattn_desc *desc, const diffpaged_cache *cache,
                                  const void *q1, const void *q2, const void *k1, const void *k2,
                                  const void *v, void *q1_out, void *q2_out,
                                  const diffattn_strides *strides, const int64_t *slots,
                                  const diffrotary_table *table, const int32_t *positions,
                                  void *stream);

/*
 * diffragged_fwd — the differential head's forward of all new tokens against
 * their sequences' pages: any numbers of them, from none and one to a whole
 * prompt.
 *
 * q1, q2: device [N, H, d], bf16 or (DIFFATTN_E4M3_QK) e4m3; out: bf16 [N, H, 2d];
 * strides[0..2] those of q1, q2, out (as above) or NULL; lambda fp32 [H], norm_w
 * fp32 [H, 2d], 16-byte aligned, or NULL.  The formula, norms,
 * heads, causal (token i sees the keys up to its own position; 0: all kv_len[b])
 * and what masked and unused places hold are as in diffpaged_fwd: a row that
 * sees no key is zero, a value that is not finite reaches those rows only that
 * see it, and makes its column (with a head norm the row) of them NaN.
 * A page number outside the pool, a length outside the table or rows outside
 * 0 .. N store DIFFATTN_ERR_PAGE: rows that would have read such a page are NaN
 * (others of the sequence may be), so are all of a bad length, and those of a
 * sequence whose q_start is wrong are not written (of the whole batch where its
 * sequences, wrong ones apart, have more than N rows together).
 *
 * Precision.  Logits, references, sums and both maps' products with V are held
 * in fp32, whatever the lengths.  A weight enters the product with V as one bf16
 * number (in diffpaged_fwd as two): before the norm an output may be off by 2^-8
 * of sum (map1 + |lambda| map2) |v|, beside its own rounding.  Measured against
 * 64 bits, outputs are off by 0.0018 to 0.0024 of their size, those of
 * diffpaged_fwd by 0.0016 to 0.0017, bf16's rounding alone.  Where both maps of a
 * row lean on one key, these roundings cancel as the maps do at d = 128; at
 * d = 64 they do so for a key among the first 128 that a CTA takes of the row,
 * and others show as 1 / |1 - lambda|: such rows were off by up to 0.008 with
 * lambda = 0.8 and 0.2 with 0.95 (in diffpaged_fwd by 0.002).
 *
 * workspace: as for diffpaged_fwd; its size does not depend on the lengths.
 * desc: B sequences, N rows, H, d (64 or 128), dtype, causal, headnorm, eps,
 * lambda_init.  Domain: H / kv_heads <= 64, page_size a multiple of 16, and
 * kv_heads (N / floor(128 kv_heads / H) + B) (5 max_pages page_size / 128 + 20) <
 * 2^31 (a call of 65536 rows of 32 heads over 8 key/value heads in tables of a
 * million keys comes to a third of that).
 */
diffattn_status diffragged_fwd(const diffattn_desc *desc, const diffpaged_cache *cache,
                               const int32_t *q_start, const void *q1, const void *q2,
                               const float *lambda, const float *norm_w, void *out,
                               const diffattn_strides *strides, void *workspace,
                               size_t workspace_bytes, void *stream);

/* Workspace bytes of diffragged_fwd (host-only apart from the SM count). */
diffattn_status diffragged_fwd_plan(const diffattn_desc *desc, const diffpaged_cache *cache,
                                    size_t *workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* DIFFATTN_RAGGED_H */
