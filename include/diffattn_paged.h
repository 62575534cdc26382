/*
 * Paged key/value cache of the differential-attention head: the operators of
 * a decoding step (part of libdiffattn; types and status codes as in
 * diffattn.h, whose conventions hold here too: caller-owned device buffers,
 * nothing allocated, calls asynchronous on `stream`, validation before any
 * launch, no C++ exception across the ABI).
 *
 * A cache keeps the keys and values of B sequences in pages of page_size
 * tokens.  Page page_table[b][t / page_size] holds, at row t % page_size, the
 * rows k1, k2 (d wide) and v (2d wide) of token t of sequence b, for each of
 * kv_heads key/value heads.  kv_len[b] is the sequence's length; it counts the
 * tokens of the step in progress, so the N newest tokens of a call sit at the
 * positions kv_len[b] - N + i, i = 0 .. N - 1.  A negative position is padding
 * (kv_len[b] < N: prompts padded at the front; kv_len[b] = 0: an idle row of
 * the batch): it is never written and its output row is zero.  All lengths and
 * the table are read on the device, so a captured graph replays with new ones.
 *
 * A decoding step: the caller raises kv_len, diffpaged_append writes the new
 * tokens' rows, diffpaged_fwd attends and may add each key's weight to the
 * cache's weights, and diffpaged_evict, when a sequence has outgrown its
 * budget, keeps the keys of the largest weights.
 *
 * A page number outside 0 .. num_pages - 1 or a length outside
 * 0 .. max_pages * page_size is found on the device: nothing outside the pool
 * is touched, DIFFATTN_ERR_PAGE is stored in desc->status_dev (when given),
 * and that sequence's output rows are NaN (fwd), its rows on valid pages are
 * written (append; nothing of it where its length is bad), it is left as it is
 * (evict; the weights of fwd).  Entries of the table past a sequence's length
 * are not read, and by append only those of the new tokens, by evict only those
 * of the sequences that it cuts.
 *
 * Sequences may share pages (a common prefix) in a call that only reads them:
 * diffpaged_fwd without accumulate.  A page that a call writes (append: those
 * of the new tokens; fwd with accumulate and evict: all) stands once only in
 * the table, else its contents afterwards are undefined.  Calls that write a
 * cache are ordered with all others on it (same stream, or synchronised).
 *
 * The kernels are launched with programmatic stream serialisation: they may
 * start while the kernel before them on the stream drains, and wait for its
 * end before they touch memory.
 */
#ifndef DIFFATTN_PAGED_H
#define DIFFATTN_PAGED_H

#include "diffattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache.  Element (page, head, row, c) of k1, k2 or v sits at page * s.b +
 * head * s.h + row * s.n + c of its tensor, s its strides: the pages may be
 * stored head by head ([pages, kv_heads, page_size, width]) or token by token
 * ([pages, page_size, kv_heads, width]).  Strides are positive multiples of 16
 * bytes and below 2^39 elements, and the tensors 16-byte aligned.  The rows
 * of k1, k2 and v do not overlap (one buffer may hold them side by side). */
typedef struct diffpaged_cache {
    void *k1;                  /* bf16, or e4m3 with DIFFATTN_E4M3_QK; width d */
    void *k2;                  /* as k1 */
    void *v;                   /* bf16, width 2d */
    float *weights;            /* fp32 [num_pages, kv_heads, page_size] or NULL */
    const int32_t *page_table; /* int32 [B, max_pages] */
    int32_t *kv_len;           /* int32 [B]; written by diffpaged_evict alone */
    diffattn_strides k1_strides, k2_strides, v_strides;
    int64_t num_pages;         /* >= 1 */
    int64_t kv_heads;          /* >= 1 */
    int64_t max_pages;         /* >= 1 */
    int32_t page_size;         /* a multiple of 16; max_pages * page_size < 2^30 */
    int32_t reserved;          /* 0 */
} diffpaged_cache;

/*
 * diffpaged_append — write the N newest tokens' rows to the cache.
 *
 * k1, k2: device bf16 [B, kv_heads, N, d]; v: device bf16 [B, kv_heads, N, 2d];
 * strides[0..2] theirs in elements (the rules of diffattn_fwd_strided), or
 * NULL when they are contiguous.  Any N >= 0: one token or a prompt.  With
 * DIFFATTN_E4M3_QK the k1 and k2 values are rounded to the nearest e4m3 value,
 * ties to even, beyond +-448 to +-448 (NaN stays NaN); v is copied.  Where the
 * cache has weights, those of the written tokens are set to zero.
 * desc: B, N, d (64 or 128), dtype (DIFFATTN_BF16 or DIFFATTN_E4M3_QK); H =
 * kv_heads; the other fields are checked but not used.
 */
diffattn_status diffpaged_append(const diffattn_desc *desc, const diffpaged_cache *cache,
                                 const void *k1, const void *k2, const void *v,
                                 const diffattn_strides *strides, void *stream);

/*
 * diffpaged_fwd — the differential head's forward of the N newest tokens of
 * each sequence against its cache.
 *
 *   out = norm((map1 - lambda_h map2) V), the formula, head norms (headnorm 0,
 *   1, 2), w and (1 - lambda_init) of diffattn_fwd
 *
 * q1, q2: device [B, H, N, d], bf16 or (DIFFATTN_E4M3_QK) e4m3; out: device
 * bf16 [B, H, N, 2d]; strides[0..2] those of q1, q2, out, or NULL when
 * contiguous; lambda fp32 [H], norm_w fp32 [H, 2d] or NULL.  H is a multiple of
 * kv_heads: query head h reads key/value head h / (H / kv_heads).  causal = 1:
 * token i sees the keys up to its own position; 0: all kv_len[b] keys.  A row
 * that sees no key is zero.  What masked or unused places of the pages hold
 * (NaN and infinities too) has no influence.  A key whose logit is -infinity
 * has no weight beside others.  A NaN or infinite value (v) that a row sees
 * makes its column of the row NaN or infinite, an infinite one NaN as well
 * (inf - inf in the two maps' difference and in the products that make it up),
 * and with a head norm the whole row NaN.
 *
 * accumulate != 0 also adds, for every key j of a sequence and each key/value
 * head, sum |map1[j] - lambda_h map2[j]| over the N tokens and the query heads
 * that read it, to cache->weights (a fixed order of addition: repeated runs
 * give the same bits).
 *
 * The products with V add up in fp32 and drop what does not fit, over the keys
 * that one CTA takes of an item: up to 2^18 of them that is below an output's
 * rounding; where values are of one sign, outputs are 0.5 % too small after 2^20
 * keys and 2 % after 2^22 (measured).
 *
 * workspace: caller-owned scratch of at least the bytes diffpaged_fwd_plan
 * gives for the same desc and cache sizes, 256-byte aligned; its contents on
 * entry do not matter; calls (and captured graphs) that share one must be
 * ordered.  NULL is fine when the plan gives 0.  It goes by the table's
 * capacity, not by the lengths: with accumulate about 8 bytes per query head,
 * new token and place (B * H * N * max_pages * page_size), beside partial
 * states of at most 128 KB per SM.
 *
 * Domain (else DIFFATTN_ERR_UNSUPPORTED): d 64 or 128, DIFFATTN_BF16 or
 * DIFFATTN_E4M3_QK, N <= 16, H / kv_heads <= 64, page_size a multiple of 16,
 * an sm_103 device.  A longer run of new tokens (a chunk of a prompt) has no
 * form over pages: diffattn_fwd_kv takes contiguous keys and values of equal
 * lengths with as many heads as the queries (for e4m3 keys d = 64 and head
 * norms 0 and 1 only), so its rows have to be gathered and repeated first.
 */
diffattn_status diffpaged_fwd(const diffattn_desc *desc, const diffpaged_cache *cache,
                              const void *q1, const void *q2, const float *lambda,
                              const float *norm_w, void *out, const diffattn_strides *strides,
                              int accumulate, void *workspace, size_t workspace_bytes,
                              void *stream);

/* Workspace bytes of diffpaged_fwd (host-only apart from the SM count). */
diffattn_status diffpaged_fwd_plan(const diffattn_desc *desc, const diffpaged_cache *cache,
                                   int accumulate, size_t *workspace_bytes);

/*
 * diffpaged_evict — cut every sequence longer than `keep` down to `keep` keys.
 *
 * Each key/value head chooses for itself: the last `recent` keys stay, and of
 * the others the keep - recent of the largest cache->weights (equal weights:
 * the lower position stays; a NaN counts as +infinity, -0 as 0).  The kept
 * keys' rows and weights move to positions 0 .. keep - 1 in their order, in
 * place; rows at positions >= keep stay as they were; kv_len[b] becomes keep,
 * and the sequence's pages past ceil(keep / page_size) are free for the caller.
 * (So each cache that is evicted from, a layer's for instance, needs a kv_len
 * of its own: with a shared one the second cache's sequences would be short
 * already.)
 * Sequences of at most `keep` keys are left as they are.  0 <= recent <= keep.
 * (Positions count from the front of the cache: rotary or other position
 * information is already in the stored keys.)
 *
 * workspace as for diffpaged_fwd, its size from diffpaged_evict_plan.
 * desc: B, d, dtype as above, H = kv_heads; N is not used.
 */
diffattn_status diffpaged_evict(const diffattn_desc *desc, const diffpaged_cache *cache,
                                int64_t keep, int64_t recent, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Workspace bytes of diffpaged_evict (host-only). */
diffattn_status diffpaged_evict_plan(const diffattn_desc *desc, const diffpaged_cache *cache,
                                     int64_t keep, size_t *workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* DIFFATTN_PAGED_H */
