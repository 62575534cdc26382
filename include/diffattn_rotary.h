/*
 * Rotary positions for the queries and keys of the differential-attention head
 * (part of libdiffattn; types, status codes and conventions as in diffattn.h).
 *
 * The first `rot` channels of a row are rot / 2 pairs, (i, i + rot / 2) or,
 * with neighbours, (2i, 2i + 1).  At position p pair i is turned by the angle
 * p f_i and scaled:
 *
 *   y_a = m (x_a cos(p f_i) - x_b sin(p f_i))
 *   y_b = m (x_a sin(p f_i) + x_b cos(p f_i))
 *
 * and the other channels are copied.  Its gradient is the turn by -p f_i.
 *
 * Frequencies are kept in turns per position as 64-bit fractions: p f_i is then
 * an integer product that wraps as angles do, without rounding for any 64-bit
 * position.  What a far position adds is the error of the fraction itself, below
 * 2^-55 of a turn as diffrotary_frequencies works it out in fp64: the angle is off
 * by |p| 2^-55 of a turn, 2^-24 at p = 2^31.
 */
#ifndef DIFFATTN_ROTARY_H
#define DIFFATTN_ROTARY_H

#include "diffattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum diffrotary_scaling {
    DIFFROTARY_NONE = 0,   /* f_i = base^(-2i / rot), m = 1 */
    DIFFROTARY_LINEAR = 1, /* f_i / factor */
    DIFFROTARY_NTK = 2,    /* base grows by factor^(rot / (rot - 2)) */
    DIFFROTARY_PARTS = 3   /* f_i (g + (1 - g) / factor), g = clamp((original f_i / (2 pi) - slow)
                              / (fast - slow), 0, 1): pairs that turn at least `fast` times within
                              the `original` positions stay, those of at most `slow` turns are
                              stretched; m = 0.1 ln(factor) + 1 */
} diffrotary_scaling;

typedef struct diffrotary_table {
    const uint64_t *freq; /* device [rot / 2]: turns per position in units of 2^-64 */
    int32_t rot;          /* channels that are turned: a multiple of 16, at most d */
    int32_t neighbours;   /* pairs (2i, 2i + 1) instead of (i, i + rot / 2) */
    float scale;          /* m */
    int32_t reserved;     /* 0 */
} diffrotary_table;

/*
 * diffrotary_frequencies — the table's contents (host only): writes rot / 2
 * fractions to freq (host memory) and m to scale.  base > 1, factor >= 1;
 * DIFFROTARY_PARTS also takes original > 0 and 0 <= slow < fast.
 */
diffattn_status diffrotary_frequencies(int32_t rot, double base, int32_t scaling, double factor,
                                       double original, double fast, double slow, uint64_t *freq,
                                       float *scale);

/*
 * diffrotary_apply — turns the rows of up to four tensors (q1, q2, k1, k2, each
 * with its own number of heads).
 *
 * x[k], y[k], k < count: device [B, heads[k], N, d], 16-byte aligned, with the
 * element strides strides[2 k] (x) and strides[2 k + 1] (y), rows contiguous
 * (positive multiples of 16 bytes, below 2^39 elements), or strides NULL when
 * all are contiguous.  y[k] may be x[k] with the same strides (in place);
 * otherwise outputs overlap neither one another nor the inputs.
 * positions: device int32, row i of batch b at positions[b * position_stride + i]
 * (position_stride 0: the same for all batches), any values; NULL: start + i.
 * inverse != 0 turns back (the gradient: x holds dy, y receives dx).
 * desc: B, N, d (64 or 128), dtype DIFFATTN_BF16 or DIFFATTN_F32; H is not used
 * (the tensors have their own); B * N < 2^31.
 */
diffattn_status diffrotary_apply(const diffattn_desc *desc, const diffrotary_table *table,
                                 int32_t count, const void *const *x, void *const *y,
                                 const int64_t *heads, const diffattn_strides *strides,
                                 const int32_t *positions, int64_t position_stride, int64_t start,
                                 int32_t inverse, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DIFFATTN_ROTARY_H */
