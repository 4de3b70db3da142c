/*
 * qrotary.h -- queries and keys rotated by their position, and keys and values
 * appended to the 4-bit cache of qcache.h, in one call.  It stands between the
 * q/k/v product and the attention of a decoder block, in the place of
 * qcache_write.
 *
 * The first rot_dim dimensions of a query's or key's head are turned in pairs
 * (a, b), pair i by the angle  position * freqs[i]:
 *
 *   a' = a cos - b sin,   b' = b cos + a sin
 *   QROTARY_HALVES       pair i = dimensions i and rot_dim / 2 + i
 *   QROTARY_NEIGHBOURS   pair i = dimensions 2 i and 2 i + 1
 *
 * The others are left as they are.  The angle (a product in 64 bits, the
 * position exact), its sine and cosine, and the turn are formed in 64 bits;
 * the result is rounded to fp32 and from there to FP16 (q_out in fp32: to
 * fp32).  Turned keys and the values are then quantised into the cache as
 * qcache_write does.
 */
#ifndef QROTARY_H
#define QROTARY_H

#include "qcache.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QROTARY_HALVES = 0, QROTARY_NEIGHBOURS = 1 } qrotary_style;

/*
 *   rot_dim    a multiple of 16, 16 .. head_dim.
 *   style      qrotary_style.
 *   axes       axes of a position (time, height, width, ...), 1 .. 16.
 *   freqs      [rot_dim / 2] device memory, radians per position of each pair.
 *   pair_axis  int32 [rot_dim / 2] device memory, the axis by which each pair turns, or NULL: axis 0.
 *              A pair with an axis outside 0 .. axes - 1 is not turned.
 *   positions  int32 [axes][n_tok] device memory, or NULL (axes == 1): a row's own position in its
 *              sequence, as qcache.h defines it.  Where a row is stored goes by that in either case.
 * All are read when the kernel runs.
 */
typedef struct {
  int32_t rot_dim, style, axes;
  const double* freqs;
  const int32_t* pair_axis;
  const int32_t* positions;
} qrotary;

/*
 * q, q_out: n_q_heads heads (0 .. 65535; 0: neither is looked at), each FP16 or fp32; q_out may be q itself, with the
 * same type and strides, and overlaps nothing else that the call reads or writes.  k, v: as qcache_write, n_heads
 * heads; they are not changed.  A row that is on no page is turned all the same.
 * Errors: as qcache_write, plus INVALID_ARG (null or misaligned arrays, positions NULL with axes above 1, q_out
 * of overlapping vectors, or in q's place with another type or stride), UNSUPPORTED (rot_dim, style, axes, n_q_heads).
 */
int qrotary_write(const qcache_shape* shape, void* cache, const qcache_seqs* seqs, const qrotary* rotary,
                  int32_t n_q_heads, const qcache_rows* q, const qcache_rows* q_out, const qcache_rows* k,
                  const qcache_rows* v, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QROTARY_H */
