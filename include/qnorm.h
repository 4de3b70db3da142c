/*
 * qnorm.h -- the norms after and before a block, fused with the gate and the
 * residual stream between them, for MI355X (gfx950).  Row by row, with n
 * columns:
 *
 *   b   = y, or norm(y) * post + post_bias
 *   h'  = scale * h + gate * b
 *   out = norm(h') * pre + pre_bias
 *
 *   norm(x) = x / sqrt(mean(x^2) + eps)                              QNORM_RMS
 *   norm(x) = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps)      QNORM_LAYER
 *
 * Everything is fp32, and h' and its norm 64 bits where out is fp32 or blocks,
 * until one rounding of h' and of out to their types; the second norm takes h'
 * before its rounding.  out may be rows in MX blocks
 * (qmx.h), which the next product takes.
 *
 * Statuses are qgemv_status; the entry point does not abort, throw, print,
 * allocate or synchronise, and is thread-safe.  The device of `stream` must be
 * current.  All arrays are device memory.
 */
#ifndef QNORM_H
#define QNORM_H

#include "qmx.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QNORM_RMS = 0, QNORM_LAYER = 1 } qnorm_kind;

/* Types of out beyond qgemv_dtype: rows in MX blocks of a qmx_format, quantised with clip == 0. */
enum { QNORM_OUT_E2M1 = 16, QNORM_OUT_E4M3 = 17 };

/*
 * An array of the call, or data NULL: none.  Row r starts at element r * ld (ld
 * 0: the same vector for every row); type: qgemv_dtype.  data is 16-byte aligned,
 * ld a multiple of 8.
 */
typedef struct {
  void* data;
  int32_t type;
  int64_t ld;
} qnorm_rows;

/*
 *   rows       0 .. 2^26 (0: nothing is done), and, to the next multiple of 128, fewer than 2^35 / (cols, or 512, to the next
 *              power of two).
 *   cols       a multiple of 8 (out in blocks: of 32), 8 .. 32768.
 *   y, h       at least one of them.  Without y, h' = scale * h, and neither gate nor post is given.
 *   gate       or none: 1.  ld 0: a factor per column.
 *   post, post_bias, pre, pre_bias   vectors (ld is not looked at).  Without post, y is not normalised and there is no
 *              post_bias; without pre there is no out and no pre_bias.
 *   h_out      or none: h' is not written.
 *   out        given where pre is; type qgemv_dtype, or QNORM_OUT_E2M1 / QNORM_OUT_E4M3: data is then 256-byte aligned, of
 *              qmx_bytes bytes, and ld is not looked at.
 * h_out and out (not both) may be y or h itself, with the same type and ld.  They overlap nothing else that the call reads or
 * writes, and their rows do not overlap.
 */
typedef struct {
  int32_t rows, cols, kind;
  float eps, scale;
  qnorm_rows y, h, gate, post, post_bias, pre, pre_bias, h_out, out;
} qnorm_args;

/*
 * Errors: INVALID_ARG (null args, misalignment, a combination excluded above, a
 * negative or not finite eps, scale not finite, no output, outputs of overlapping rows, both outputs in
 * one place, an output in y's or h's with another type or ld), UNSUPPORTED (rows, cols, kind, types), HIP.
 */
int qnorm_run(const qnorm_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QNORM_H */
