/*
 * qmx.h -- rows in microscaled blocks (MX), and the product of two sets of
 * them on the scaled MFMAs of MI355X (gfx950).  They stand next to the
 * products of qgemv.h: weights in 4-bit floats, any number of activation rows.
 *
 * Storage.  A row is cut into blocks of 32 consecutive columns.  A block holds
 * one exponent byte b (the power of two 2^(b - 127); 255: the block is NaN) and
 * 32 elements, each the value element * 2^(b - 127):
 *
 *   QMX_E2M1   4 bits: sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   QMX_E4M3   8 bits: sign, 4 exponent bits, 3 mantissa bits, up to 448 (0x7F and 0xFF are NaN)
 *
 * Quantising a block with the largest magnitude `top` takes the power of two
 *
 *   clip == 0   the smallest 2^e with top <= largest element * 2^e: nothing saturates
 *   clip != 0   2^(floor(log2 top) - floor(log2 largest element)): the elements that then
 *               lie above the largest are held at it
 *
 * with e >= -126, and rounds value / 2^e to the nearest element, ties to even.
 * A block with a value that is not finite is NaN.
 *
 * Rows in blocks lie in one device allocation of the caller's, 256-byte aligned,
 * of qmx_bytes bytes, in the library's own order (csrc/qmx_layout.h).
 *
 * Statuses are qgemv_status; no entry point aborts, throws, prints, allocates
 * or synchronises, and all are thread-safe.  The device of `stream` must be
 * current.  All arrays are device memory.
 */
#ifndef QMX_H
#define QMX_H

#include "qgemv_epilogue.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QMX_E2M1 = 0, QMX_E4M3 = 1 } qmx_format;

/*
 *   rows    0 .. 2^26 (0: nothing is done; weights have 1 or more); with rows in tiles of 16 and columns in chunks of 128,
 *           fewer than 2^26 of these.
 *   cols    a multiple of 32, 32 .. 2^20.
 *   format  qmx_format.
 */
typedef struct {
  int32_t rows, cols, format;
} qmx_shape;

/* Bytes of such rows in blocks.  Host only.  Errors: INVALID_ARG (null pointer, a negative count, no columns), UNSUPPORTED. */
int qmx_bytes(const qmx_shape* shape, size_t* bytes);

/*
 * Quantise x [rows][cols], FP16 or fp32 (qgemv_dtype), row r from element r * ldx
 * on; x is 16-byte aligned and ldx a multiple of 8 (0: every row the same).
 * Errors: INVALID_ARG (null pointer, misalignment), UNSUPPORTED (shape, type), HIP.
 */
int qmx_quantize(const qmx_shape* shape, void* blocks, const void* x, int32_t x_type, int64_t ldx, int32_t clip,
                 void* stream);

/* The inverse: the values that the blocks stand for, rounded once to x's type.  Rows of x must not overlap.  Errors: as qmx_quantize. */
int qmx_values(const qmx_shape* shape, const void* blocks, void* x, int32_t x_type, int64_t ldx, void* stream);

/*
 * From and to plain arrays, dense: codes [rows][cols / 2] bytes with the lower
 * column in the lower nibble (E2M1) or [rows][cols] bytes (E4M3), 16-byte
 * aligned, and exponents [rows][cols / 32] bytes.  Errors: as qmx_quantize.
 */
int qmx_pack(const qmx_shape* shape, void* blocks, const void* codes, const void* exponents, void* stream);
int qmx_unpack(const qmx_shape* shape, const void* blocks, void* codes, void* exponents, void* stream);

/*
 * The right-hand side of a product: rows in blocks (x_type QMX_IN_BLOCKS; ldx is
 * not looked at), or FP16 or fp32 rows (qgemv_dtype; alignment as
 * qmx_quantize), which are quantised to `format` on the way, clip == 0.
 */
enum { QMX_IN_BLOCKS = -1 };
typedef struct {
  const void* data;
  int32_t rows, format, x_type;
  int64_t ldx;
} qmx_input;

/* Workspace of qmx_run for these counts (x->data is not looked at); 0 for x in blocks.  Host only.  Errors: as qmx_run. */
int qmx_run_ws(const qmx_shape* w, const qmx_input* x, const qgemv_epilogue* e, size_t* bytes);

/*
 * y = epilogue(x W^T), with the epilogue of qgemv_epilogue.h: y[t][i], M = w->rows,
 * any number of rows t.  W: E2M1.  Products are exact, sums fp32.
 * ws: device memory, 256-byte aligned, of qmx_run_ws bytes (0: may be NULL),
 * contents undefined before and after; calls that may overlap in time need one
 * each.  y overlaps nothing that the call reads, except that it may be the residual
 * itself, with the same type and row stride.
 * Errors: INVALID_ARG (null pointer, misalignment, counts below 1, ldy or ldr
 * shorter than a row, the residual in y's place with another type or row stride),
 * UNSUPPORTED (shape, type, format, activation, gated with an odd M, 2^24 tiles
 * of 64 x 64 outputs or more), SIZE (ws_bytes too small), HIP.
 */
int qmx_run(const qmx_shape* w, const void* w_blocks, const qmx_input* x, void* y, const qgemv_epilogue* e, void* ws,
            size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMX_H */
