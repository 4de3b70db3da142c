/*
 * qcache.h -- a paged key/value cache held in 4 bits, and attention over it,
 * for MI355X (gfx950).  They stand between the q/k/v products and the output
 * product of a decoder block (qgemv.h, qgemv_epilogue.h).
 *
 * Storage.  A head's key or value vector of a token is cut into groups of
 * `group` consecutive dimensions.  A value v is rounded to FP16; then, per group,
 *
 *   lo = min v,   s = fp16((max v - lo) / 15),   q = clamp(rint((v - lo) / s), 0, 15)   (q = 0 where s = 0)
 *
 * with max v - lo, the two quotients and rint in FP32, round to nearest even;
 * where lo + 15 s would pass 65504, s is the FP16 below.  The value held is
 * lo + s q.  A group with a value that is not finite (or not finite in FP16)
 * has s = NaN and is read back as NaN.
 *
 * The cache is one device allocation of the caller of qcache_bytes bytes:
 * n_pages pages of page_size token slots of every head.  Its inner layout is
 * the library's own (csrc/qcache_layout.h).
 *
 * Sequences.  Every call describes the same batch (qcache_seqs):
 *   n_seq     sequences; n_tok  rows of the call's k, v, q or out.
 *   q_start   int32 [n_seq + 1], non-decreasing, q_start[0] = 0: sequence s owns the
 *             rows [q_start[s], q_start[s+1]); or NULL: one row per sequence,
 *             n_tok = n_seq.  Rows from q_start[n_seq] on are padding: not
 *             read, and left as they were.
 *   lens      int32 [n_seq]: tokens of the sequence, the call's own included:
 *             with n rows, row i stands at position lens[s] - n + i.
 *             0 (or less): an empty sequence.
 *   pages     int32 [n_seq][max_pages]: page of positions [p page_size,
 *             (p + 1) page_size).  A negative id, or one of n_pages or more, is no
 *             page.
 * A position that is negative, at or past max_pages * page_size, or on no page
 * holds nothing: it is not written, reads back as 0 and is not attended.
 * These three arrays are device memory and are read when the kernels run, so
 * a captured call sees their values at replay.
 *
 * Statuses are qgemv_status; no entry point aborts, throws, prints, allocates
 * or synchronises, and all are thread-safe.  The device of `stream` must be
 * current.  Calls that touch the same pages must be ordered by the caller.
 */
#ifndef QCACHE_H
#define QCACHE_H

#include "qgemv_epilogue.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   n_pages    1 .. 2^31 - 1.
 *   n_heads    key/value heads, 1 .. 65535.
 *   head_dim   64, 128 or 256.
 *   page_size  tokens of a page: a power of two, 16 .. 1024.
 *   group      32, 64 or 128, at most head_dim.
 */
typedef struct {
  int32_t n_pages, n_heads, head_dim, page_size, group;
} qcache_shape;

typedef struct {
  int32_t n_seq, n_tok, max_pages;
  const int32_t* q_start;
  const int32_t* lens;
  const int32_t* pages;
} qcache_seqs;

/*
 * Rows of vectors [n_tok][heads][head_dim] in device memory: the vector of row
 * t and head h starts at element t * tok_stride + h * head_stride.  type:
 * qgemv_dtype.  data is 16-byte aligned and both strides are multiples of 8
 * elements, so that vectors start on 16 bytes.  Vectors that are written must
 * not overlap; of those only read, a stride may be 0.
 */
typedef struct {
  void* data;
  int32_t type;
  int64_t tok_stride, head_stride;
} qcache_rows;

/* Bytes of the cache.  Host only.  Errors: INVALID_ARG (null pointer, a count below 1), UNSUPPORTED. */
int qcache_bytes(const qcache_shape* shape, size_t* bytes);

/*
 * Quantise the rows of k and v (FP16 or fp32, of one type) into their
 * positions.  cache: 256-byte aligned.  Two rows of one call at one position
 * of one page (pages shared between sequences at positions that the call
 * writes) leave either row's values or a mixture there.
 * Errors: INVALID_ARG (null pointer, misalignment, a negative count, n_tok
 * other than n_seq without q_start, k and v of different types), UNSUPPORTED
 * (shape, type; n_seq above 2^28; max_pages * page_size above 2^31 - 1025;
 * ceil(u / 2) * n_heads at 2^24, the workgroups of a launch, or more, with u =
 * n_seq, or n_tok / 16 + 2 n_seq with q_start), HIP.  n_seq or n_tok 0: nothing
 * is done.
 */
int qcache_write(const qcache_shape* shape, void* cache, const qcache_seqs* seqs, const qcache_rows* k,
                 const qcache_rows* v, void* stream);

/*
 * The inverse: row t of k and v gets the value held at the position where
 * qcache_write would have put row t, rounded once to the rows' type (lo + s q
 * formed in FP32).  Errors: as qcache_write.
 */
int qcache_read(const qcache_shape* shape, const void* cache, const qcache_seqs* seqs, const qcache_rows* k,
                const qcache_rows* v, void* stream);

/*
 * Workspace of qcache_attend for these counts (seqs' arrays are not looked
 * at).  Host only.  Errors: as qcache_attend.
 */
int qcache_attend_ws(const qcache_shape* shape, const qcache_seqs* seqs, int32_t n_q_heads, size_t* bytes);

/*
 * out[t][h] = sum_p softmax_p(scale q[t][h] . k[p][h / r]) v[p][h / r],  r = n_q_heads / n_heads,
 * over the positions p of row t's sequence up to row t's own.  A row with no
 * such position is 0.  q and out are FP16; scores, softmax statistics and sums
 * are fp32, the weights two FP16 (22 bits), the values that they multiply FP16.
 * n_q_heads: a multiple of n_heads, at most 65535.  scale: finite, also times log2 e.
 * ws: device memory, 256-byte aligned, of qcache_attend_ws bytes, contents
 * undefined before and after; calls that may overlap in time need one each.
 * Meant for a step's few rows per sequence; any number is taken, in tiles of
 * 16 (row, head) pairs that each read the sequence's cache.
 * Errors: INVALID_ARG, UNSUPPORTED (also where n_seq, n_tok and max_pages
 * allow 2^31 blocks of 128 tokens or more), SIZE (ws_bytes too small), HIP.
 */
int qcache_attend(const qcache_shape* shape, const void* cache, const qcache_seqs* seqs, int32_t n_q_heads,
                  const qcache_rows* q, const qcache_rows* out, float scale, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QCACHE_H */
