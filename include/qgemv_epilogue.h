/*
 * qgemv_epilogue.h -- the quantized product of qgemv.h with an epilogue.
 *
 *   t[b][i] = (W x[b])[i] + bias[i]
 *   y[b][i] = act(t[b][i]) + residual[b][i]                                  (gated == 0)
 *   y[b][i] = act(t[b][2i]) * t[b][2i + 1] + residual[b][i],  i < M / 2      (gated != 0)
 *
 * W is any plan of qgemv_create, in any of its formats.  The gated form takes
 * weights whose rows alternate between a gate and an up projection (rows are
 * independent in every format, so interleaving two weight sets row by row is
 * done on the canonical arrays, before qgemv_repack).
 *
 * Sums, bias, activation and residual are fp32; y is rounded once to its type.
 * An FP16 y is what the next product takes as x.
 */
#ifndef QGEMV_EPILOGUE_H
#define QGEMV_EPILOGUE_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QGEMV_ACT_NONE = 0,      /* t                                                            */
  QGEMV_ACT_RELU = 1,      /* max(t, 0)                                                    */
  QGEMV_ACT_GELU = 2,      /* t/2 (1 + erf(t / sqrt 2))                                    */
  QGEMV_ACT_GELU_TANH = 3, /* t/2 (1 + tanh(sqrt(2/pi) (t + 0.044715 t^3)))                */
  QGEMV_ACT_SILU = 4       /* t / (1 + exp(-t))                                            */
} qgemv_act;

typedef enum { QGEMV_F16 = 0, QGEMV_F32 = 1 } qgemv_dtype;

/*
 *   act, gated     see above; gated needs an even M.
 *   y_type, bias_type, residual_type   qgemv_dtype of each array (checked also
 *                  where the array is NULL).
 *   bias           [M] device memory, or NULL.
 *   residual       [batch][M or M / 2] device memory, or NULL.  It may be y
 *                  itself, with the same type and row stride (each element is
 *                  read before it is written); any other overlap of y with x,
 *                  bias or residual is not allowed.
 *   ldy, ldr       elements between the batch rows of y and of residual; 0
 *                  means dense (M, or M / 2 when gated).
 */
typedef struct {
  int32_t act, gated;
  int32_t y_type, bias_type, residual_type;
  const void* bias;
  const void* residual;
  int64_t ldy, ldr;
} qgemv_epilogue;

/*
 * Enqueue the product with its epilogue on `stream`.  x_dev, batch, workspace,
 * stream capture and concurrency: as qgemv_run.  y_dev: device memory aligned
 * to its type; every output element is written and nothing between the rows of
 * a strided y is touched.
 * Errors: as qgemv_run, plus INVALID_ARG (null e, arrays not aligned to their
 * type, ldy or ldr shorter than a row), UNSUPPORTED (unknown activation or
 * type, gated with an odd M).
 */
int qgemv_run_epilogue(qgemv_handle h, const void* x_dev, void* y_dev, int32_t batch, const qgemv_epilogue* e,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_EPILOGUE_H */
