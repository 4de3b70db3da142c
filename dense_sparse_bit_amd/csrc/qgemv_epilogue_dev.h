// qgemv_epilogue_dev.h -- the kernels' side of include/qgemv_epilogue.h: what
// every product's epilogue computes and the check of its arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qgemv_epilogue.h"

namespace {

// ---------------------------------------------------------------------------
// Epilogue of a product: t = (W x)[row] + bias[row], then act(t) or, gated,
// act(t[2i]) * t[2i + 1] with the gate and up rows interleaved, plus the
// residual, rounded once to the output type.  It runs on the fp32 sums that
// the kernel holds anyway, so it moves only its own operands: the bias and
// residual are read and y written once, by the thread that owns the output
// (a residual that is y itself is read before it is written).  Every kernel
// is built with and without it, so that a plain product's code stays as it is.
// ---------------------------------------------------------------------------
template <bool EPI>
struct EpiArg {};

template <>
struct EpiArg<true> {
  const void* bias;
  const void* residual;
  void* y;
  int64_t ldy, ldr;  // elements between batch rows
  int act, gated, y32, bias32, res32;

  static __device__ __forceinline__ float load(const void* p, int f32, int64_t i) {
    return f32 ? ((const float*)p)[i] : (float)((const _Float16*)p)[i];
  }
  __device__ __forceinline__ float biased(float v, int row) const { return bias ? v + load(bias, bias32, row) : v; }
  __device__ __forceinline__ float activate(float t) const {
    switch (act) {
      case QGEMV_ACT_RELU: return t < 0.f ? 0.f : t;  // a NaN stays one
      // 1 + erf(z) = erfc(-z) and (1 + tanh u) / 2 = 1 / (1 + exp(-2u)): for t below zero the sums on the left cancel
      // (gelu(-5) would be off by 4 %, gelu(-6) would be 0), the right sides keep a relative error of a few ulps.
      case QGEMV_ACT_GELU: return 0.5f * t * erfcf(t * -0.70710678f);
      case QGEMV_ACT_GELU_TANH: return t / (1.f + expf(-1.5957691f * (t * __builtin_fmaf(0.044715f * t, t, 1.f))));
      case QGEMV_ACT_SILU: return t / (1.f + expf(-t));
      default: return t;
    }
  }
  __device__ __forceinline__ void store(int n, int col, float v) const {
    if (residual) v += load(residual, res32, n * ldr + col);
    if (y32) ((float*)y)[n * ldy + col] = v;
    else ((_Float16*)y)[n * ldy + col] = (_Float16)v;
  }
  __device__ __forceinline__ void put(int n, int row, float v) const { store(n, row, activate(biased(v, row))); }
  // row is even; g and u are the sums of rows row and row + 1
  __device__ __forceinline__ void put_gated(int n, int row, float g, float u) const {
    store(n, row >> 1, activate(biased(g, row)) * biased(u, row + 1));
  }
};

// Check an epilogue for M rows of weights and fill the kernels' argument.
int fill_epilogue(int M, void* y, const qgemv_epilogue* e, EpiArg<true>& a) {
  if (!e) return QGEMV_ERR_INVALID_ARG;
  if (e->act < QGEMV_ACT_NONE || e->act > QGEMV_ACT_SILU) return QGEMV_ERR_UNSUPPORTED;
  for (int t : {e->y_type, e->bias_type, e->residual_type})
    if (t != QGEMV_F16 && t != QGEMV_F32) return QGEMV_ERR_UNSUPPORTED;
  if (e->gated && M % 2) return QGEMV_ERR_UNSUPPORTED;
  const int64_t mo = e->gated ? M / 2 : M;
  const int64_t ldy = e->ldy ? e->ldy : mo, ldr = e->ldr ? e->ldr : mo;
  if (ldy < mo || ldr < mo) return QGEMV_ERR_INVALID_ARG;
  auto misaligned = [](const void* q, int t) { return (uintptr_t)q % (t == QGEMV_F32 ? 4 : 2) != 0; };
  if (misaligned(y, e->y_type) || misaligned(e->bias, e->bias_type) || misaligned(e->residual, e->residual_type))
    return QGEMV_ERR_INVALID_ARG;
  a.bias = e->bias;
  a.residual = e->residual;
  a.y = y;
  a.ldy = ldy;
  a.ldr = ldr;
  a.act = e->act;
  a.gated = e->gated != 0;
  a.y32 = e->y_type == QGEMV_F32;
  a.bias32 = e->bias_type == QGEMV_F32;
  a.res32 = e->residual_type == QGEMV_F32;
  return QGEMV_OK;
}

}  // namespace
