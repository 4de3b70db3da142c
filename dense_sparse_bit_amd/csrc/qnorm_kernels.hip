// qnorm_kernels.hip -- the norms after and before a block, fused with the gate
// and the residual stream (include/qnorm.h).

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/qnorm.h"
#include "qgemv_decode.h"
#include "qgemv_internal.h"
#include "qmx_blocks.h"
#include "qmx_layout.h"
#include "qnorm_sums.h"

using namespace qgemv_dev;
using namespace qmx_dev;
using qmx_layout::Geo;

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct Arr {
  char* data;
  int f32;
  int64_t ld;
};

struct NormArgs {
  Arr y, h, gate, post, post_bias, pre, pre_bias, h_out, out;
  Geo g;  // out in blocks
  int rows, cols, by_tile;
  float eps, scale;
  double inv_n;
};

__device__ __forceinline__ void load8(const Arr& a, int64_t row, int col, float (&v)[8]) {
  const int64_t e = row * a.ld + col;
  if (a.f32) {
    const floatx4_t* p = (const floatx4_t*)((const float*)a.data + e);
    const floatx4_t x = p[0], y = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i], v[4 + i] = y[i];
  } else {
    const half8_t x = *(const half8_t*)((const _Float16*)a.data + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
  }
}
// Eight values as they lie in memory: half the registers where they are FP16 (the second half is then not set).
struct Raw8 {
  u32x4_t a, b;
};
__device__ __forceinline__ Raw8 raw8(const Arr& a, int64_t row, int col) {
  const int64_t e = row * a.ld + col;
  Raw8 r;
  r.a = *(const u32x4_t*)(a.data + (a.f32 ? 4 : 2) * e);
  if (a.f32) r.b = *(const u32x4_t*)(a.data + 4 * e + 16);
  return r;
}
__device__ __forceinline__ void of_raw8(const Arr& a, const Raw8& r, float (&v)[8]) {
  if (a.f32) {
    const floatx4_t x = __builtin_bit_cast(floatx4_t, r.a), y = __builtin_bit_cast(floatx4_t, r.b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i], v[4 + i] = y[i];
  } else {
    const half8_t x = __builtin_bit_cast(half8_t, r.a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
  }
}
// A double between two floats as the one of them whose last bit is set: what it is rounded to from there, by fewer bits, is what the
// double is rounded to.  (To the nearest float, 8 of 2^23 values would come to lie in the middle between two E4M3 elements.)
__device__ __forceinline__ float to_odd(double x) {
  u32x2_t w = __builtin_bit_cast(u32x2_t, x);
  const uint32_t rest = ((w[0] & 0x1FFFFFFFu) + 0x1FFFFFFFu) & 0x20000000u;  // the float's last bit, if any below it is set
  w[0] = (w[0] & 0xE0000000u) | rest;
  return (float)__builtin_bit_cast(double, w);
}
__device__ __forceinline__ float to_odd(float x) { return x; }

template <class F>
__device__ __forceinline__ void store8(const Arr& a, int64_t row, int col, const F (&x)[8]) {
  const int64_t e = row * a.ld + col;
  if (a.f32) {
    floatx4_t* p = (floatx4_t*)((float*)a.data + e);
    p[0] = (floatx4_t){(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
    p[1] = (floatx4_t){(float)x[4], (float)x[5], (float)x[6], (float)x[7]};
  } else {
    half8_t t;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f = to_odd(x[i]);
      // As it stands: the compiler would see that the step to fp32 loses nothing that counts, leave it out, and round 64 bits to
      // FP16 by some forty instructions (8190 x 4096 of an FP16 stream into E4M3 59 us, so 76).
      if constexpr (!std::is_same_v<F, float>) asm("" : "+v"(f));
      t[i] = (_Float16)f;
    }
    *(half8_t*)((_Float16*)a.data + e) = t;
  }
}

// ---------------------------------------------------------------------------
// W waves take a row; a lane holds V runs of 8 columns of it in registers
// from the first load to the last store, so every array is read or written
// once.  Means and mean squares (of the centred values, so nothing cancels) are sums over the
// lane, the wave, and the row's waves by way of LDS.
//
// Among such calls in a graph, 8190 rows of 4096 columns take 53 us in FP16 (268 MB, 5.0 TB/s, a copy's rate), 93 us from FP16
// with a gate a row and an fp32 stream into E4M3 blocks (437 MB, 4.7); a row of 8192 with both norms 4.6 us: a launch, the
// loads, two sums' meetings.  Alone, the caches clean, 49 and 87 us; behind 256 MiB of writes, whose lines have to leave first,
// 65 and 105.  With an FP16 stream into E4M3 blocks 60 us (236 MB, 3.9): the 64 bits show there.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float mad(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double mad(double a, double b, double c) { return __builtin_fma(a, b, c); }

// 64 bits by the steps of wave_sum, in two halves.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_mov(double v) {
  const u32x2_t w = __builtin_bit_cast(u32x2_t, v);
  return __builtin_bit_cast(double, (u32x2_t){(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROW_MASK, 0xF, false),
                                              (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROW_MASK, 0xF, false)});
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_mov<0xB1, 0xF>(v);
  v += dpp_mov<0x4E, 0xF>(v);
  v += dpp_mov<0x141, 0xF>(v);
  v += dpp_mov<0x140, 0xF>(v);
  v += dpp_mov<0x142, 0xA>(v);
  v += dpp_mov<0x143, 0xC>(v);
  const u32x2_t w = __builtin_bit_cast(u32x2_t, v);
  return __builtin_bit_cast(double, (u32x2_t){(uint32_t)__builtin_amdgcn_readlane((int)w[0], 63),
                                              (uint32_t)__builtin_amdgcn_readlane((int)w[1], 63)});
}

// last: where the row's last sum lies (qnorm_sums.h).
template <int W, class F>
__device__ __forceinline__ F row_sum(F v, char* s_sum, int& last, int wave) {
  static_assert(W <= qnorm_sums::kWaves && W * (int)sizeof(F) <= qnorm_sums::kHalf, "a sum's parts lie in one half");
  v = wave_sum(v);
  if constexpr (W > 1) {
    F* at = (F*)(s_sum + (last = qnorm_sums::next(last)));
    if ((threadIdx.x & 63) == 0) at[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) v += at[i];
  }
  return v;
}

// 1 / sqrt(m).  In fp32 in two parts: what the root and the reciprocal round off is the same for the whole row.
__device__ __forceinline__ void inverse_root(float m, float& r, float& lo) {
  const float s = sqrtf(m);
  r = 1.f / s;
  const float off = __builtin_fmaf(-r, s, 1.f) - 0.5f * (r * r) * __builtin_fmaf(-s, s, m);
  lo = s > 0.f && s < INFINITY ? r * off : 0.f;
}
__device__ __forceinline__ void inverse_root(double m, double& r, double& lo) {
  r = __builtin_amdgcn_rsq(m);  // specified to 2^29 ulp, 2^-23; one Newton step leaves 1.5 times its square, 2^-45
  lo = r < INFINITY && r > 0.0 ? 0.5 * r * __builtin_fma(-m * r, r, 1.0) : 0.0;
}

// OUT: 0 FP16 rows or none, 1 E2M1, 2 E4M3, 3 fp32 rows.  From 1 on h' and its norm are formed in 64 bits: in fp32 some of
// 8190 x 4096 values, next to a border between two elements, fall on its other side, and where one is its block's largest the 31
// others take another step too.  That is 93 us of them into E4M3 (fp32: 88; everything in 64 bits, the norm of y too: 103).
template <int W, int V, bool LAYER, int OUT>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W)
k_qnorm(NormArgs a) {
  using F = std::conditional_t<OUT == 0, float, double>;
  __shared__ __align__(16) char s_sum[qnorm_sums::kBytes];
  int last = 0;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go to the eight XCDs in turn.  by_tile: the 16 rows of a tile of blocks to one, whose L2 then holds whole lines of it
  // (8190 x 4096 into E4M3 with a gate and an fp32 stream, in fp32, 88 us, otherwise 99, and 42 MB more are written).
  constexpr int R = W == 1 ? 4 : 1, B = 16 / R;  // rows of a workgroup, workgroups of a tile
  const int seq = blockIdx.x >> 3;
  const int group = (OUT == 1 || OUT == 2) && a.by_tile ? (8 * (seq / B) + (blockIdx.x & 7)) * B + seq % B : blockIdx.x;
  const int row = R * group + (W == 1 ? wave : 0);
  if (row >= a.rows) return;
  const int first = 8 * (W == 1 ? lane : (int)threadIdx.x);
  constexpr int step = 8 * 64 * W;
  float y[V][8];
  Raw8 h8[V], g8[V];
  auto norm = [&](auto& x, const Arr& weight, const Arr& bias) {
    using F = std::remove_reference_t<decltype(x[0][0])>;
    constexpr bool ahead = V <= 2;  // weights on their way while the sums are formed, where there are registers for them
    Raw8 w8[V], b8[V];
    auto weights = [&](int j, int col) {
      w8[j] = raw8(weight, 0, col);
      if (bias.data) b8[j] = raw8(bias, 0, col);
    };
    if constexpr (ahead) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (first + j * step < a.cols) weights(j, first + j * step);
    }
    const F inv_n = (F)a.inv_n;
    F mean = 0;
    if constexpr (LAYER) {
      F sum = 0;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += x[j][i];
      mean = row_sum<W>(sum, s_sum, last, wave) * inv_n;
    }
    F sq = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (LAYER) x[j][i] = first + j * step < a.cols ? x[j][i] - mean : 0;
        sq = mad(x[j][i], x[j][i], sq);
      }
    F r, lo;
    inverse_root(mad(row_sum<W>(sq, s_sum, last, wave), inv_n, (F)a.eps), r, lo);
    if constexpr (!std::is_same_v<F, float>) r += lo;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = first + j * step;
      if (col >= a.cols) continue;
      if constexpr (!ahead) weights(j, col);
      float w[8], b[8];
      of_raw8(weight, w8[j], w);
      if (bias.data) of_raw8(bias, b8[j], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const F t = std::is_same_v<F, float> ? mad(x[j][i], lo, x[j][i] * r) : x[j][i] * r;
        x[j][i] = bias.data ? mad(t, (F)w[i], (F)b[i]) : t * (F)w[i];
      }
    }
  };
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = first + j * step;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[j][i] = 0.f;
    if (col >= a.cols) continue;
    if (a.y.data) load8(a.y, row, col, y[j]);
    if (a.h.data) h8[j] = raw8(a.h, row, col);
    if (a.gate.data) g8[j] = raw8(a.gate, row, col);
  }
  if (a.post.data) norm(y, a.post, a.post_bias);
  F x[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = first + j * step;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j][i] = y[j][i];
    if (col >= a.cols) continue;
    if (a.gate.data) {
      float gt[8];
      of_raw8(a.gate, g8[j], gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] *= (F)gt[i];
    }
    if (a.h.data) {
      float h[8];
      of_raw8(a.h, h8[j], h);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = a.y.data ? mad((F)a.scale, (F)h[i], x[j][i]) : (F)a.scale * (F)h[i];
    }
    if (a.h_out.data) store8(a.h_out, row, col, x[j]);
  }
  if (!a.pre.data) return;
  norm(x, a.pre, a.pre_bias);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = first + j * step;
    if constexpr (OUT == 0 || OUT == 3) {
      if (col < a.cols) store8(a.out, row, col, x[j]);
    } else {
      // the columns up to the chunk's end are zeros
      constexpr int FMT = OUT == 1 ? kE2M1 : kE4M3;
      if (col >= 128 * a.g.chunks) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_odd(x[j][i]);
      uint32_t w[2];
      const uint32_t byte = mx_quad<FMT>(v, false, w);
      const int tile = row >> 4, r = row & 15, chunk = col >> 7, c = (col & 127) >> 3;
      uint8_t* to = (uint8_t*)a.out.data + tile * a.g.tile_bytes + (int64_t)chunk * (FMT ? 2048 : 1024);
      if constexpr (FMT == kE2M1) *(uint32_t*)(to + lane_bytes<FMT>(r, c)) = w[0];
      else *(u32x2_t*)(to + lane_bytes<FMT>(r, c)) = (u32x2_t){w[0], w[1]};
      if ((c & 3) == 0) {
        uint8_t* ex = (uint8_t*)a.out.data + a.g.exps + ((int64_t)tile * a.g.quads + (chunk >> 2)) * 256 + (chunk & 3);
        ex[4 * (16 * (c >> 2) + r)] = (uint8_t)byte;
      }
    }
  }
}

// ---- host side ----------------------------------------------------------------
template <int W, int V, bool LAYER>
hipError_t launch(const NormArgs& a, int out, hipStream_t st) {
  const int grid = a.by_tile ? (a.rows + 127) / 128 * (W == 1 ? 32 : 128) : W == 1 ? (a.rows + 3) / 4 : a.rows;
  const int threads = W == 1 ? 256 : 64 * W;
  auto go = [&](auto k) { hipLaunchKernelGGL(k, dim3(grid), dim3(threads), 0, st, a); };
  if (out == 0) go(k_qnorm<W, V, LAYER, 0>);
  else if (out == 1) go(k_qnorm<W, V, LAYER, 1>);
  else if (out == 2) go(k_qnorm<W, V, LAYER, 2>);
  else go(k_qnorm<W, V, LAYER, 3>);
  return hipGetLastError();
}
// As many waves a row as have 8 columns a lane: the shortest way through for few rows, and the fewest registers for many
// (8190 rows of 4096: 53 us in FP16 by 8 waves, 58 by 4; 256 rows of 2048: 4.8 by 4, 5.8 by 2).  Past 4096 columns of
// many rows 8 waves with 16 a lane: 8190 x 8192 with an fp32 stream 164 us, by 16 waves 177; 256 x 8192 8.8 and 8.5.
template <bool LAYER>
hipError_t by_size(const NormArgs& a, int out, hipStream_t st) {
  const int n = a.cols;
  if (n <= 512) return launch<1, 1, LAYER>(a, out, st);
  if (n <= 1024) return launch<2, 1, LAYER>(a, out, st);
  if (n <= 2048) return launch<4, 1, LAYER>(a, out, st);
  if (n <= 4096) return launch<8, 1, LAYER>(a, out, st);
  if (n <= 8192) return a.rows <= 256 ? launch<16, 1, LAYER>(a, out, st) : launch<8, 2, LAYER>(a, out, st);
  if (n <= 16384) return launch<16, 2, LAYER>(a, out, st);
  return launch<16, 4, LAYER>(a, out, st);
}

int check_array(const qnorm_rows& r, bool vector) {
  if (!r.data) return QGEMV_OK;
  if (r.type != QGEMV_F16 && r.type != QGEMV_F32) return QGEMV_ERR_UNSUPPORTED;
  if ((uintptr_t)r.data % 16 || (!vector && r.ld % 8)) return QGEMV_ERR_INVALID_ARG;
  return QGEMV_OK;
}
// An output at the place of an input: each thread then has to store where it loaded.
bool shifted(const qnorm_rows& out, const qnorm_rows& in, int rows) {
  return out.data && out.data == in.data && (out.type != in.type || (rows > 1 && out.ld != in.ld));
}
Arr array(const qnorm_rows& r) { return Arr{(char*)r.data, r.type == QGEMV_F32, r.ld}; }

}  // namespace

extern "C" int qnorm_run(const qnorm_args* p, void* stream) {
  if (!p) return QGEMV_ERR_INVALID_ARG;
  if (p->rows < 0 || p->cols < 1) return QGEMV_ERR_INVALID_ARG;
  if (p->rows > qmx_layout::kMaxRows || p->cols % 8 || p->cols > 32768) return QGEMV_ERR_UNSUPPORTED;
  if (p->kind != QNORM_RMS && p->kind != QNORM_LAYER) return QGEMV_ERR_UNSUPPORTED;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->scale)) return QGEMV_ERR_INVALID_ARG;
  if (p->rows == 0) return QGEMV_OK;
  const bool has_y = p->y.data, has_pre = p->pre.data, blocks = p->out.type == QNORM_OUT_E2M1 || p->out.type == QNORM_OUT_E4M3;
  if ((!has_y && !p->h.data) || (!has_y && (p->gate.data || p->post.data))) return QGEMV_ERR_INVALID_ARG;
  if ((p->post_bias.data && !p->post.data) || (p->pre_bias.data && !has_pre)) return QGEMV_ERR_INVALID_ARG;
  if (has_pre != (p->out.data != nullptr) || (!p->out.data && !p->h_out.data)) return QGEMV_ERR_INVALID_ARG;
  // by_size has a thread for 8 columns of the next power of two, 512 at least, rows in tiles of 16 on eight XCDs: 2^32 are past a launch
  if (((int64_t)p->rows + 127 & ~127ll) << (p->cols <= 512 ? 9 : 32 - __builtin_clz(p->cols - 1)) >= 1ll << 35) return QGEMV_ERR_UNSUPPORTED;
  int st;
  for (const qnorm_rows* r : {&p->y, &p->h, &p->gate, &p->h_out})
    if ((st = check_array(*r, false))) return st;
  for (const qnorm_rows* r : {&p->post, &p->post_bias, &p->pre, &p->pre_bias})
    if ((st = check_array(*r, true))) return st;
  if (p->rows > 1 && p->h_out.data && p->h_out.ld < p->cols) return QGEMV_ERR_INVALID_ARG;
  NormArgs a{};
  int out = 0;
  if (has_pre && blocks) {
    if ((uintptr_t)p->out.data % 256) return QGEMV_ERR_INVALID_ARG;
    const qmx_shape s = {p->rows, p->cols, p->out.type - QNORM_OUT_E2M1};
    size_t n;
    if ((st = qmx_bytes(&s, &n))) return st;
    a.g = qmx_layout::geo(s.rows, s.cols, s.format);
    out = 1 + s.format;
  } else if (has_pre) {
    if ((st = check_array(p->out, false))) return st;
    if (p->rows > 1 && p->out.ld < p->cols) return QGEMV_ERR_INVALID_ARG;
    if (p->out.type == QGEMV_F32) out = 3;
  }
  if (p->out.data && p->out.data == p->h_out.data) return QGEMV_ERR_INVALID_ARG;
  for (const qnorm_rows* r : {&p->h_out, &p->out})
    if (shifted(*r, p->y, p->rows) || shifted(*r, p->h, p->rows)) return QGEMV_ERR_INVALID_ARG;
  a.y = array(p->y), a.h = array(p->h), a.gate = array(p->gate), a.h_out = array(p->h_out), a.out = array(p->out);
  a.post = array(p->post), a.post_bias = array(p->post_bias), a.pre = array(p->pre), a.pre_bias = array(p->pre_bias);
  a.rows = p->rows, a.cols = p->cols, a.eps = p->eps, a.scale = p->scale;
  a.inv_n = 1.0 / p->cols;
  a.by_tile = (out == 1 || out == 2) && p->rows >= 512;  // fewer would fill the XCDs unevenly
  const hipError_t e = p->kind == QNORM_LAYER ? by_size<true>(a, out, (hipStream_t)stream)
                                              : by_size<false>(a, out, (hipStream_t)stream);
  if (e == hipSuccess) return QGEMV_OK;
  qgemv_set_hip_error((int)e);
  return QGEMV_ERR_HIP;
}
