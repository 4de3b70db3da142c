// qrotary_kernels.hip -- queries and keys turned by their position, keys and
// values into the 4-bit cache (include/qrotary.h; writing's parts in qcache_dev.h).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/qrotary.h"
#include "qcache_dev.h"

namespace {

typedef double doublex2_t __attribute__((ext_vector_type(2)));

struct Turn {
  const double* freqs;
  const int32_t* pair_axis;
  const int32_t* positions;
  int pairs, axes, n_tok, halves;
};

// ---------------------------------------------------------------------------
// A workgroup of four waves takes one unit (16 positions of a sequence) and some
// of its heads.  It first forms the unit's sines and cosines in LDS, which all
// heads share; then its waves take the heads' keys, values and queries in turn.
//
// The angle p f is formed in 64 bits and reduced exactly: t = p f / 2 pi in two
// parts, less its nearest integer.  Turning in 64 bits as well costs nothing
// that shows (an FP64 multiply-add issues at the rate of an FP32 one, and the call is
// bound by HBM), and makes the FP16 key, and with it the 4-bit code, that
// of the exact turn: in fp32 one FP16 in some 10^4 would fall on the other side of
// a rounding border, and with it, where it is a group's end, the group's step.
// ---------------------------------------------------------------------------
constexpr int kTable = 16;  // tokens of a unit

// Pair i of token t: 16 bytes at (t * pairs + place(i)); 8 neighbouring pairs, which a lane takes, lie pairs / 8 apart, so
// that neighbouring lanes read neighbouring 16 bytes.
__device__ __forceinline__ int place(int i, int pairs) { return (i & 7) * (pairs >> 3) + (i >> 3); }

__device__ __forceinline__ doublex2_t cos_sin(int pos, double f) {
  constexpr double k1 = 0.15915494309189535, k2 = -9.8393384282593e-18;  // 1 / 2 pi
  const double a = (double)pos * f;
  const double t = a * k1;
  const double lo = __builtin_fma(a, k1, -t) + a * k2;
  const double r = (t - __builtin_rint(t)) + lo;
  double s, c;
  sincospi(2.0 * r, &s, &c);
  return (doublex2_t){c, s};
}

__device__ __forceinline__ void load_run(const Rows& r, int64_t e, float (&v)[8]) {
  if (r.f32) {
    const floatx4_t* p = (const floatx4_t*)((const float*)r.data + e);
    const floatx4_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const half8_t a = *(const half8_t*)((const _Float16*)r.data + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
  }
}
__device__ __forceinline__ void store_run(const Rows& r, int64_t e, const float (&v)[8]) {
  if (r.f32) {
    floatx4_t* p = (floatx4_t*)((float*)r.data + e);
    p[0] = (floatx4_t){v[0], v[1], v[2], v[3]};
    p[1] = (floatx4_t){v[4], v[5], v[6], v[7]};
  } else {
    half8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    *(half8_t*)((_Float16*)r.data + e) = h;
  }
}

__device__ __forceinline__ void turn(float& a, float& b, doublex2_t cs) {
  const double x = a, y = b;
  a = (float)__builtin_fma(x, cs[0], -(y * cs[1]));
  b = (float)__builtin_fma(y, cs[0], x * cs[1]);
}

// Run r (8 dimensions) of the vector at element e, turned.  tab: the token's pairs.
__device__ __forceinline__ void turned_run(const Rows& src, int64_t e, int r, const Turn& tn, const doublex2_t* tab,
                                           float (&v)[8]) {
  load_run(src, e + 8 * r, v);
  const int runs = tn.pairs >> 2;  // of the turned dimensions
  if (r >= runs) return;
  if (tn.halves) {
    const bool second = r >= runs / 2;
    const int first = second ? r - runs / 2 : r;
    float o[8];
    load_run(src, e + 8 * (second ? first : r + runs / 2), o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a = second ? o[i] : v[i], b = second ? v[i] : o[i];
      turn(a, b, tab[i * (tn.pairs >> 3) + first]);
      v[i] = second ? b : a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(v[2 * i], v[2 * i + 1], tab[place(4 * r + i, tn.pairs)]);
  }
}

template <int D, int NG>
__global__ void __launch_bounds__(256)
k_qrotary_write(uint8_t* __restrict__ cache, Seqs sq, Turn tn, Rows q, Rows qo, Rows k, Rows v, int heads, int q_heads,
                int split) {
  using L = Geo<D, NG>;
  extern __shared__ doublex2_t s_tab[];
  const int idx = blockIdx.x / split, part = blockIdx.x - idx * split;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const UnitTask x = unit_task(sq, idx);
  if (x.s < 0) return;
  const int t0 = max(x.p0 - 16 * x.u, 0), t1 = min(x.p0 + x.n - 16 * x.u, 16);  // the unit's tokens
  const int row0 = x.row + 16 * x.u - x.p0;                                     // row of token 0
  for (int i = threadIdx.x; i < (t1 - t0) * tn.pairs; i += 256) {
    const int t = t0 + i / tn.pairs, pair = i % tn.pairs;
    const int axis = tn.pair_axis ? tn.pair_axis[pair] : 0;
    doublex2_t cs = {1.0, 0.0};
    if ((uint32_t)axis < (uint32_t)tn.axes) {
      const int pos = tn.positions ? tn.positions[(int64_t)axis * tn.n_tok + row0 + t] : 16 * x.u + t;
      cs = cos_sin(pos, tn.freqs[pair]);
    }
    s_tab[t * tn.pairs + place(pair, tn.pairs)] = cs;
  }
  __syncthreads();
  const int p = sq.page(x.s, x.u);
  if (p >= 0) {
    const int h0 = (int)((int64_t)heads * part / split), h1 = (int)((int64_t)heads * (part + 1) / split);
    for (int i = 2 * h0 + w; i < 2 * h1; i += 4) {
      const int h = i >> 1;
      uint8_t* unit = cache + unit_at(p, x.u, h, heads, sq.up_shift, L::bytes);
      if (i & 1) {
        write_values<D, NG>(unit, v, x, h, lane);
        continue;
      }
      const int t = lane & 15, kq = lane >> 4;
      const bool on = t >= t0 && t < t1;
      uint32_t pk[4 * L::ND];
#pragma unroll
      for (int j = 0; j < L::ND; ++j) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.f;
        if (on) turned_run(k, (int64_t)(row0 + t) * k.ts + (int64_t)h * k.hs, 4 * j + kq, tn, s_tab + t * tn.pairs, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) pk[4 * j + e] = pk_h(y[2 * e], y[2 * e + 1]);
      }
      store_keys<D, NG>(unit, pk, on, lane);
    }
  }
  // Queries: a lane takes two runs of a head, the two that turn together or two neighbours.
  constexpr int SL = D / 16, VW = 64 / SL;  // lanes of a head, heads of a wave
  const int q0 = (int)((int64_t)q_heads * part / split), q1 = (int)((int64_t)q_heads * (part + 1) / split);
  const int groups = (q1 - q0 + VW - 1) / VW;
  const int slot = lane % SL;
  const int runs = tn.pairs >> 2;
  const bool joint = tn.halves && slot < runs / 2;
  const int r0 = joint ? slot : 2 * slot, r1 = joint ? slot + runs / 2 : 2 * slot + 1;
  for (int i = w; i < (t1 - t0) * groups; i += 4) {
    const int t = t0 + i / groups, h = q0 + (i % groups) * VW + lane / SL;
    if (h >= q1) continue;
    const doublex2_t* tab = s_tab + t * tn.pairs;
    const int64_t e = (int64_t)(row0 + t) * q.ts + (int64_t)h * q.hs;
    const int64_t eo = (int64_t)(row0 + t) * qo.ts + (int64_t)h * qo.hs;
    float a[8], b[8];
    load_run(q, e + 8 * r0, a);
    load_run(q, e + 8 * r1, b);
    if (joint) {
#pragma unroll
      for (int j = 0; j < 8; ++j) turn(a[j], b[j], tab[j * (tn.pairs >> 3) + slot]);
    } else if (!tn.halves && r0 < runs) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        turn(a[2 * j], a[2 * j + 1], tab[place(4 * r0 + j, tn.pairs)]);
        turn(b[2 * j], b[2 * j + 1], tab[place(4 * r1 + j, tn.pairs)]);
      }
    }
    store_run(qo, eo + 8 * r0, a);
    store_run(qo, eo + 8 * r1, b);
  }
}

// ---- host side ----------------------------------------------------------------
int check_turn(const qcache_shape* sh, const qrotary* r) {
  if (!r) return QGEMV_ERR_INVALID_ARG;
  if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > sh->head_dim) return QGEMV_ERR_UNSUPPORTED;
  if (r->style != QROTARY_HALVES && r->style != QROTARY_NEIGHBOURS) return QGEMV_ERR_UNSUPPORTED;
  if (r->axes < 1 || r->axes > 16) return QGEMV_ERR_UNSUPPORTED;
  if (!r->freqs || (uintptr_t)r->freqs % 8 || (uintptr_t)r->pair_axis % 4 || (uintptr_t)r->positions % 4)
    return QGEMV_ERR_INVALID_ARG;
  if (!r->positions && r->axes > 1) return QGEMV_ERR_INVALID_ARG;
  return QGEMV_OK;
}

struct Launch {
  uint8_t* cache;
  Seqs sq;
  Turn tn;
  Rows q, qo, k, v;
  int heads, q_heads, split;
};
template <int D, int NG>
hipError_t launch(Dims<D, NG>, const Launch& a, uint32_t grid, hipStream_t st) {
  hipLaunchKernelGGL((k_qrotary_write<D, NG>), dim3(grid), dim3(256), (size_t)kTable * a.tn.pairs * 16, st, a.cache, a.sq, a.tn,
                     a.q, a.qo, a.k, a.v, a.heads, a.q_heads, a.split);
  return hipGetLastError();
}

}  // namespace

extern "C" {

int qrotary_write(const qcache_shape* shape, void* cache, const qcache_seqs* seqs, const qrotary* rotary,
                  int32_t n_q_heads, const qcache_rows* q, const qcache_rows* q_out, const qcache_rows* k,
                  const qcache_rows* v, void* stream) {
  int st = check_copy(shape, cache, seqs, k, v);
  if (st) return st;
  if ((st = check_turn(shape, rotary))) return st;
  if (n_q_heads < 0) return QGEMV_ERR_INVALID_ARG;
  if (n_q_heads > 65535) return QGEMV_ERR_UNSUPPORTED;
  if (seqs->n_seq == 0 || seqs->n_tok == 0) return QGEMV_OK;
  Rows qr{}, qo{};
  if (n_q_heads > 0) {
    if ((st = check_rows(q)) || (st = check_rows(q_out))) return st;
    qr = device_rows(q);
    qo = device_rows(q_out);
    if ((seqs->n_tok > 1 && qo.ts < shape->head_dim) || (n_q_heads > 1 && qo.hs < shape->head_dim))
      return QGEMV_ERR_INVALID_ARG;
  }
  const Seqs sq = device_seqs(shape, seqs);
  const Turn tn = {rotary->freqs, rotary->pair_axis, rotary->positions, rotary->rot_dim / 2, rotary->axes, seqs->n_tok,
                   rotary->style == QROTARY_HALVES};
  const int64_t units = seqs->q_start ? (int64_t)seqs->n_tok / 16 + 2 * (int64_t)seqs->n_seq : seqs->n_seq;
  // few units: their heads are dealt out to more workgroups, each of which forms the sines for itself
  const int most = shape->n_heads > n_q_heads ? shape->n_heads : n_q_heads;
  int64_t split = units >= 1024 ? 1 : (1024 + units - 1) / units;
  if (split > most) split = most;
  if (units * split * 256 > 0xFFFFFFFFll) return QGEMV_ERR_UNSUPPORTED;
  const Launch go = {(uint8_t*)cache, sq, tn, qr, qo, device_rows(k), device_rows(v), shape->n_heads, n_q_heads, (int)split};
  const uint32_t grid = (uint32_t)(units * split);
  return hip_status(by_shape(shape, [&](auto d) { return launch(d, go, grid, (hipStream_t)stream); }));
}

}  // extern "C"
