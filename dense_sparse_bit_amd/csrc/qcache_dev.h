// qcache_dev.h -- what the cache's kernels share: the batch of a call, units of
// 16 positions, quantising them into the cache, and the checks of the arguments
// (include/qcache.h; storage in qcache_layout.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/qcache.h"
#include "qcache_layout.h"
#include "qgemv_decode.h"
#include "qgemv_internal.h"

using namespace qcache_layout;
using namespace qgemv_dev;

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ floatx4_t mfma(u32x4_t a, u32x4_t b, floatx4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                0, 0);
}
__device__ __forceinline__ float h2f(uint16_t h) { return (float)__builtin_bit_cast(_Float16, h); }
__device__ __forceinline__ uint16_t f2h(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
__device__ __forceinline__ bool not_finite(uint16_t h) { return (h & 0x7C00u) == 0x7C00u; }

// The batch of a call, by value (see include/qcache.h).
struct Seqs {
  const int32_t* q_start;
  const int32_t* lens;
  const int32_t* pages;
  int n_seq, n_tok, max_pages, n_pages;
  int up_shift;  // log2 of units per page
  int cap;       // positions a table row covers

  __device__ __forceinline__ int start(int s) const {
    return q_start ? min(max(q_start[s], 0), n_tok) : s;
  }
  // Page of unit u (of 16 positions) of sequence s, or -1.
  __device__ __forceinline__ int page(int s, int u) const {
    const int i = u >> up_shift;
    if (u < 0 || i >= max_pages) return -1;
    const int p = pages[(int64_t)s * max_pages + i];
    return (uint32_t)p < (uint32_t)n_pages ? p : -1;
  }
};

// Byte offset of unit u of a sequence, on page p, of head h.
__device__ __forceinline__ int64_t unit_at(int p, int u, int h, int heads, int up_shift, int unit) {
  return ((((int64_t)p * heads + h) << up_shift) + (u & ((1 << up_shift) - 1))) * unit;
}

struct Rows {
  char* data;
  int64_t ts, hs;  // element strides
  int f32;
};

// A register that another lane is about to read (a lane swap, DPP) has to have been written two instructions before.
// The compiler sees to that after its own instructions, but it does not look into inline asm (pk_min below).
__device__ __forceinline__ uint32_t settled(uint32_t v) {
  asm("s_nop 1" : "+v"(v));
  return v;
}

// Lanes i ^ 16, then i ^ 32: each swap leaves the two partners' values in its two results.
template <class Op>
__device__ __forceinline__ uint32_t over_column(uint32_t v, Op op) {  // the four lanes of a column
  v = settled(v);
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = settled(op(a[0], a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return op(b[0], b[1]);
}
__device__ __forceinline__ float column_max(float v) {
  return __uint_as_float(over_column(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
  }));
}
__device__ __forceinline__ float column_sum(float v) {
  return __uint_as_float(over_column(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
  }));
}

typedef float floatx2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_h(float a, float b) {  // round to nearest even
  return as_u32(__builtin_convertvector((floatx2_t){a, b}, half2_t));
}
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }  // 1 ulp; results below 2^-126 are 0

// x / d for 0 <= x < 2^31 as a multiplication: M = 2^(31 + sh) / d + 1, 2^(sh - 1) < d <= 2^sh.
struct Divisor {
  uint32_t d, mul, sh;
  __device__ __forceinline__ int of(int x) const {
    return d == 1 ? x : (int)(__umulhi((uint32_t)x, mul) >> (sh - 1));
  }
};
inline Divisor divisor(int d) {
  uint32_t sh = 0;
  while ((1u << sh) < (uint32_t)d) ++sh;
  return Divisor{(uint32_t)d, (uint32_t)((((uint64_t)1 << (31 + sh)) / (uint32_t)d) + 1), sh};
}

// ---------------------------------------------------------------------------
// Writing and reading back.
//
// A wave takes the keys, or the values, of one unit (16 positions of one
// head), and a lane holds of them what it holds in the attention's operands:
// of the keys one token and D/32 runs of 8 dimensions, of the values D/16
// dimensions of four tokens.  So a unit's codes are one contiguous 16 bytes
// a lane (head_dim 128), and rows of FP16 or fp32 are read and written in runs
// of 16 bytes or more.
//
// Long calls are bound by HBM, at a copy's rate (4.8 TB/s) or above: 65536 tokens
// of 8 heads x 128 take 70 us to write from FP16 (352 MB), 119 us from fp32
// (621 MB), and 52 and 96 us to read.  Writing sits close to the VALU as well:
// with fp32 divisions (22 instructions a value; some 11 now) it took 112 us.
// A step of 16 tokens of 32 heads takes 3.4 us either way, a launch.
//
// Waves are numbered without knowing the lengths: sequence s owns the numbers
// from (its first row / 16) + 2 s on, which leaves room for a unit at either end
// that its rows only partly fill.
// ---------------------------------------------------------------------------
struct UnitTask {
  int s, u;        // sequence (-1: none) and unit (may be negative)
  int row, n, p0;  // rows [row, row + n) stand at positions p0 ..
};
__device__ __forceinline__ UnitTask unit_task(const Seqs& sq, int idx) {
  UnitTask x;
  x.s = -1;
  if (!sq.q_start) {
    if (idx >= sq.n_seq) return x;
    x.s = x.row = idx;
    x.n = 1;
    x.p0 = max(sq.lens[idx], 0) - 1;
    x.u = x.p0 >> 4;
    return x;
  }
  // the last s whose first number is at most idx, 64 probes at a time
  auto number = [&](int s) { return (sq.start(s) >> 4) + 2 * s; };
  const int lane = threadIdx.x & 63;
  int lo = 0;
  for (int cnt = sq.n_seq; cnt > 1;) {
    const int step = (cnt + 63) >> 6, s = lo + lane * step;
    const int c = __builtin_popcountll(__ballot(s < lo + cnt && number(s) <= idx));
    const int skip = max(c - 1, 0) * step;
    lo += skip;
    cnt = min(step, cnt - skip);
  }
  x.row = sq.start(lo);
  x.n = sq.start(lo + 1) - x.row;
  if (x.n <= 0) return x;
  x.p0 = max(sq.lens[lo], 0) - x.n;
  x.u = (x.p0 >> 4) + idx - number(lo);
  if (16 * x.u >= x.p0 + x.n) return x;
  x.s = lo;
  return x;
}
// Workgroups of two units each.  T: Seqs or qcache_seqs.
template <class T>
inline int64_t unit_workgroups(const T& sq, int heads) {
  const int64_t waves = sq.q_start ? (int64_t)sq.n_tok / 16 + 2 * (int64_t)sq.n_seq : sq.n_seq;
  return (waves + 1) / 2 * heads;
}

// N consecutive elements (a multiple of 4) as FP16 pairs.  Rows are read once, past the L2's own keeping (65536 tokens
// written and read, the inputs from HBM: 241 -> 217 us).
template <int N>
__device__ __forceinline__ void load_pairs(const Rows& r, int64_t e, uint32_t* h) {
  if (r.f32) {
    const floatx4_t* p = (const floatx4_t*)((const float*)r.data + e);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const floatx4_t x = __builtin_nontemporal_load(p + i);
      h[2 * i] = pk_h(x[0], x[1]);
      h[2 * i + 1] = pk_h(x[2], x[3]);
    }
  } else if constexpr (N % 8 == 0) {
    const u32x4_t* p = (const u32x4_t*)((const _Float16*)r.data + e);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const u32x4_t x = __builtin_nontemporal_load(p + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[4 * i + k] = x[k];
    }
  } else {
    const u32x2_t x = *(const u32x2_t*)((const _Float16*)r.data + e);
    h[0] = x[0], h[1] = x[1];
  }
}
// Outputs are stored 16 bytes a lane, lanes side by side, so that 128 or more bytes of a row leave together: only then
// may they pass the L2 by: 65536 tokens are read in 52 us instead of 84 in FP16, in 96 instead of 151 in fp32 (pieces of
// 64 bytes: 60 and 130; of 16 bytes: 225 in fp32).
__device__ __forceinline__ void stream_out(char* to, u32x4_t x) { __builtin_nontemporal_store(x, (u32x4_t*)to); }

// The lane's two quads 2 kq, 2 kq + 1 of the 8 that the lanes of a column hold become quads kq and 4 + kq.
__device__ __forceinline__ void by_column(u32x4_t& x, u32x4_t& y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto a = __builtin_amdgcn_permlane16_swap(x[i], y[i], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(a[0], a[1], false, false);
    x[i] = b[0], y[i] = b[1];
  }
}

// Two neighbouring lanes hold y and z of a token each; then y of both is the first token's and z the second's, in the
// even lane what was y and in the odd lane what was z.
__device__ __forceinline__ void by_pair(u32x4_t& y, u32x4_t& z, bool odd) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t mine = odd ? y[i] : z[i];
    const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp((int)mine, (int)mine, 0xB1, 0xF, 0xF, false);  // i ^ 1
    if (odd) y[i] = other;
    else z[i] = other;
  }
}

// The lane's quads Q m .. + Q - 1 of the 16 Q that 16 neighbouring lanes hold are stored at `row`, by way of LDS.
template <int Q>
__device__ __forceinline__ void store_row(char* row, u32x4_t (&x)[Q], int lane, u32x4_t* lds, bool on) {
  const int m = lane & 15;
  if constexpr (Q > 1) {
    u32x4_t* mine = lds + (lane >> 4) * (16 * Q);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < Q; ++i) mine[Q * m + i] = x[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < Q; ++i) x[i] = mine[16 * i + m];
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < Q; ++i) stream_out(row + 16 * (16 * i + m), x[i]);
}

// Minimum and maximum of FP16 pairs, written out: the compiler's own quieten their operands first, which doubles them.
__device__ __forceinline__ uint32_t pk_min(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("v_pk_min_f16 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("v_pk_max_f16 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}
// (min of the low halves, min of the negated high halves)
__device__ __forceinline__ uint32_t pk_min_neg(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("v_pk_min_f16 %0, %1, %2 neg_hi:[1,1]" : "=v"(d) : "v"(a), "v"(b));
  return d;
}
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("v_pk_max_u16 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}

// Of FP16 pairs: (smallest, -largest), and the largest |bits| of either half.  0x7C00 and more are not finite; the
// minimum passes a NaN by.
struct Extent {
  uint32_t ends, top;
};
template <int N>
__device__ __forceinline__ Extent extent(const uint32_t* h) {
  uint32_t lo = h[0], hi = h[0], top = h[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < N; ++i) {
    lo = pk_min(lo, h[i]);
    hi = pk_max(hi, h[i]);
    top = pk_max_u16(top, h[i] & 0x7FFF7FFFu);
  }
  return Extent{pk_min_neg(perm(hi, lo, 0x05040100u), perm(hi, lo, 0x07060302u)), top};
}
__device__ __forceinline__ bool bad_top(uint32_t t) { return (t & 0xFFFFu) >= 0x7C00u || t >= 0x7C000000u; }

// What a group's codes are formed with.  A quotient a / b is formed as q0 = a y, q0 + (a - q0 b) y, with y = 1 / b to
// about an ulp: a - q0 b is exact, so the sum is within 2^-45 of a / b before its one rounding, and a / b, a of 24 bits
// over b of 11 (s) or 4 (15), is no nearer than 2^-36 to a rounding border without lying on it: it is fp32(a / b).
struct Step {
  float lo, s, inv;
  uint16_t s16, lo16;
};
__device__ __forceinline__ float quotient(float a, float b, float y) {
  const float q0 = a * y;
  return __builtin_fmaf(__builtin_fmaf(-q0, b, a), y, q0);
}
__device__ __forceinline__ Step make_step(uint32_t ends, bool bad) {
  Step t;
  t.lo16 = (uint16_t)ends;
  t.lo = h2f(t.lo16);
  uint16_t s = f2h(quotient(-h2f((uint16_t)(ends >> 16)) - t.lo, 15.f, 1.f / 15.f));
  if (__builtin_fmaf(15.f, h2f(s), t.lo) > 65504.f) --s;  // the FP16 below (s > 0 here)
  t.s = h2f(s);
  const float y = __builtin_amdgcn_rcpf(t.s);  // 1 ulp; s is 2^-24 or more, or 0
  t.inv = s == 0 || bad ? 0.f : __builtin_fmaf(__builtin_fmaf(-t.s, y, 1.f), y, y);
  t.s16 = bad ? (uint16_t)0x7E00u : s;
  if (bad) t.lo16 = 0;
  return t;
}
// min(rint(fp32((v - lo) / s)), 15) in the low bits of a float's bits: adding 1.5 2^23 rounds to an integer, to even.
__device__ __forceinline__ uint32_t code(const Step& t, uint16_t h) {
  const float q = quotient(__builtin_fmaf(h2f(h), 1.f, -t.lo), t.s, t.inv);
  return __float_as_uint(fminf(q, 15.f) + 12582912.f);
}
// The low 16 bits are a + 16 b + 256 c + 4096 d; the upper are not used.
__device__ __forceinline__ uint32_t nibbles(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return (((((d << 4) + c) << 4) + b) << 4) + a;
}
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return perm(b, a, 0x05040100u); }

// Quantises and stores a unit's keys: v holds, as FP16 pairs, the lane's runs of its token (zeros where it is not on).
template <int D, int NG>
__device__ __forceinline__ void store_keys(uint8_t* unit, const uint32_t (&v)[4 * Geo<D, NG>::ND], bool on, int lane) {
  using L = Geo<D, NG>;
  constexpr int R = L::G / 32;  // runs of a group
  const int t = lane & 15, kq = lane >> 4;
  Extent m[NG];
  uint32_t top = 0;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    m[g] = extent<4 * R>(v + 4 * R * g);
    m[g].ends = over_column(m[g].ends, pk_min);
    top = pk_max_u16(top, m[g].top);
  }
  const bool some_bad = __ballot(bad_top(top)) != 0;
  uint32_t w[L::ND];
  uint16_t ks[NG], kl[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const Step st = make_step(m[g].ends, some_bad && bad_top(over_column(m[g].top, pk_max_u16)));
    ks[g] = st.s16;
    kl[g] = st.lo16;
#pragma unroll
    for (int j = g * R; j < (g + 1) * R; ++j) {  // nibble i + 4 e: dimension 2 i + e of the run
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = code(st, (uint16_t)(v[4 * j + i / 2] >> (16 * (i & 1))));
      w[j] = low_halves(nibbles(c[0], c[2], c[4], c[6]), nibbles(c[1], c[3], c[5], c[7]));
    }
  }
  if (!on) return;
  uint32_t* to = (uint32_t*)unit + lane * L::ND;
  if constexpr (L::ND == 2) {
    *(u32x2_t*)to = (u32x2_t){w[0], w[1]};
  } else {
#pragma unroll
    for (int j = 0; j < L::ND; j += 4) *(u32x4_t*)(to + j) = (u32x4_t){w[j], w[j + 1], w[j + 2], w[j + 3]};
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
    if ((g & 3) == kq) {
      ((uint16_t*)(unit + L::off_ks))[((t >> 2) * NG + g) * 4 + (t & 3)] = ks[g];
      ((uint16_t*)(unit + L::off_kl))[t * NG + g] = kl[g];
    }
}

template <int D, int NG>
__device__ __forceinline__ void write_keys(uint8_t* unit, const Rows& k, const UnitTask& x, int h, int lane) {
  using L = Geo<D, NG>;
  const int kq = lane >> 4, pos = 16 * x.u + (lane & 15);
  const bool on = pos >= x.p0 && pos < x.p0 + x.n;
  uint32_t v[4 * L::ND];
#pragma unroll
  for (int i = 0; i < 4 * L::ND; ++i) v[i] = 0;
  if (on) {
    const int64_t e = (int64_t)(x.row + pos - x.p0) * k.ts + (int64_t)h * k.hs + 8 * kq;
#pragma unroll
    for (int j = 0; j < L::ND; ++j) load_pairs<8>(k, e + 32 * j, v + 4 * j);
  }
  store_keys<D, NG>(unit, v, on, lane);
}

// Over the 2, 4, 8 or 16 neighbouring lanes of a group.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  v = settled(v);
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}
template <int N, class Op>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, Op op) {
  v = op(v, dpp_u32<0xB1>(v));                       // i ^ 1
  if constexpr (N > 2) v = op(v, dpp_u32<0x4E>(v));   // i ^ 2
  if constexpr (N > 4) v = op(v, dpp_u32<0x141>(v));  // the other four of eight
  if constexpr (N > 8) v = op(v, dpp_u32<0x140>(v));  // the other eight of sixteen
  return v;
}

template <int D, int NG>
__device__ __forceinline__ void write_values(uint8_t* unit, const Rows& v, const UnitTask& x, int h, int lane) {
  using L = Geo<D, NG>;
  constexpr int DL = D / 16, N = L::G / DL;  // dimensions of a lane, lanes of a group
  const int m = lane & 15, kq = lane >> 4;
  uint32_t r[4][DL / 2];
  bool on[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = 16 * x.u + 4 * kq + i;
    on[i] = pos >= x.p0 && pos < x.p0 + x.n;
#pragma unroll
    for (int j = 0; j < DL / 2; ++j) r[i][j] = 0;
    if (on[i]) load_pairs<DL>(v, (int64_t)(x.row + pos - x.p0) * v.ts + (int64_t)h * v.hs + DL * m, r[i]);
  }
  Extent e[4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = extent<DL / 2>(r[i]);
    e[i].ends = over_lanes<N>(e[i].ends, pk_min);
    top = pk_max_u16(top, e[i].top);
  }
  const bool some_bad = __ballot(bad_top(top)) != 0;
  uint32_t half[4][L::NC];  // of token i: in the low 16 bits, its dimensions 4 c .. 4 c + 3
  uint16_t vs[4], vl[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Step st = make_step(e[i].ends, some_bad && bad_top(over_lanes<N>(e[i].top, pk_max_u16)));
    vs[i] = st.s16;
    vl[i] = st.lo16;
#pragma unroll
    for (int c = 0; c < L::NC; ++c) {
      uint32_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = code(st, (uint16_t)(r[i][2 * c + k / 2] >> (16 * (k & 1))));
      half[i][c] = nibbles(q[0], q[1], q[2], q[3]);
    }
  }
  uint32_t* to = (uint32_t*)(unit + L::off_v) + lane * L::ND;
  uint16_t* stats = (uint16_t*)(unit + L::off_vs) + (kq * NG + m / N) * 8;
  const bool first = m % N == 0;
  if (on[0] && on[1] && on[2] && on[3]) {
    uint32_t w[L::ND];
#pragma unroll
    for (int tp = 0; tp < 2; ++tp)
#pragma unroll
      for (int c = 0; c < L::NC; ++c) w[tp * L::NC + c] = low_halves(half[2 * tp][c], half[2 * tp + 1][c]);
    if constexpr (L::ND == 2) {
      *(u32x2_t*)to = (u32x2_t){w[0], w[1]};
    } else {
#pragma unroll
      for (int j = 0; j < L::ND; j += 4) *(u32x4_t*)(to + j) = (u32x4_t){w[j], w[j + 1], w[j + 2], w[j + 3]};
    }
    if (first) {
      auto two = [](uint16_t a, uint16_t b) { return (uint32_t)a | ((uint32_t)b << 16); };
      *(u32x4_t*)stats = (u32x4_t){two(vs[0], vs[1]), two(vs[2], vs[3]), two(vl[0], vl[1]), two(vl[2], vl[3])};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!on[i]) continue;
#pragma unroll
    for (int c = 0; c < L::NC; ++c) ((uint16_t*)to)[2 * ((i >> 1) * L::NC + c) + (i & 1)] = (uint16_t)half[i][c];
    if (first) {
      stats[i] = vs[i];
      stats[4 + i] = vl[i];
    }
  }
}

// ---- host side ----------------------------------------------------------------
int hip_status(hipError_t e) {
  if (e == hipSuccess) return QGEMV_OK;
  qgemv_set_hip_error((int)e);
  return QGEMV_ERR_HIP;
}

int check_shape(const qcache_shape* sh) {
  if (!sh) return QGEMV_ERR_INVALID_ARG;
  if (sh->n_pages < 1 || sh->n_heads < 1) return QGEMV_ERR_INVALID_ARG;
  if (sh->n_heads > 65535) return QGEMV_ERR_UNSUPPORTED;
  if (sh->head_dim != 64 && sh->head_dim != 128 && sh->head_dim != 256) return QGEMV_ERR_UNSUPPORTED;
  if (sh->page_size < 16 || sh->page_size > 1024 || (sh->page_size & (sh->page_size - 1))) return QGEMV_ERR_UNSUPPORTED;
  if ((sh->group != 32 && sh->group != 64 && sh->group != 128) || sh->group > sh->head_dim) return QGEMV_ERR_UNSUPPORTED;
  return QGEMV_OK;
}

int check_counts(const qcache_shape* sh, const qcache_seqs* sq) {
  if (!sq || sq->n_seq < 0 || sq->n_tok < 0 || sq->max_pages < 0) return QGEMV_ERR_INVALID_ARG;
  if (sq->n_seq > 1 << 28) return QGEMV_ERR_UNSUPPORTED;
  if ((int64_t)sq->max_pages * sh->page_size > 0x7FFFFFFF - 1024) return QGEMV_ERR_UNSUPPORTED;
  return QGEMV_OK;
}

int check_seqs(const qcache_shape* sh, const qcache_seqs* sq) {
  const int st = check_counts(sh, sq);
  if (st) return st;
  if (sq->n_seq == 0 || sq->n_tok == 0) return QGEMV_OK;
  if (!sq->lens || (!sq->pages && sq->max_pages > 0)) return QGEMV_ERR_INVALID_ARG;
  if (!sq->q_start && sq->n_tok != sq->n_seq) return QGEMV_ERR_INVALID_ARG;
  if ((uintptr_t)sq->q_start % 4 || (uintptr_t)sq->lens % 4 || (uintptr_t)sq->pages % 4) return QGEMV_ERR_INVALID_ARG;
  return QGEMV_OK;
}

int check_rows(const qcache_rows* r) {
  if (!r || !r->data || (uintptr_t)r->data % 16) return QGEMV_ERR_INVALID_ARG;
  if (r->type != QGEMV_F16 && r->type != QGEMV_F32) return QGEMV_ERR_UNSUPPORTED;
  if (r->tok_stride % 8 || r->head_stride % 8) return QGEMV_ERR_INVALID_ARG;
  return QGEMV_OK;
}

Seqs device_seqs(const qcache_shape* sh, const qcache_seqs* sq) {
  Seqs d;
  d.q_start = sq->q_start;
  d.lens = sq->lens;
  d.pages = sq->pages;
  d.n_seq = sq->n_seq;
  d.n_tok = sq->n_tok;
  d.max_pages = sq->max_pages;
  d.n_pages = sh->n_pages;
  d.up_shift = __builtin_ctz(sh->page_size / kUnit);
  d.cap = sq->max_pages * sh->page_size;
  return d;
}

Rows device_rows(const qcache_rows* r) { return Rows{(char*)r->data, r->tok_stride, r->head_stride, r->type == QGEMV_F32}; }

// Calls f with the <head_dim, groups> of the shape as integral constants.
template <int D, int NG>
struct Dims {};
template <class F>
hipError_t by_shape(const qcache_shape* sh, F f) {
  const int ng = sh->head_dim / sh->group;
  if (sh->head_dim == 64) return ng == 1 ? f(Dims<64, 1>{}) : f(Dims<64, 2>{});
  if (sh->head_dim == 128) return ng == 1 ? f(Dims<128, 1>{}) : ng == 2 ? f(Dims<128, 2>{}) : f(Dims<128, 4>{});
  return ng == 2 ? f(Dims<256, 2>{}) : ng == 4 ? f(Dims<256, 4>{}) : f(Dims<256, 8>{});
}

// The checks that calls which write or read rows have in common.
int check_copy(const qcache_shape* shape, const void* cache, const qcache_seqs* seqs, const qcache_rows* k,
                      const qcache_rows* v) {
  int st = check_shape(shape);
  if (st) return st;
  if (!cache || (uintptr_t)cache % 256) return QGEMV_ERR_INVALID_ARG;
  if ((st = check_seqs(shape, seqs))) return st;
  if (seqs->n_seq == 0 || seqs->n_tok == 0) return QGEMV_OK;
  if ((st = check_rows(k)) || (st = check_rows(v))) return st;
  if (k->type != v->type) return QGEMV_ERR_INVALID_ARG;
  // a grid holds fewer than 2^32 threads
  if (unit_workgroups(*seqs, shape->n_heads) * 256 > 0xFFFFFFFFll) return QGEMV_ERR_UNSUPPORTED;
  return QGEMV_OK;
}

}  // namespace
