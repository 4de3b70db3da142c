// qcache_kernels.hip -- the 4-bit paged key/value cache: writing, reading back,
// and attention over it (include/qcache.h; storage in qcache_layout.h).

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

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

template <int D, int NG>
__device__ __forceinline__ void write_keys(uint8_t* unit, const Rows& k, const UnitTask& x, int h, int lane) {
  using L = Geo<D, NG>;
  constexpr int R = L::G / 32;  // runs of a group
  const int t = lane & 15, kq = lane >> 4, pos = 16 * x.u + t;
  const bool on = pos >= x.p0 && pos < x.p0 + x.n;
  uint32_t v[4 * L::ND];
#pragma unroll
  for (int i = 0; i < 4 * L::ND; ++i) v[i] = 0;
  if (on) {
    const int64_t e = (int64_t)(x.row + pos - x.p0) * k.ts + (int64_t)h * k.hs + 8 * kq;
#pragma unroll
    for (int j = 0; j < L::ND; ++j) load_pairs<8>(k, e + 32 * j, v + 4 * j);
  }
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

// Four waves a workgroup: two units' keys and values.  Neighbouring workgroups take the heads of the same rows, which
// are neighbours in memory.
template <int D, int NG>
__global__ void __launch_bounds__(256)
k_qcache_write(uint8_t* __restrict__ cache, Seqs sq, Rows k, Rows v, int heads, Divisor by_heads) {
  const int pair = by_heads.of(blockIdx.x), h = blockIdx.x - pair * heads;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const UnitTask x = unit_task(sq, pair * 2 + (w >> 1));
  if (x.s < 0) return;
  const int p = sq.page(x.s, x.u);
  if (p < 0) return;
  uint8_t* unit = cache + unit_at(p, x.u, h, heads, sq.up_shift, Geo<D, NG>::bytes);
  if (w & 1) write_values<D, NG>(unit, v, x, h, lane);
  else write_keys<D, NG>(unit, k, x, h, lane);
}

template <int D, int NG>
__global__ void __launch_bounds__(256)
k_qcache_read(const uint8_t* __restrict__ cache, Seqs sq, Rows k, Rows v, int heads, Divisor by_heads) {
  using L = Geo<D, NG>;
  __shared__ u32x4_t s_row[2][D > 64 ? 64 * (D / 64) : 1];  // a value wave's row pieces, of fp32
  const int pair = by_heads.of(blockIdx.x), h = blockIdx.x - pair * heads;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const UnitTask x = unit_task(sq, pair * 2 + (w >> 1));
  if (x.s < 0) return;
  const int p = sq.page(x.s, x.u);
  const uint8_t* unit = cache + unit_at(max(p, 0), x.u, h, heads, sq.up_shift, L::bytes);
  const int n = lane & 15, kq = lane >> 4;
  uint32_t c[L::ND];
#pragma unroll
  for (int i = 0; i < L::ND; ++i) c[i] = 0;
  const uint32_t* from = (const uint32_t*)(unit + ((w & 1) ? L::off_v : 0)) + lane * L::ND;
  if (p >= 0) {
    if constexpr (L::ND == 2) {
      const u32x2_t y = *(const u32x2_t*)from;
      c[0] = y[0], c[1] = y[1];
    } else {
#pragma unroll
      for (int i = 0; i < L::ND; i += 4) {
        const u32x4_t y = *(const u32x4_t*)(from + i);
        c[i] = y[0], c[i + 1] = y[1], c[i + 2] = y[2], c[i + 3] = y[3];
      }
    }
  }
  if (w & 1) {
    constexpr int DL = D / 16, N = L::G / DL;
    u32x4_t st = {0u, 0u, 0u, 0u};
    if (p >= 0) st = *(const u32x4_t*)(unit + L::off_vs + (kq * NG + n / N) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = 16 * x.u + 4 * kq + i, hs = 16 * (i & 1);
      const bool on = pos >= x.p0 && pos < x.p0 + x.n;
      const float s = h2f((uint16_t)(st[i / 2] >> hs)), lo = h2f((uint16_t)(st[2 + i / 2] >> hs));
      float o[DL];
#pragma unroll
      for (int j = 0; j < DL; ++j) o[j] = lo + s * (float)((c[(i >> 1) * L::NC + j / 4] >> (hs + 4 * (j & 3))) & 15u);
      const int64_t e = (int64_t)(x.row + pos - x.p0) * v.ts + (int64_t)h * v.hs;
      if (v.f32) {
        u32x4_t y[DL / 4];
#pragma unroll
        for (int j = 0; j < DL / 4; ++j)
          y[j] = __builtin_bit_cast(u32x4_t, (floatx4_t){o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]});
        store_row<DL / 4>(v.data + 4 * e, y, lane, s_row[w >> 1], on);
      } else if constexpr (DL >= 8) {
        u32x4_t y[DL / 8];
#pragma unroll
        for (int j = 0; j < DL / 2; ++j) y[j / 4][j & 3] = pk_h(o[2 * j], o[2 * j + 1]);
        store_row<DL / 8>(v.data + 2 * e, y, lane, s_row[w >> 1], on);
      } else if (on) {
        __builtin_nontemporal_store((u32x2_t){pk_h(o[0], o[1]), pk_h(o[2], o[3])}, (u32x2_t*)(v.data + 2 * e + 8 * n));
      }
    }
  } else {
    float s[NG], lo[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      s[g] = lo[g] = 0.f;
      if (p >= 0) {
        s[g] = h2f(((const uint16_t*)(unit + L::off_ks))[((n >> 2) * NG + g) * 4 + (n & 3)]);
        lo[g] = h2f(((const uint16_t*)(unit + L::off_kl))[n * NG + g]);
      }
    }
    // the rows of the lane's token pair; lane n even has the first half of each of its 128-byte pieces, n odd the second
    const int pos = 16 * x.u + (n & ~1);
    const bool on0 = pos >= x.p0 && pos < x.p0 + x.n, on1 = pos + 1 >= x.p0 && pos + 1 < x.p0 + x.n;
    const int64_t el = k.f32 ? 4 : 2;
    char* row0 = k.data + el * ((int64_t)(x.row + pos - x.p0) * k.ts + (int64_t)h * k.hs) + 64 * (n & 1) + 16 * kq;
    char* row1 = row0 + el * k.ts;
    auto put = [&](int at, u32x4_t y, u32x4_t z) {
      by_pair(y, z, n & 1);
      if (on0) stream_out(row0 + at, y);
      if (on1) stream_out(row1 + at, z);
    };
#pragma unroll
    for (int j2 = 0; j2 < L::ND; j2 += 2) {
      float o[2][8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int g = 32 * (j2 + r) / L::G;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[r][i] = lo[g] + s[g] * (float)((c[j2 + r] >> (16 * (i & 1) + 4 * (i / 2))) & 15u);
      }
      if (k.f32) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          u32x4_t y = __builtin_bit_cast(u32x4_t, (floatx4_t){o[r][0], o[r][1], o[r][2], o[r][3]});
          u32x4_t z = __builtin_bit_cast(u32x4_t, (floatx4_t){o[r][4], o[r][5], o[r][6], o[r][7]});
          by_column(y, z);
          put(128 * (j2 + r), y, z);
        }
      } else {
        u32x4_t y, z;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = pk_h(o[0][2 * i], o[0][2 * i + 1]), z[i] = pk_h(o[1][2 * i], o[1][2 * i + 1]);
        put(64 * j2, y, z);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Attention.
//
// An item is one tile of up to 16 (row, query head) pairs of one sequence and
// key/value head; its positions are cut into blocks of 128.  All items' blocks,
// one after another, are cut into equal ranges, one per workgroup, so that
// ragged batches keep every CU busy whatever the lengths (which only the
// device knows).  Inside a block wave w takes positions 32 w .. + 31:
//
//   S = K q      rows = tokens, columns = the tile's pairs.  The A operands are
//                the codes as they are: (w >> 4i) & 0x000f000f is a pair of
//                FP16 subnormals c 2^-24, which the MFMA takes exactly.  Where
//                i is odd the nibble stays 4 bits up and q is divided by 16
//                instead.  Each group's sum is scaled by its step in fp32; the
//                lowest values are one more MFMA, lo[token][group] times the
//                sum of q over the group (as an FP16 part and its FP16 rest).
//   p = exp2(S - m), with a reference m per column: 7 below the largest score
//                when it was set, set anew only when a score passes it by 15.
//                So p lies below 2^15, and FP16 holds what is 2^-31 of the largest.
//   O = V^T p    rows = dimensions; p is already where the B operand wants it, as
//                an FP16 part and its FP16 rest, each in an MFMA.  Values are
//                formed in FP16, lo + s q rounded once.
//
// Without the rest of p its rounding counts as much as the values' and the
// output's do: 3.3e-4 of the outputs' 2-norm in all, 2.7e-4 with it, 2.1e-4 for
// the output's alone.  It costs 1 to 5 % (16 x 8 heads x 32768: 128 -> 134 us).
//
// q is scaled per row by a power of two so that its largest element is in
// [64, 128): sums over a group stay in FP16's range.  Elements are exact down to
// 2^-20 of the largest, those divided by 16 down to 2^-16 of it; what is smaller
// is rounded by at most 2^-31 and 2^-27 of the largest.
//
// A wave's next 32 positions are copied from HBM straight into its own part of
// LDS while it works on the current ones; the units' statistics, which 4 or 16
// lanes share, then cross HBM once.  Registers would not do: two tiles of them
// leave two waves a SIMD (63 against 51 us for 32 heads x 32768 positions), and
// a second tile ahead in LDS (keys and values in rings of their own) costs more
// copy instructions than it hides (128 -> 136 us for 16 x 8 heads x 32768).
//
// Long contexts are bound by what three workgroups a CU keep on its way from
// HBM: 4.9 TB/s (168 MB, 34 us without the join), 5.3 to 5.7 (672 MB, 119 to 127 us; a copy of
// the same card: 4.8, a plain read: 6.8) with the VALU busy for 68 to 73 % of the CUs' cycles.
// The loop's counters and addresses are scalars, more than fit: the compiler keeps
// 72 to 83 of them in lanes of vector registers, and starting a tile's copy reads
// some ten of them back.  Short contexts are bound by the chain of loads
// (lengths, pages, tile) of one workgroup: 8 us for 32 heads x 181 positions.
//
// At the end of an item's blocks the four waves' (m, sum, O) meet in LDS.  An
// item that lies in one workgroup's range is finished there; otherwise each
// workgroup leaves a partial (at most two per workgroup: the item it starts in,
// slot 0, and the one it ends in, slot 1), and k_qcache_join adds them in order.
// ---------------------------------------------------------------------------
// How `total` blocks are cut into `grid` ranges: the first rem have q + 1, the others q.
struct Cut {
  int q, rem;
  __device__ __forceinline__ Cut(int total, int grid) : q(total / grid), rem(total - total / grid * grid) {}
  __device__ __forceinline__ int begin(int g) const { return g * q + min(g, rem); }
  __device__ __forceinline__ int range_of(int x) const {  // the range of block x
    const int y = x - rem * (q + 1);
    return y < 0 ? x / (q + 1) : rem + y / q;
  }
};

struct AttendArgs {
  Seqs sq;
  const uint8_t* cache;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  float* ws_o;   // [grid][2][rows][D]
  float* ws_ml;  // [grid][2][rows][4]: m, sum, k_l (m's unit), -
  int* ws_join;  // [grid][4]: last workgroup of the item that this one ends in (-1: none), its first row, item, rows
  int heads, per, rows, grid;
  int whole;  // ranges are cut between items only: every item is one workgroup's
  Divisor by_heads, by_per;
  float scale2;  // scale * log2 e
};

// Sequence s: its length, first row and rows, the blocks of an item, an item's cost and the items.  The cost is what
// ranges are cut by: one per block and kItemCost for the item's start and end (its pages and q, the waves'
// meeting), which come after the blocks; or 1, where ranges are cut between items only.
// Ragged batches gain (31 sequences of 100 to 9000 positions: 55 us without the cost, 40 with), others are as they were.
constexpr int kItemCost = 3;
struct SeqWork {
  int len, first, n, nb, cost, items;
};
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int s) {
  SeqWork w;
  w.first = a.sq.start(s);
  w.n = a.sq.q_start ? max(a.sq.start(s + 1) - w.first, 0) : 1;
  w.len = a.sq.lens[s];  // not cut to cap: positions count from the true end
  w.nb = (min(max(w.len, 0), a.sq.cap) + kBlock - 1) / kBlock;
  w.cost = w.nb == 0 ? 0 : a.whole ? 1 : w.nb + kItemCost;
  w.items = ((w.n * a.per + 15) >> 4) * a.heads;
  return w;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {  // inclusive
  v = dpp_add<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8: inside the rows of 16
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // lane 15 of rows 0, 2 to rows 1, 3
  return dpp_add<0x143, 0xC>(v);  // lane 31 to rows 2, 3
}

// The same value, unknown to the compiler: what is computed from it stays where it is written, instead of being
// kept in registers across a loop that has none to spare.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// -1, unknown to the compiler: p - h as h * -1 + p is one instruction with h's conversion from FP16.
__device__ __forceinline__ float minus_one() {
  float v = -1.f;
  asm("" : "+s"(v));
  return v;
}

// (w & mask) | magic in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t d;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(d) : "v"(w), "s"(mask), "v"(magic));
  return d;
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kNonTemporal = 2;

// Copy `bytes` (a multiple of 16, the same for all lanes) from src to LDS, 16 bytes a lane and round; with no source, zeros.
template <int BYTES>
__device__ __forceinline__ void copy_to_lds(const uint8_t* src, bool real, uint8_t* dst, int lane) {
  const rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(src), (short)0, real ? BYTES : 0, 0x00020000);
#pragma unroll
  for (int o = 0; o < BYTES; o += 1024)
    if (o + 1024 <= BYTES || o + 16 * lane < BYTES)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(dst + o), 16, 16 * lane, o, 0,
                                               kNonTemporal);
}

// What a lane holds of one unit: the keys' part, and the values' part.
template <int D, int NG>
struct KeyRegs {
  uint32_t k[D / 32], ks[2 * NG], kl[(NG + 1) / 2];
};
template <int D>
struct ValueRegs {
  uint32_t v[D / 32], vs[4];
};

template <int N>
__device__ __forceinline__ void read_dwords(const uint8_t* p, uint32_t* d) {
  if constexpr (N == 1) {
    d[0] = *(const uint32_t*)p;
  } else if constexpr (N == 2) {
    const u32x2_t x = *(const u32x2_t*)p;
    d[0] = x[0], d[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4_t x = ((const u32x4_t*)p)[i / 4];
      d[i] = x[0], d[i + 1] = x[1], d[i + 2] = x[2], d[i + 3] = x[3];
    }
  }
}

template <int D, int NG>
__device__ __forceinline__ void read_keys(const uint8_t* unit, int lane, KeyRegs<D, NG>& r) {
  using L = Geo<D, NG>;
  const int n = lane & 15, kq = lane >> 4;
  read_dwords<L::ND>(unit + lane * (4 * L::ND), r.k);
  read_dwords<2 * NG>(unit + L::off_ks + kq * (8 * NG), r.ks);
  if constexpr (NG == 1) r.kl[0] = ((const uint16_t*)(unit + L::off_kl))[n];
  else read_dwords<NG / 2>(unit + L::off_kl + n * (2 * NG), r.kl);
}

// The values' part of a tile's two units.  Written out, with the wait in the
// same block, because the next tile's copy into LDS is then under way: the
// compiler, not knowing which bytes it writes, would wait for it before any LDS
// read of its own.
template <int D, int NG>
__device__ __forceinline__ void read_values(const uint8_t* tile, int lane, ValueRegs<D> (&r)[2]) {
  using L = Geo<D, NG>;
  const int n = lane & 15, kq = lane >> 4;
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)tile;
  const uint32_t av = at + L::off_v + (uint32_t)lane * (4 * L::ND);
  const uint32_t as = at + L::off_vs + (uint32_t)(kq * NG + n * (D / 16) / L::G) * 16;
  u32x4_t s0, s1;
  if constexpr (L::ND == 2) {
    u32x2_t v0, v1;
    asm volatile(
        "ds_read_b64 %0, %4\n\tds_read_b64 %1, %4 offset:%6\n\tds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:%6\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v0), "=&v"(v1), "=&v"(s0), "=&v"(s1)
        : "v"(av), "v"(as), "n"(L::bytes)
        : "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i) r[0].v[i] = v0[i], r[1].v[i] = v1[i];
  } else if constexpr (L::ND == 4) {
    u32x4_t v0, v1;
    asm volatile(
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%6\n\tds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:%6\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v0), "=&v"(v1), "=&v"(s0), "=&v"(s1)
        : "v"(av), "v"(as), "n"(L::bytes)
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) r[0].v[i] = v0[i], r[1].v[i] = v1[i];
  } else {
    u32x4_t v0, v1, v2, v3;
    asm volatile(
        "ds_read_b128 %0, %6\n\tds_read_b128 %1, %6 offset:16\n\tds_read_b128 %2, %6 offset:%8\n\t"
        "ds_read_b128 %3, %6 offset:%9\n\tds_read_b128 %4, %7\n\tds_read_b128 %5, %7 offset:%8\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v0), "=&v"(v1), "=&v"(v2), "=&v"(v3), "=&v"(s0), "=&v"(s1)
        : "v"(av), "v"(as), "n"(L::bytes), "n"(L::bytes + 16)
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) r[0].v[i] = v0[i], r[0].v[4 + i] = v1[i], r[1].v[i] = v2[i], r[1].v[4 + i] = v3[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) r[0].vs[i] = s0[i], r[1].vs[i] = s1[i];
}

// Scores of a tile: st[e][i] = token 4 kq + i of unit e against column n, in units of the column's k_l.
template <int D, int NG>
__device__ __forceinline__ void tile_scores(const KeyRegs<D, NG> (&r)[2], const u32x4_t (&qf)[D / 32], u32x4_t qs,
                                            float (&st)[2][4]) {
  using L = Geo<D, NG>;
  const floatx4_t zero = {0.f, 0.f, 0.f, 0.f};
  floatx4_t acc[2];
  float t[2][4];
  auto scale = [&](int g) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float step = h2f((uint16_t)(r[e].ks[2 * g + i / 2] >> (16 * (i & 1))));
        t[e][i] = __builtin_fmaf(step, acc[e][i], g == 0 ? 0.f : t[e][i]);  // + 0: one instruction, with the conversion
      }
  };
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    floatx4_t nxt[2] = {zero, zero};
#pragma unroll
    for (int j = g * (L::G / 32); j < (g + 1) * (L::G / 32); ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t w = r[e].k[j], w8 = w >> 8;
        nxt[e] = mfma((u32x4_t){w & 0x000F000Fu, w & 0x00F000F0u, w8 & 0x000F000Fu, w8 & 0x00F000F0u}, qf[j], nxt[e]);
      }
    if (g > 0) scale(g - 1);
    acc[0] = nxt[0];
    acc[1] = nxt[1];
  }
  floatx4_t la[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    u32x4_t lo = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < (NG + 1) / 2; ++i) lo[i] = r[e].kl[i];
    la[e] = mfma(lo, qs, zero);
  }
  scale(NG - 1);
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) st[e][i] = t[e][i] * 16777216.f + la[e][i];  // the codes were c 2^-24
}

// Workgroups of a CU at once, by their registers (with 4 of head_dim 128, groups of 32 spill: 51 -> 61 us for 32 heads
// x 32768 positions, and with larger groups the additional partials cost more than they bring: 32 -> 36 us for sixteen
// ragged sequences).
constexpr int attend_resident(int D) { return D == 256 ? 2 : D == 128 ? 3 : 4; }

template <int D, int NG>
constexpr int attend_lds() {  // the waves' tiles; then, over them, their O, m and sums
  const int ring = 4 * 2 * 2 * Geo<D, NG>::bytes, meet = 4 * 16 * (D + 4) * 4 + (2 * 4 + 1) * 16 * 4;
  return ring > meet ? ring : meet;
}

template <int D, int NG>
__global__ void __launch_bounds__(256, attend_resident(D))
k_qcache_attend(AttendArgs a) {
  using L = Geo<D, NG>;
  constexpr int DL = D / 16;  // dimensions of a lane of V^T p, MFMAs of it
  __shared__ __align__(16) uint8_t lds[attend_lds<D, NG>()];
  float(*s_o)[16][D + 4] = (float(*)[16][D + 4])lds;
  float(*s_m)[16] = (float(*)[16])(lds + 4 * 16 * (D + 4) * 4);
  float(*s_l)[16] = s_m + 4;
  float* s_k = s_l[4];
  const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* ring = lds + w * (4 * L::bytes);  // two tiles
  const Seqs& sq = a.sq;

  // The lane's sequence of the 64 from sc on, and the blocks up to its end in that chunk.
  SeqWork mine;
  int sc, cnt, inc;
  auto load_chunk = [&](int s0) {
    sc = s0;
    mine = SeqWork{0, 0, 0, 0, 0, 0};
    if (s0 + lane < sq.n_seq) mine = seq_work(a, s0 + lane);
    cnt = mine.cost * mine.items;
    inc = wave_scan(cnt);
  };
  auto of_lane = [&](int i) {
    auto get = [&](int v) { return __builtin_amdgcn_readlane(v, i); };
    return SeqWork{get(mine.len), get(mine.first), get(mine.n), get(mine.nb), get(mine.cost), get(mine.items)};
  };

  // All blocks; rows of empty sequences become 0 on the way.  Every workgroup looks at every sequence, 64 a round: 16
  // sequences of 8192 positions take 40 us, among 128 in all 41, among 512 51, among 4096 159.
  int total = 0;
  for (int s0 = 0; s0 < sq.n_seq; s0 += 64) {
    load_chunk(s0);
    total += __builtin_amdgcn_readlane(inc, 63);
    uint64_t none = __ballot(mine.items > 0 && mine.nb == 0);
    if (none) none = __ballot(mine.items > 0 && mine.nb == 0 && (s0 + lane) % (int)gridDim.x == (int)blockIdx.x);
    for (; none; none &= none - 1) {
      const SeqWork x = of_lane(__builtin_ctzll(none));
      const int per_row = a.per * a.heads * (D / 8);
      for (int i = 0; i < x.n; ++i)
        for (int e = threadIdx.x; e < per_row; e += 256)
          *(u32x4_t*)(a.out + (int64_t)(x.first + i) * a.o_ts + (int64_t)(e / (D / 8)) * a.o_hs + 8 * (e % (D / 8))) =
              (u32x4_t){0u, 0u, 0u, 0u};
    }
  }
  const int grid = min(a.grid, total);  // no range is empty, so an item's partials are consecutive workgroups'
  int* join = a.ws_join + 4 * blockIdx.x;
  if ((int)blockIdx.x >= grid) {
    if (threadIdx.x == 0) join[0] = -1;
    return;
  }
  // This workgroup's range [b0, b1) of all blocks, the sequence it starts in, and the place there.
  const Cut cut(total, grid);
  const int b0 = cut.begin(blockIdx.x), b1 = cut.begin(blockIdx.x + 1);
  int s = 0, at = 0;
  for (int s0 = 0, base = 0; s0 < sq.n_seq; s0 += 64) {
    if (sc != s0) load_chunk(s0);
    const uint64_t past = __ballot(base + inc > b0);
    if (past) {
      const int i = __builtin_ctzll(past);
      s = s0 + i;
      at = b0 - (base + __builtin_amdgcn_readlane(inc, i) - __builtin_amdgcn_readlane(cnt, i));
      break;
    }
    base += __builtin_amdgcn_readlane(inc, 63);
  }
  SeqWork sw = of_lane(s - sc);
  int item = at / sw.cost, blk = at - item * sw.cost;
  int start = b0 - at;  // first part of the sequence
  bool tail = false;

  for (int left = b1 - b0; left > 0;) {
    if (item == sw.items) {
      start += sw.cost * sw.items;
      item = blk = 0;
      do {
        if (++s >= sq.n_seq) {  // only if q_start or lens have changed meanwhile
          if (threadIdx.x == 0) join[0] = -1;
          return;
        }
        const SeqWork x = seq_work(a, s);
        auto get = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        sw = SeqWork{get(x.len), get(x.first), get(x.n), get(x.nb), get(x.cost), get(x.items)};
      } while (sw.cost * sw.items == 0);
    }
    const int parts = min(sw.cost - blk, left);
    const int k0 = blk, k1 = a.whole ? sw.nb : min(blk + parts, sw.nb), nt = k1 - k0;
    const int it = item;
    // moved on here, in front of every branch on the lane: the loop's counters stay scalar
    left -= parts;
    blk = 0;
    ++item;
    if (nt <= 0) continue;  // only the cost of its end
    const int rt = a.by_heads.of(it), h = it - rt * a.heads;
    const int nrows = min(16, sw.n * a.per - rt * 16);

    // Last positions that the tile's first and last row and the column's row may look at, plus 1.
    const int r = rt * 16 + n, qi = a.by_per.of(r), hg = r - qi * a.per;
    const bool real = n < nrows;
    const int lim = real ? min(max(sw.len - sw.n + qi + 1, 0), sq.cap) : 0;
    const int lim_min = min(max(sw.len - sw.n + a.by_per.of(rt * 16) + 1, 0), sq.cap);
    const int lim_max = min(max(sw.len - sw.n + a.by_per.of(rt * 16 + nrows - 1) + 1, 0), sq.cap);

    // Loads: the pages of this wave's first 32 tiles (positions 128 k + 32 w .. + 31 for k in [k0, k1); lane
    // 2 j + e: unit e of tile j), q, and the first tile.
    int pg = -1;
    auto fetch_pages = [&](int j0) {
      const int j = j0 + (lane >> 1), u = 8 * (k0 + j) + 2 * w + (lane & 1);
      pg = j < nt && 16 * u < lim_max ? sq.page(s, u) : -1;
    };
    fetch_pages(0);
    half8_t qv[L::ND];
    {
      const uint16_t* qp = a.q + (int64_t)(sw.first + qi) * a.q_ts + (int64_t)(h * a.per + hg) * a.q_hs + 8 * kq;
#pragma unroll
      for (int j = 0; j < L::ND; ++j) {
        qv[j] = (half8_t){0, 0, 0, 0, 0, 0, 0, 0};
        if (real) qv[j] = *(const half8_t*)(qp + 32 * j);
      }
    }
    int p0, p1;  // pages of the two units of the tile being copied
    auto issue = [&](int j) {
      uint8_t* to = ring + (j & 1) * (2 * L::bytes);
      p0 = __builtin_amdgcn_readlane(pg, 2 * (j & 31));
      p1 = __builtin_amdgcn_readlane(pg, 2 * (j & 31) + 1);
      const int u = 8 * (k0 + j) + 2 * w;
      if (sq.up_shift > 0 && p0 >= 0) {
        // both units on one page, side by side; the second may lie past the last position, but not past the page
        copy_to_lds<2 * L::bytes>(a.cache + unit_at(p0, u, h, a.heads, sq.up_shift, L::bytes), true, to, lane);
      } else {
        copy_to_lds<L::bytes>(a.cache + unit_at(max(p0, 0), u, h, a.heads, sq.up_shift, L::bytes), p0 >= 0, to, lane);
        copy_to_lds<L::bytes>(a.cache + unit_at(max(p1, 0), u + 1, h, a.heads, sq.up_shift, L::bytes), p1 >= 0,
                              to + L::bytes, lane);
      }
    };
    issue(0);

    // q: B operands, scaled by 2^e (and by 1/16 more where the code pair stays shifted).
    u32x4_t qf[L::ND];
    u32x4_t qs = {0u, 0u, 0u, 0u};
    float k_l, raise;  // log2 units of a score; 15 of them as scores, how far one may pass m
    {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < L::ND; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf((float)qv[j][i]));
      top = column_max(top);
      const int e = top > 0.f && top <= 65504.f ? 6 - ilogbf(top) : 0;
      // never 0 nor infinite, and 15 / k_l finite: all meet infinities below
      k_l = fminf(fmaxf(ldexpf(fabsf(a.scale2), -e), 1e-37f), 1e30f);
      raise = 15.f / k_l;
      const float up = a.scale2 < 0.f ? -ldexpf(1.f, e) : ldexpf(1.f, e);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int j = g * (L::G / 32); j < (g + 1) * (L::G / 32); ++j) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = (float)qv[j][i] * up;
            sum += x[i];
            if (i & 2) x[i] *= 0.0625f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[j][i] = pk_h(x[2 * i], x[2 * i + 1]);
        }
        sum = column_sum(sum);
        const uint16_t hi = f2h(sum), lo = f2h(sum - h2f(hi));
        const uint32_t part = kq == 0 ? hi : kq == 1 ? lo : 0u;
        qs[g / 2] |= part << (16 * (g & 1));
      }
    }

    floatx4_t o[DL];
#pragma unroll
    for (int j = 0; j < DL; ++j) o[j] = (floatx4_t){0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, mu = 0.f, l = 0.f;  // m as a score; m, but 0 while it is -inf; sum of p

    const float minus = minus_one();
    for (int j = 0; j < nt; ++j) {
      const int base = 128 * (k0 + j) + 32 * w;
      const bool on0 = p0 >= 0, on1 = p1 >= 0;
      const uint8_t* here = ring + (j & 1) * (2 * L::bytes);
      KeyRegs<D, NG> kr[2];
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this tile has landed
      read_keys<D, NG>(here, lane, kr[0]);
      read_keys<D, NG>(here + L::bytes, lane, kr[1]);
      if (j + 1 < nt) {
        if (((j + 1) & 31) == 0) fetch_pages(j + 1);
        issue(j + 1);  // over the tile before this one
      }
      if (base >= lim_max || !(on0 || on1)) continue;
      const bool edge = base + 32 > lim_min || !on0 || !on1;  // some of the tile is masked for some row
      float st[2][4];
      tile_scores<D, NG>(kr, qf, qs, st);
      if (edge) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((e ? on1 : on0) && base + 16 * e + 4 * kq + i < lim)) st[e][i] = -INFINITY;
      }
      float top = st[0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, st[i / 4][i % 4]);
      if (__ballot(top - m > raise)) {  // the difference: m + raise could be rounded past what FP16 holds
        const float mn = fmaxf(m, column_max(top) - raise * (7.f / 15.f));
        const float f = mn == m ? 1.f : exp2_(k_l * (m - mn));
        m = mn;
        mu = mn == -INFINITY ? 0.f : mn;
        l *= f;
#pragma unroll
        for (int j2 = 0; j2 < DL; ++j2) o[j2] *= f;
      }
      u32x4_t pf, pr;  // p in FP16, and the rest of it
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // the difference first: exact near the maximum, however large the scores are
          p[i] = exp2_(k_l * (st[e][i] - mu));
          l += p[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          pf[2 * e + i] = pk_h(p[2 * i], p[2 * i + 1]);
          const half2_t y = as_h2(pf[2 * e + i]);
          pr[2 * e + i] = pk_h(__builtin_fmaf((float)y[0], minus, p[2 * i]), __builtin_fmaf((float)y[1], minus, p[2 * i + 1]));
        }
      }
      ValueRegs<D> c[2];
      read_values<D, NG>(here, lane, c);
      if (edge) {
        // Value statistics of tokens that no row sees may be anything: they become 0, and so do those of NaN
        // groups, whose NaN goes only to the columns that see the token (one MFMA of FP16 ones: per dimension
        // run and column, how many of the NaN groups' tokens the column sees).
        u32x4_t bad = {0u, 0u, 0u, 0u}, vis = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = base + 16 * e + 4 * kq + i, hs = 16 * (i & 1);
            const bool on = e ? on1 : on0, held = pos < lim_max && on;
            const uint16_t vs = (uint16_t)(c[e].vs[i / 2] >> hs), vl = (uint16_t)(c[e].vs[2 + i / 2] >> hs);
            const bool drop = !held || not_finite(vs) || not_finite(vl);
            if (drop) {
              c[e].vs[i / 2] &= ~(0xFFFFu << hs);
              c[e].vs[2 + i / 2] &= ~(0xFFFFu << hs);
            }
            if (held && drop) bad[2 * e + i / 2] |= 0x3C00u << hs;
            if (pos < lim && on) vis[2 * e + i / 2] |= 0x3C00u << hs;
          }
        if (__ballot((bad[0] | bad[1] | bad[2] | bad[3]) != 0)) {
          const floatx4_t x = mfma(bad, vis, (floatx4_t){0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (x[i] > 0.f)
#pragma unroll
              for (int j2 = 0; j2 < DL; ++j2) o[j2][i] = NAN;
        }
      }
      // Values: dword [tp][cc] of unit e, nibble i -> dimension 4 cc + i of tokens (2 tp, 2 tp + 1).
#pragma unroll
      for (int cc = 0; cc < L::NC; ++cc) {
        uint32_t wv[4], w8[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          wv[x] = c[x / 2].v[(x & 1) * L::NC + cc];
          w8[x] = wv[x] >> 8;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u32x4_t av;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const half2_t y = as_h2(and_or(i < 2 ? wv[x] : w8[x], (i & 1) ? 0x00F000F0u : 0x000F000Fu, kMagic));
            const _Float16 inv = (_Float16)((i & 1) ? 0.0625f : 1.f), off = (_Float16)((i & 1) ? -64.f : -1024.f);
            const half2_t q = y * (half2_t){inv, inv} + (half2_t){off, off};
            av[x] = as_u32(q * as_h2(c[x / 2].vs[x & 1]) + as_h2(c[x / 2].vs[2 + (x & 1)]));
          }
          o[4 * cc + i] = mfma(av, pf, o[4 * cc + i]);
          o[4 * cc + i] = mfma(av, pr, o[4 * cc + i]);
        }
      }
    }

    // The four waves meet.  o[j][i] is dimension (4 kq + i) DL + j of column n.
    const int tid = opaque((int)threadIdx.x);
    l = column_sum(l);
    __syncthreads();  // every wave has read its last tile
    if (real) {
      const int c = tid & 15, k4 = (tid >> 4) & 3;
      if (k4 == 0) {
        s_m[w][c] = m;
        if (w == 0) s_k[c] = k_l;
        s_l[w][c] = l;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < DL; j += 4)
          *(floatx4_t*)&s_o[w][c][(4 * k4 + i) * DL + j] = (floatx4_t){o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]};
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == sw.nb;
    tail = k0 == 0 && k1 < sw.nb;
    for (int x = tid; x < nrows * (D / 4); x += 256) {
      const int row = x / (D / 4), d = 4 * (x - row * (D / 4));
      const float mx = fmaxf(fmaxf(s_m[0][row], s_m[1][row]), fmaxf(s_m[2][row], s_m[3][row]));
      const float mu = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      floatx4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = exp2_(s_k[row] * (s_m[u][row] - mu));
        sum += f * s_l[u][row];
        v += f * *(const floatx4_t*)&s_o[u][row][d];
      }
      if (whole) {
        const int rr = rt * 16 + row, i = a.by_per.of(rr);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const u32x2_t y = {pk_h(v[0] * inv, v[1] * inv), pk_h(v[2] * inv, v[3] * inv)};
        *(u32x2_t*)(a.out + (int64_t)(sw.first + i) * a.o_ts + (int64_t)(h * a.per + rr - i * a.per) * a.o_hs + d) = y;
      } else {
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (k0 > 0 ? 0 : 1)) * a.rows + row;
        *(floatx4_t*)(a.ws_o + slot * D + d) = v;
        if (d == 0) {
          *(floatx4_t*)(a.ws_ml + 4 * slot) = (floatx4_t){mx, sum, s_k[row], 0.f};
        }
      }
    }
    if (tail && tid == 0) {
      *(int4*)join = make_int4(cut.range_of(start + it * sw.cost + sw.nb - 1), sw.first, it, nrows);
    }
    __syncthreads();
  }
  if (!tail && threadIdx.x == 0) join[0] = -1;
}

// Workgroup g adds, in order, the partials of the item that attention's
// workgroup g began and did not finish.  Thread x takes four dimensions of a
// row and every PG-th partial, then PG threads' sums meet in LDS.
constexpr int kJoinThreads = 512;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
k_qcache_join(AttendArgs a) {
  __shared__ floatx4_t s_v[kJoinThreads];
  __shared__ float s_m[kJoinThreads], s_l[kJoinThreads];
  const int4 j = *(const int4*)(a.ws_join + 4 * blockIdx.x);
  const int g = blockIdx.x, last = min(j.x, a.grid - 1), first = j.y, item = j.z, nrows = j.w;
  if (last < 0) return;
  const int rt = a.by_heads.of(item), h = item - rt * a.heads;
  static_assert(16 * (256 / 4) <= 2 * kJoinThreads, "at most two passes");
  const int width = min(nrows * (D / 4), kJoinThreads), pg = kJoinThreads / width;
  const int grp = threadIdx.x / width, x1 = threadIdx.x - grp * width;
  for (int x0 = 0; x0 < nrows * (D / 4); x0 += width) {
    const int x = x0 + x1, row = x / (D / 4), d = 4 * (x - row * (D / 4));
    const bool on = grp < pg && row < nrows;
    float m = -INFINITY, l = 0.f;
    floatx4_t v = {0.f, 0.f, 0.f, 0.f};
    float k_l = 1.f;  // the same in all of a row's partials
    auto add = [&](float pm, float pl, floatx4_t pv) {
      const float mn = fmaxf(m, pm), mu = mn == -INFINITY ? 0.f : mn;
      const float f = exp2_(k_l * (m - mu)), pf = exp2_(k_l * (pm - mu));
      l = f * l + pf * pl;
      v = f * v + pf * pv;
      m = mn;
    };
    if (on) {
#pragma unroll 4
      for (int i = g + grp; i <= last; i += pg) {
        const int64_t slot = ((int64_t)i * 2 + (i == g ? 1 : 0)) * a.rows + row;
        const floatx4_t ml = *(const floatx4_t*)(a.ws_ml + 4 * slot);
        k_l = ml[2];
        add(ml[0], ml[1], *(const floatx4_t*)(a.ws_o + slot * D + d));
      }
    }
    if (pg > 1) {
      s_v[threadIdx.x] = v;
      s_m[threadIdx.x] = m;
      s_l[threadIdx.x] = l;
      __syncthreads();
      if (on && grp == 0)
        for (int i = 1; i < pg; ++i) add(s_m[x1 + i * width], s_l[x1 + i * width], s_v[x1 + i * width]);
    }
    if (on && grp == 0) {
      const int rr = rt * 16 + row, i = a.by_per.of(rr);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const u32x2_t y = {pk_h(v[0] * inv, v[1] * inv), pk_h(v[2] * inv, v[3] * inv)};
      *(u32x2_t*)(a.out + (int64_t)(first + i) * a.o_ts + (int64_t)(h * a.per + rr - i * a.per) * a.o_hs + d) = y;
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

template <int D, int NG>
hipError_t launch_write(Dims<D, NG>, uint8_t* cache, const Seqs& sq, const Rows& k, const Rows& v, int heads,
                        hipStream_t st) {
  hipLaunchKernelGGL((k_qcache_write<D, NG>), dim3((uint32_t)unit_workgroups(sq, heads)), dim3(256), 0, st, cache, sq, k, v,
                     heads, divisor(heads));
  return hipGetLastError();
}
template <int D, int NG>
hipError_t launch_read(Dims<D, NG>, const uint8_t* cache, const Seqs& sq, const Rows& k, const Rows& v, int heads,
                       hipStream_t st) {
  hipLaunchKernelGGL((k_qcache_read<D, NG>), dim3((uint32_t)unit_workgroups(sq, heads)), dim3(256), 0, st, cache, sq, k, v,
                     heads, divisor(heads));
  return hipGetLastError();
}

// The launch of an attention call: workgroups, and partial rows per slot.
struct AttendPlan {
  int grid, rows;
  bool whole;
  size_t bytes;
};

int attend_plan(const qcache_shape* sh, const qcache_seqs* sq, int32_t n_q_heads, AttendPlan& p) {
  int st = check_shape(sh);
  if (st == QGEMV_OK) st = check_counts(sh, sq);
  if (st) return st;
  if (n_q_heads < 1) return QGEMV_ERR_INVALID_ARG;
  if (n_q_heads > 65535 || n_q_heads % sh->n_heads) return QGEMV_ERR_UNSUPPORTED;
  const int per = n_q_heads / sh->n_heads;
  // a sequence of n rows has ceil(n per / 16) tiles: at most n per / 16 + 1, and one per sequence with one row each
  const int64_t tiles = sq->q_start ? sq->n_seq + (int64_t)sq->n_tok * per / 16
                                    : (int64_t)sq->n_seq * ((per + 15) / 16);
  const int64_t items = tiles * sh->n_heads;
  const int64_t cap = (int64_t)sq->max_pages * sh->page_size;
  const int64_t blocks = (cap + kBlock - 1) / kBlock;
  if (items > 0x7FFFFFFF / (blocks + kItemCost)) return QGEMV_ERR_UNSUPPORTED;
  if ((int64_t)sq->n_tok * per > 0x7FFFFFFF - 16) return QGEMV_ERR_UNSUPPORTED;
  // Up to 4 blocks an item (by the table's width, which the host knows): a workgroup takes whole items, and there
  // is nothing to join.  A further block costs it about 1.5 us, the join's launch 5 us.
  p.whole = blocks <= 4;
  // As many workgroups as the 256 CUs hold at once: with more, the last ones start when the first have ended and
  // the launch takes two rounds (32 heads x 32768 positions: 51 us with 1024 workgroups where 768 fit, 40 with 768).
  const int64_t all = p.whole ? items : items * blocks;
  const int most = 256 * attend_resident(sh->head_dim);
  p.grid = all < 1 ? 1 : all < most ? (int)all : most;
  p.rows = sq->q_start || per > 16 ? 16 : per;
  p.bytes = (size_t)p.grid * (2 * (size_t)p.rows * (sh->head_dim + 4) * 4 + 16);
  return QGEMV_OK;
}

template <int D, int NG>
hipError_t launch_attend(Dims<D, NG>, const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
  hipLaunchKernelGGL((k_qcache_attend<D, NG>), dim3(p.grid), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.whole) return e;
  hipLaunchKernelGGL((k_qcache_join<D>), dim3(p.grid), dim3(kJoinThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

extern "C" {

int qcache_bytes(const qcache_shape* shape, size_t* bytes) {
  const int st = check_shape(shape);
  if (st) return st;
  if (!bytes) return QGEMV_ERR_INVALID_ARG;
  *bytes = (size_t)shape->n_pages * shape->n_heads * (shape->page_size / kUnit) * unit_bytes(shape->head_dim, shape->group);
  return QGEMV_OK;
}

static int check_copy(const qcache_shape* shape, const void* cache, const qcache_seqs* seqs, const qcache_rows* k,
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

int qcache_write(const qcache_shape* shape, void* cache, const qcache_seqs* seqs, const qcache_rows* k,
                 const qcache_rows* v, void* stream) {
  const int st = check_copy(shape, cache, seqs, k, v);
  if (st || seqs->n_seq == 0 || seqs->n_tok == 0) return st;
  const Seqs sq = device_seqs(shape, seqs);
  return hip_status(by_shape(shape, [&](auto d) {
    return launch_write(d, (uint8_t*)cache, sq, device_rows(k), device_rows(v), shape->n_heads, (hipStream_t)stream);
  }));
}

int qcache_read(const qcache_shape* shape, const void* cache, const qcache_seqs* seqs, const qcache_rows* k,
                const qcache_rows* v, void* stream) {
  const int st = check_copy(shape, cache, seqs, k, v);
  if (st || seqs->n_seq == 0 || seqs->n_tok == 0) return st;
  const Seqs sq = device_seqs(shape, seqs);
  return hip_status(by_shape(shape, [&](auto d) {
    return launch_read(d, (const uint8_t*)cache, sq, device_rows(k), device_rows(v), shape->n_heads,
                       (hipStream_t)stream);
  }));
}

int qcache_attend_ws(const qcache_shape* shape, const qcache_seqs* seqs, int32_t n_q_heads, size_t* bytes) {
  AttendPlan p;
  const int st = attend_plan(shape, seqs, n_q_heads, p);
  if (st) return st;
  if (!bytes) return QGEMV_ERR_INVALID_ARG;
  *bytes = p.bytes;
  return QGEMV_OK;
}

int qcache_attend(const qcache_shape* shape, const void* cache, const qcache_seqs* seqs, int32_t n_q_heads,
                  const qcache_rows* q, const qcache_rows* out, float scale, void* ws, size_t ws_bytes, void* stream) {
  AttendPlan p;
  int st = attend_plan(shape, seqs, n_q_heads, p);
  if (st) return st;
  const float scale2 = scale * 1.4426950408889634f;
  if (!cache || (uintptr_t)cache % 256 || !std::isfinite(scale2)) return QGEMV_ERR_INVALID_ARG;
  if ((st = check_seqs(shape, seqs))) return st;
  if (seqs->n_seq == 0 || seqs->n_tok == 0) return QGEMV_OK;
  if ((st = check_rows(q)) || (st = check_rows(out))) return st;
  if (q->type != QGEMV_F16 || out->type != QGEMV_F16) return QGEMV_ERR_UNSUPPORTED;
  if (!ws || (uintptr_t)ws % 256) return QGEMV_ERR_INVALID_ARG;
  if (ws_bytes < p.bytes) return QGEMV_ERR_SIZE;
  AttendArgs a;
  a.sq = device_seqs(shape, seqs);
  a.cache = (const uint8_t*)cache;
  a.q = (const uint16_t*)q->data;
  a.out = (uint16_t*)out->data;
  a.q_ts = q->tok_stride;
  a.q_hs = q->head_stride;
  a.o_ts = out->tok_stride;
  a.o_hs = out->head_stride;
  a.ws_o = (float*)ws;
  a.ws_ml = a.ws_o + (size_t)p.grid * 2 * p.rows * shape->head_dim;
  a.ws_join = (int*)(a.ws_ml + (size_t)p.grid * 2 * p.rows * 4);
  a.heads = shape->n_heads;
  a.per = n_q_heads / shape->n_heads;
  a.rows = p.rows;
  a.grid = p.grid;
  a.whole = p.whole;
  a.by_heads = divisor(a.heads);
  a.by_per = divisor(a.per);
  a.scale2 = scale2;
  return hip_status(by_shape(shape, [&](auto d) { return launch_attend(d, a, p, (hipStream_t)stream); }));
}

}  // extern "C"
