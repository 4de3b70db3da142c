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
  int pairs, log_pairs, axes, n_tok, halves;  // log_pairs: of the power of two from pairs on
};

// ---------------------------------------------------------------------------
// A workgroup of four waves takes one unit (16 positions of a sequence) and some
// of its heads.  It first forms the unit's sines and cosines in LDS, which all
// heads share; then its waves take the heads' values, keys and queries in turn.
//
// The angle p f is formed in 64 bits and reduced exactly: t = p f / 2 pi in two
// parts, less its nearest quarter.  Turning in 64 bits as well costs nothing
// that shows (the call is bound by HBM), and makes the FP16 key, and with it the 4-bit
// code, that of the exact turn: in fp32 one FP16 in some 10^4 would fall on the
// other side of a rounding border, and with it, where it is a group's end, the
// group's step.
//
// 30021 tokens of 64 query and 8 key/value heads x 128 (1.14 GB): 229 to 234 us among such calls (three axes 240), 4.9 TB/s, a
// copy's rate; alone, the caches clean, 217, and behind 256 MiB of writes 255.  Their writing alone takes 36.  Steps there: 390 with a load, its turn and its store at a time; 270
// with four heads' loads at once; 229 with the next heads' loads ahead of the turn, and the keys turned like queries and passed
// to the lanes that quantise them by way of LDS (155 to 256 registers before, 98 to 147 after).
// ---------------------------------------------------------------------------
constexpr int kTable = 16;  // tokens of a unit

// Pair i of token t: 16 bytes at (t * pairs + place(i)); 8 neighbouring pairs, which a lane takes, lie pairs / 8 apart, so
// that neighbouring lanes read neighbouring 16 bytes.
__device__ __forceinline__ int place(int i, int pairs) { return (i & 7) * (pairs >> 3) + (i >> 3); }

// (cos, sin) of p f.  With t = p f / 2 pi less its nearest quarter, |x| = 2 pi |t| <= pi / 4: Taylor's series to x^13 and
// x^14 are within 3e-14, and the quarter turns them.
__device__ __forceinline__ doublex2_t cos_sin(int pos, double f) {
  constexpr double k1 = 0.15915494309189535, k2 = -9.8393384282593e-18;  // 1 / 2 pi
  const double a = (double)pos * f;
  const double t = a * k1;
  const double lo = __builtin_fma(a, k1, -t) + a * k2;
  const double n = __builtin_rint(4.0 * t);  // exact, as is what it leaves of t
  const double x = 6.283185307179586 * (__builtin_fma(-0.25, n, t) + lo), z = x * x;
  double s = 1.0 / 6227020800.0, c = -1.0 / 87178291200.0;
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  s = __builtin_fma(x * z, s, x);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  // the quarter, modulo 4; an angle that is not finite is NaN either way
  const int q = (int)(n - 4.0 * __builtin_floor(0.25 * n));
  const double cc = q & 1 ? s : c, ss = q & 1 ? c : s;
  return (doublex2_t){q == 1 || q == 2 ? -cc : cc, q >= 2 ? -ss : ss};
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

// In the place of the cosine of a pair without an axis, which is left as it is: cosine 1 and sine 0 would make it NaN where its partner is
// not finite.
constexpr double kStays = 2.0;

__device__ __forceinline__ void turn(float& a, float& b, doublex2_t cs) {
  const double x = a, y = b;
  const bool stays = cs[0] == kStays;
  a = stays ? a : (float)__builtin_fma(x, cs[0], -(y * cs[1]));
  b = stays ? b : (float)__builtin_fma(y, cs[0], x * cs[1]);
}

// What a lane takes of a head of D dimensions: two runs of 8, the two that turn together or two neighbours.
template <int D>
struct Slot {
  static constexpr int lanes = D / 16, heads = 64 / lanes;  // lanes of a head, heads of a wave
  int slot, r0, r1;
  bool joint, apart;  // turned as pairs of runs, or within runs

  __device__ __forceinline__ Slot(const Turn& tn, int lane) {
    slot = lane % lanes;
    const int runs = tn.pairs >> 2;  // of the turned dimensions
    joint = tn.halves && slot < runs / 2;
    apart = !tn.halves && 2 * slot < runs;
    r0 = joint ? slot : 2 * slot;
    r1 = joint ? slot + runs / 2 : 2 * slot + 1;
  }
  // tab: the token's pairs
  __device__ __forceinline__ void turned(float (&a)[8], float (&b)[8], const Turn& tn, const doublex2_t* tab) const {
    if (joint) {
#pragma unroll
      for (int j = 0; j < 8; ++j) turn(a[j], b[j], tab[j * (tn.pairs >> 3) + slot]);
    } else if (apart) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        turn(a[2 * j], a[2 * j + 1], tab[place(4 * r0 + j, tn.pairs)]);
        turn(b[2 * j], b[2 * j + 1], tab[place(4 * r1 + j, tn.pairs)]);
      }
    }
  }
};

// A unit's keys of one head, turned and stored: turned as queries are, a token's D / 16 lanes side by side, and by way of the
// wave's LDS to the lanes that quantise them.
template <int D>
constexpr int key_stride() { return 2 * D + 16; }  // bytes of a token, 16 of them for the banks

template <int D, int NG>
__device__ __forceinline__ void turned_keys(uint8_t* unit, const Rows& k, const Turn& tn, const doublex2_t* s_tab,
                                            uint8_t* s_key, int64_t row0, int h, int t0, int t1, int lane) {
  constexpr int ND = Geo<D, NG>::ND;
  const Slot<D> sl(tn, lane);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 2
  for (int tt = 0; tt < 16; tt += Slot<D>::heads) {
    const int t = tt + lane / Slot<D>::lanes;
    float a[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (t >= t0 && t < t1) {
      const int64_t e = (row0 + t) * k.ts + (int64_t)h * k.hs;
      load_run(k, e + 8 * sl.r0, a);
      load_run(k, e + 8 * sl.r1, b);
      sl.turned(a, b, tn, s_tab + t * tn.pairs);
    }
    u32x4_t x, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pk_h(a[2 * i], a[2 * i + 1]), y[i] = pk_h(b[2 * i], b[2 * i + 1]);
    *(u32x4_t*)(s_key + t * key_stride<D>() + 16 * sl.r0) = x;
    *(u32x4_t*)(s_key + t * key_stride<D>() + 16 * sl.r1) = y;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int t = lane & 15, kq = lane >> 4;
  uint32_t pk[4 * ND];
#pragma unroll
  for (int j = 0; j < ND; ++j) {
    const u32x4_t x = *(const u32x4_t*)(s_key + t * key_stride<D>() + 16 * (4 * j + kq));
#pragma unroll
    for (int i = 0; i < 4; ++i) pk[4 * j + i] = x[i];
  }
  store_keys<D, NG>(unit, pk, t >= t0 && t < t1, lane);
}

// The queries of the unit's tokens t0 .. t1 - 1, heads q0 .. q1 - 1.  U heads' loads are on their way while U others' are
// turned; the first before the sines are there.
template <int D, bool F32>
struct Queries {
  static constexpr int SL = Slot<D>::lanes, VW = Slot<D>::heads;
  static constexpr int U = F32 ? 1 : 2, N = F32 ? 2 : 1;
  const Rows &q, &qo;
  const Turn& tn;
  int64_t row0;
  int t0, q0, q1, lane, groups, items;
  Slot<D> sl;
  u32x4_t raw[U][2][N];

  __device__ __forceinline__ Queries(const Rows& q_, const Rows& qo_, const Turn& tn_, int64_t row0_, int t0_, int t1, int q0_,
                                     int q1_, int lane_)
      : q(q_), qo(qo_), tn(tn_), row0(row0_), t0(t0_), q0(q0_), q1(q1_), lane(lane_), sl(tn_, lane_) {
    groups = (q1 - q0 + VW - 1) / VW;
    items = (t1 - t0) * groups;
  }
  // Token and head of item i; the head is q1 where there is none.
  __device__ __forceinline__ void item(int i, int& t, int& h) const {
    const int g = i / max(groups, 1);
    t = t0 + g;
    h = i < items ? min(q0 + (i - g * groups) * VW + lane / SL, q1) : q1;
  }
  __device__ __forceinline__ void load(int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int t, h;
      item(i0 + 4 * u, t, h);
      if (h >= q1) continue;
      const int64_t e = (row0 + t) * q.ts + (int64_t)h * q.hs;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        raw[u][0][n] = *((const u32x4_t*)(q.data + (e + 8 * sl.r0) * (F32 ? 4 : 2)) + n);
        raw[u][1][n] = *((const u32x4_t*)(q.data + (e + 8 * sl.r1) * (F32 ? 4 : 2)) + n);
      }
    }
  }
  static __device__ __forceinline__ void unpack(const u32x4_t (&w)[N], float (&v)[8]) {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j / 4][j % 4]);
    } else {
      const half8_t x = __builtin_bit_cast(half8_t, w[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)x[j];
    }
  }
  // What was loaded for i0, turned and stored; what follows it is loaded meanwhile.
  __device__ __forceinline__ void turn_and_store(int i0, const doublex2_t* s_tab) {
    float a[U][8], b[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) unpack(raw[u][0], a[u]), unpack(raw[u][1], b[u]);
    load(i0 + 4 * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int t, h;
      item(i0 + 4 * u, t, h);
      if (h >= q1) continue;
      sl.turned(a[u], b[u], tn, s_tab + t * tn.pairs);
      const int64_t eo = (row0 + t) * qo.ts + (int64_t)h * qo.hs;
      store_run(qo, eo + 8 * sl.r0, a[u]);
      store_run(qo, eo + 8 * sl.r1, b[u]);
    }
  }
};

template <int D, int NG, bool QF32>
__global__ void __launch_bounds__(256, 3)
k_qrotary_write(uint8_t* __restrict__ cache, Seqs sq, Turn tn, Rows q, Rows qo, Rows k, Rows v, int heads, int q_heads,
                int split) {
  using L = Geo<D, NG>;
  extern __shared__ doublex2_t s_tab[];
  const int idx = blockIdx.x / split, part = blockIdx.x - idx * split;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = threadIdx.x & ((1 << tn.log_pairs) - 1);
  const int axis = tn.pair_axis && pair < tn.pairs ? tn.pair_axis[pair] : 0;
  const bool turns = pair < tn.pairs && (uint32_t)axis < (uint32_t)tn.axes;
  const double f = turns ? tn.freqs[pair] : 0.0;
  const UnitTask x = unit_task(sq, idx);
  if (x.s < 0) return;
  const int t0 = max(x.p0 - 16 * x.u, 0), t1 = min(x.p0 + x.n - 16 * x.u, 16);  // the unit's tokens
  const int row0 = x.row + 16 * x.u - x.p0;                                     // row of token 0
  const int p = sq.page(x.s, x.u);
  const int q0 = (int)((int64_t)q_heads * part / split), q1 = (int)((int64_t)q_heads * (part + 1) / split);
  Queries<D, QF32> qs(q, qo, tn, row0, t0, t1, q0, q1, lane);
  qs.load(w);
  if (pair < tn.pairs) {
    const int32_t* pos = tn.positions && turns ? tn.positions + (int64_t)axis * tn.n_tok + row0 : nullptr;
    for (int t = t0 + (threadIdx.x >> tn.log_pairs); t < t1; t += 256 >> tn.log_pairs)
      s_tab[t * tn.pairs + place(pair, tn.pairs)] = turns ? cos_sin(pos ? pos[t] : 16 * x.u + t, f) : (doublex2_t){kStays, 0.0};
  }
  const int h0 = (int)((int64_t)heads * part / split), h1 = (int)((int64_t)heads * (part + 1) / split);
  auto unit = [&](int h) { return cache + unit_at(p, x.u, h, heads, sq.up_shift, L::bytes); };
  if (p >= 0)
    for (int h = h0 + ((w + 3) & 3); h < h1; h += 4) write_values<D, NG>(unit(h), v, x, h, lane);
  __syncthreads();
  uint8_t* s_key = (uint8_t*)(s_tab + kTable * tn.pairs) + w * (kTable * key_stride<D>());
  if (p >= 0)
    for (int h = h0 + 3 - w; h < h1; h += 4) turned_keys<D, NG>(unit(h), k, tn, s_tab, s_key, row0, h, t0, t1, lane);
  for (int i = w; i < qs.items; i += 4 * Queries<D, QF32>::U) qs.turn_and_store(i, s_tab);
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

// Whether vectors of D elements, T x H of them, may overlap: those of the shorter stride one behind the other, as wholes those of
// the longer.
bool overlap(const Rows& r, int64_t T, int64_t H, int64_t D) {
  if (T == 1 || H == 1) return T * H > 1 && (T > 1 ? r.ts : r.hs) < D;
  const bool tokens = r.ts < r.hs;
  const int64_t in = tokens ? r.ts : r.hs, out = tokens ? r.hs : r.ts, n = tokens ? T : H;
  return in < D || (out - D) / in < n - 1;
}

// q_out at the place of q: each lane then has to store where it loaded.
bool shifted(const qcache_rows& out, const qcache_rows& in, int64_t T, int64_t H) {
  return out.data == in.data && (out.type != in.type || (T > 1 && out.tok_stride != in.tok_stride) ||
                                 (H > 1 && out.head_stride != in.head_stride));
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
  auto go = [&](auto kernel) {
    // once per instantiation (thread-safe static initialisation): 66 KiB with head_dim 256
    static const hipError_t attr = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                       kTable * (D / 2) * 16 + 4 * kTable * key_stride<D>());
    if (attr != hipSuccess) return attr;
    const size_t lds = (size_t)kTable * a.tn.pairs * 16 + 4 * kTable * key_stride<D>();
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), lds, st, a.cache, a.sq, a.tn, a.q, a.qo, a.k,
                       a.v, a.heads, a.q_heads, a.split);
    return hipGetLastError();
  };
  return a.q.f32 ? go(k_qrotary_write<D, NG, true>) : go(k_qrotary_write<D, NG, false>);
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
    if (overlap(qo, seqs->n_tok, n_q_heads, shape->head_dim)) return QGEMV_ERR_INVALID_ARG;
    if (shifted(*q_out, *q, seqs->n_tok, n_q_heads)) return QGEMV_ERR_INVALID_ARG;
  }
  const Seqs sq = device_seqs(shape, seqs);
  const Turn tn = {rotary->freqs, rotary->pair_axis, rotary->positions, rotary->rot_dim / 2,
                   32 - __builtin_clz(rotary->rot_dim / 2 - 1), rotary->axes, seqs->n_tok,
                   rotary->style == QROTARY_HALVES};
  const int64_t units = seqs->q_start ? (int64_t)seqs->n_tok / 16 + 2 * (int64_t)seqs->n_seq : seqs->n_seq;
  // Few units: their heads are dealt out to more workgroups, each of which forms the sines for itself, so a unit of up to 16
  // tokens keeps four heads together.  As many as the CUs hold (head_dim 256: two of them fill a CU's LDS; a step's single
  // tokens gain nothing from more than 512).  4 x 2043 tokens of 32 + 32 heads: 519 workgroups 99 us, 1038 71, 2076 81;
  // 300 tokens of 32 + 8 heads: 21 x 8 workgroups 12.9 us, 21 x 32 15.4; 8 x 512 tokens of 16 + 4 heads x 256: 272
  // workgroups 33 us, 816 41, where the bytes take 18: two workgroups, eight waves, a CU hide little of their loads' latency (32000
  // tokens 162, the bytes 139).
  int64_t most = shape->n_heads > n_q_heads ? shape->n_heads : n_q_heads;
  if (seqs->q_start) most = (most + 3) / 4;
  const int64_t want = shape->head_dim == 256 ? 256 : seqs->q_start ? 768 : 512;
  int64_t split = units >= want ? 1 : (want + units - 1) / units;
  if (split > most) split = most;
  if (units * split * 256 > 0xFFFFFFFFll) return QGEMV_ERR_UNSUPPORTED;
  const Launch go = {(uint8_t*)cache, sq, tn, qr, qo, device_rows(k), device_rows(v), shape->n_heads, n_q_heads, (int)split};
  const uint32_t grid = (uint32_t)(units * split);
  return hip_status(by_shape(shape, [&](auto d) { return launch(d, go, grid, (hipStream_t)stream); }));
}

}  // extern "C"
