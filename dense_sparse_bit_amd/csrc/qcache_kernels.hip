// qcache_kernels.hip -- the 4-bit paged key/value cache: writing, reading back,
// and attention over it (include/qcache.h; storage in qcache_layout.h).

#include <hip/hip_runtime.h>

#include <cmath>
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
  // Sequence of row t (-1: padding) and the row's position in it (may be negative).
  __device__ __forceinline__ int find(int t, int& pos) const {
    int s = t, first = t, n = 1;
    if (q_start) {
      int lo = 0, hi = n_seq;  // the last s with start(s) <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start(mid) <= t) lo = mid;
        else hi = mid;
      }
      s = lo;
      first = start(s);
      n = start(s + 1) - first;
      if (t < first || t >= first + n) return -1;
    }
    pos = max(lens[s], 0) - n + (t - first);
    return s;
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

__device__ __forceinline__ void load8(const Rows& r, int64_t e, float (&v)[8]) {
  if (r.f32) {
    const floatx4_t a = ((const floatx4_t*)((const float*)r.data + e))[0], b = ((const floatx4_t*)((const float*)r.data + e))[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const half8_t a = *(const half8_t*)((const _Float16*)r.data + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
  }
}
__device__ __forceinline__ void store8(const Rows& r, int64_t e, const float (&v)[8]) {
  if (r.f32) {
    floatx4_t* p = (floatx4_t*)((float*)r.data + e);
    p[0] = (floatx4_t){v[0], v[1], v[2], v[3]};
    p[1] = (floatx4_t){v[4], v[5], v[6], v[7]};
  } else {
    half8_t a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (_Float16)v[i];
    *(half8_t*)((_Float16*)r.data + e) = a;
  }
}

// ---------------------------------------------------------------------------
// Quantising.  A thread takes 8 consecutive dimensions of one token and head:
// D/8 neighbouring lanes a vector, G/8 (4, 8 or 16, inside one DPP row) a group.
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ void group_min_max(float& lo, float& hi) {
  lo = fminf(lo, dpp_mov<0xB1, 0xF>(lo)), hi = fmaxf(hi, dpp_mov<0xB1, 0xF>(hi));  // lanes i ^ 1
  lo = fminf(lo, dpp_mov<0x4E, 0xF>(lo)), hi = fmaxf(hi, dpp_mov<0x4E, 0xF>(hi));  // i ^ 2
  if constexpr (N > 4)  // the other four of eight
    lo = fminf(lo, dpp_mov<0x141, 0xF>(lo)), hi = fmaxf(hi, dpp_mov<0x141, 0xF>(hi));
  if constexpr (N > 8)  // the other eight of sixteen
    lo = fminf(lo, dpp_mov<0x140, 0xF>(lo)), hi = fmaxf(hi, dpp_mov<0x140, 0xF>(hi));
}

// Codes of the thread's 8 values and its group's s and lo.
template <int G>
__device__ __forceinline__ void quantise(float (&v)[8], uint32_t (&q)[8], uint16_t& s16, uint16_t& lo16) {
  float lo = INFINITY, hi = -INFINITY, bad = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = h2f(f2h(v[i]));
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
    bad = fmaxf(bad, not_finite(f2h(v[i])) ? 1.f : 0.f);  // fminf and fmaxf pass a NaN by
  }
  float ok = -bad;
  group_min_max<G / 8>(lo, hi);
  group_min_max<G / 8>(ok, bad);
  uint16_t s = f2h((hi - lo) / 15.f);
  if (lo + 15.f * h2f(s) > 65504.f) --s;  // the FP16 below (s > 0 here)
  const float sf = h2f(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = rintf((v[i] - lo) / sf);
    q[i] = s != 0 && bad == 0.f ? (uint32_t)fminf(fmaxf(r, 0.f), 15.f) : 0u;
  }
  s16 = bad != 0.f ? (uint16_t)0x7E00u : s;
  lo16 = bad != 0.f ? (uint16_t)0u : f2h(lo);
}

// Pair layout of 8 values: nibble i + 4 e holds value 2 i + e.
__device__ __forceinline__ uint32_t pack_pairs(const uint32_t (&q)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= (q[2 * i] << (4 * i)) | (q[2 * i + 1] << (16 + 4 * i));
  return w;
}

template <int D, int NG>
__global__ void __launch_bounds__(256)
k_qcache_write(uint8_t* __restrict__ cache, Seqs sq, Rows k, Rows v, int heads) {
  using L = Geo<D, NG>;
  constexpr int C = D / 8;  // threads of a vector
  const int t = blockIdx.x * (256 / C) + threadIdx.x / C, c = threadIdx.x % C, h = blockIdx.y;
  int pos = -1, s = -1;
  if (t < sq.n_tok) s = sq.find(t, pos);
  const int u = pos >> 4;
  const int p = s >= 0 && pos >= 0 ? sq.page(s, u) : -1;
  float kv[8] = {}, vv[8] = {};
  if (p >= 0) {
    load8(k, t * k.ts + h * k.hs + 8 * c, kv);
    load8(v, t * v.ts + h * v.hs + 8 * c, vv);
  }
  // A vector's lanes share p, so no group is split by it; all lanes take part in the group minima.
  uint32_t qk[8], qv[8];
  uint16_t ks, kl, vs, vl;
  quantise<L::G>(kv, qk, ks, kl);
  quantise<L::G>(vv, qv, vs, vl);
  if (p < 0) return;
  uint8_t* unit = cache + unit_at(p, u, h, heads, sq.up_shift, L::bytes);
  const int tk = pos & 15, kq = tk >> 2;
  // keys: chunk c is step c / 4, slice c % 4
  ((uint32_t*)unit)[((c & 3) * 16 + tk) * L::ND + (c >> 2)] = pack_pairs(qk);
  // values: two runs of four dimensions, each a 16-bit half of a dword
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int quad = 2 * c + j, m = quad / L::NC, cc = quad % L::NC;
    const uint32_t w = qv[4 * j] | (qv[4 * j + 1] << 4) | (qv[4 * j + 2] << 8) | (qv[4 * j + 3] << 12);
    ((uint16_t*)(unit + L::off_v))[2 * ((kq * 16 + m) * L::ND + ((tk >> 1) & 1) * L::NC + cc) + (tk & 1)] = (uint16_t)w;
  }
  if (c % (L::G / 8) == 0) {
    const int g = c / (L::G / 8);
    ((uint16_t*)(unit + L::off_ks))[(kq * NG + g) * 4 + (tk & 3)] = ks;
    ((uint16_t*)(unit + L::off_kl))[tk * NG + g] = kl;
    ((uint16_t*)(unit + L::off_vs))[(kq * NG + g) * 8 + (tk & 3)] = vs;
    ((uint16_t*)(unit + L::off_vs))[(kq * NG + g) * 8 + 4 + (tk & 3)] = vl;
  }
}

template <int D, int NG>
__global__ void __launch_bounds__(256)
k_qcache_read(const uint8_t* __restrict__ cache, Seqs sq, Rows k, Rows v, int heads) {
  using L = Geo<D, NG>;
  constexpr int C = D / 8;
  const int t = blockIdx.x * (256 / C) + threadIdx.x / C, c = threadIdx.x % C, h = blockIdx.y;
  if (t >= sq.n_tok) return;
  int pos = -1;
  const int s = sq.find(t, pos);
  if (s < 0) return;
  const int u = pos >> 4;
  const int p = pos >= 0 ? sq.page(s, u) : -1;
  float kv[8] = {}, vv[8] = {};
  if (p >= 0) {
    const uint8_t* unit = cache + unit_at(p, u, h, heads, sq.up_shift, L::bytes);
    const int tk = pos & 15, kq = tk >> 2, g = c / (L::G / 8);
    const uint32_t w = ((const uint32_t*)unit)[((c & 3) * 16 + tk) * L::ND + (c >> 2)];
    const float ks = h2f(((const uint16_t*)(unit + L::off_ks))[(kq * NG + g) * 4 + (tk & 3)]);
    const float kl = h2f(((const uint16_t*)(unit + L::off_kl))[tk * NG + g]);
    const float vs = h2f(((const uint16_t*)(unit + L::off_vs))[(kq * NG + g) * 8 + (tk & 3)]);
    const float vl = h2f(((const uint16_t*)(unit + L::off_vs))[(kq * NG + g) * 8 + 4 + (tk & 3)]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kv[2 * i] = kl + ks * (float)((w >> (4 * i)) & 15u);
      kv[2 * i + 1] = kl + ks * (float)((w >> (16 + 4 * i)) & 15u);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int quad = 2 * c + j, m = quad / L::NC, cc = quad % L::NC;
      const uint32_t x =
          ((const uint16_t*)(unit + L::off_v))[2 * ((kq * 16 + m) * L::ND + ((tk >> 1) & 1) * L::NC + cc) + (tk & 1)];
#pragma unroll
      for (int i = 0; i < 4; ++i) vv[4 * j + i] = vl + vs * (float)((x >> (4 * i)) & 15u);
    }
  }
  store8(k, t * k.ts + h * k.hs + 8 * c, kv);
  store8(v, t * v.ts + h * v.hs + 8 * c, vv);
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
//   p = exp2(S - m), with a running maximum m per column that is raised only
//                when a score passes it by 8 (p stays below 2^8), and the sum.
//   O = V^T p    rows = dimensions; p is already where the B operand wants it.
//                Values are formed in FP16, lo + s q rounded once.
//
// q is scaled per row by a power of two so that its largest element is in
// [64, 128): sums over a group stay in FP16's range, and q / 16 is exact down
// to 2^-20 of the largest element.
//
// At the end of an item's blocks the four waves' (m, sum, O) meet in LDS.  An
// item that lies in one workgroup's range is finished there; otherwise each
// workgroup leaves a partial (at most two per workgroup: the item it starts in
// and the one it ends in), and k_qcache_join adds an item's partials in order.
// ---------------------------------------------------------------------------
struct AttendArgs {
  Seqs sq;
  const uint8_t* cache;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  float* ws_ml;  // [grid][2][rows][2]: m, sum
  float* ws_o;   // [grid][2][rows][D]
  int heads, per, rows, grid;
  float scale2;  // scale * log2 e
};

// Blocks per item and items of sequence s.
struct SeqWork {
  int len, first, n, nb, items;
};
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int s) {
  SeqWork w;
  w.first = a.sq.start(s);
  w.n = a.sq.q_start ? max(a.sq.start(s + 1) - w.first, 0) : 1;
  w.len = a.sq.lens[s];  // not cut to cap: positions count from the true end
  w.nb = (min(max(w.len, 0), a.sq.cap) + kBlock - 1) / kBlock;
  w.items = (int)(((int64_t)w.n * a.per + 15) / 16) * a.heads;
  return w;
}

__device__ __forceinline__ int wave_scan(int v) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ float column_max(float v) {  // over the four lanes of a column
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ uint32_t pk_h(float a, float b) { return (uint32_t)f2h(a) | ((uint32_t)f2h(b) << 16); }

// What a lane loads of one unit.
template <int D, int NG>
struct UnitRegs {
  uint32_t k[D / 32], v[D / 32], ks[2 * NG], kl[(NG + 1) / 2], vs[4];
};

template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t* d) {
  if constexpr (N == 1) {
    d[0] = __builtin_nontemporal_load((const uint32_t*)p);
  } else if constexpr (N == 2) {
    const u32x2_t x = __builtin_nontemporal_load((const u32x2_t*)p);
    d[0] = x[0], d[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4_t x = __builtin_nontemporal_load((const u32x4_t*)p + i / 4);
      d[i] = x[0], d[i + 1] = x[1], d[i + 2] = x[2], d[i + 3] = x[3];
    }
  }
}

template <int D, int NG>
__device__ __forceinline__ void load_unit(const uint8_t* unit, int lane, UnitRegs<D, NG>& r) {
  using L = Geo<D, NG>;
  const int n = lane & 15, kq = lane >> 4;
  load_dwords<L::ND>(unit + lane * (4 * L::ND), r.k);
  load_dwords<L::ND>(unit + L::off_v + lane * (4 * L::ND), r.v);
  load_dwords<2 * NG>(unit + L::off_ks + kq * (8 * NG), r.ks);
  if constexpr (NG == 1) r.kl[0] = ((const uint16_t*)(unit + L::off_kl))[n];
  else load_dwords<NG / 2>(unit + L::off_kl + n * (2 * NG), r.kl);
  load_dwords<4>(unit + L::off_vs + (kq * NG + n * (D / 16) / L::G) * 16, r.vs);
}

// Scores of a unit: st[i] = token 4 kq + i against column n, in log2 units.
template <int D, int NG>
__device__ __forceinline__ void unit_scores(const UnitRegs<D, NG>& r, const u32x4_t (&qf)[D / 32], u32x4_t qs,
                                            float k_s, float k_l, float (&st)[4]) {
  using L = Geo<D, NG>;
  const floatx4_t zero = {0.f, 0.f, 0.f, 0.f};
  float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    floatx4_t acc = zero;
#pragma unroll
    for (int j = g * (L::G / 32); j < (g + 1) * (L::G / 32); ++j) {
      const uint32_t w = r.k[j], w8 = w >> 8;
      acc = mfma((u32x4_t){w & 0x000F000Fu, w & 0x00F000F0u, w8 & 0x000F000Fu, w8 & 0x00F000F0u}, qf[j], acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t[i] = h2f((uint16_t)(r.ks[2 * g + i / 2] >> (16 * (i & 1)))) * acc[i] + t[i];
  }
  u32x4_t lo = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < (NG + 1) / 2; ++i) lo[i] = r.kl[i];
  const floatx4_t la = mfma(lo, qs, zero);
#pragma unroll
  for (int i = 0; i < 4; ++i) st[i] = k_s * t[i] + k_l * la[i];
}

template <int D, int NG>
__global__ void __launch_bounds__(256)
k_qcache_attend(AttendArgs a) {
  using L = Geo<D, NG>;
  constexpr int DL = D / 16;  // dimensions of a lane of V^T p, MFMAs of it
  __shared__ __align__(16) float s_o[4][16][D + 4];
  __shared__ float s_m[4][16], s_l[4][16];
  const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Seqs& sq = a.sq;

  // The range [b0, b1) of this workgroup in the list of all blocks, and the sequence it starts in.
  int total = 0, cnt = 0, inc = 0;
  for (int s0 = 0; s0 < sq.n_seq; s0 += 64) {
    cnt = 0;
    if (s0 + lane < sq.n_seq) {
      const SeqWork x = seq_work(a, s0 + lane);
      cnt = x.nb * x.items;
    }
    inc = wave_scan(cnt);
    total += __shfl(inc, 63);
  }
  const int grid = min(a.grid, total);  // no range is empty, so an item's partials are consecutive workgroups'
  if ((int)blockIdx.x >= grid) return;
  const int b0 = (int)((int64_t)blockIdx.x * total / grid), b1 = (int)((int64_t)(blockIdx.x + 1) * total / grid);
  int s = 0, at = 0;  // sequence of b0, and b0 inside it
  for (int s0 = 0, base = 0; s0 < sq.n_seq; s0 += 64) {
    if (sq.n_seq > 64) {
      cnt = 0;
      if (s0 + lane < sq.n_seq) {
        const SeqWork x = seq_work(a, s0 + lane);
        cnt = x.nb * x.items;
      }
      inc = wave_scan(cnt);
    }
    const uint64_t past = __ballot(base + inc > b0);
    if (past) {
      const int i = __builtin_ctzll(past);
      s = s0 + i;
      at = b0 - (base + __shfl(inc, i) - __shfl(cnt, i));
      break;
    }
    base += __shfl(inc, 63);
  }
  s = __builtin_amdgcn_readfirstlane(s);
  at = __builtin_amdgcn_readfirstlane(at);
  SeqWork sw = seq_work(a, s);
  int item = at / sw.nb, blk = at - item * sw.nb;

  for (int left = b1 - b0; left > 0;) {
    if (item == sw.items) {
      item = blk = 0;
      do {
        if (++s >= sq.n_seq) return;
        sw = seq_work(a, s);
      } while (sw.nb * sw.items == 0);
    }
    const int k0 = blk, k1 = min(sw.nb, blk + left);
    const int rt = item / a.heads, h = item - rt * a.heads;
    const int nrows = min(16, sw.n * a.per - rt * 16);
    left -= k1 - k0;

    // The column's row, query head and number of positions it may look at.
    const int r = rt * 16 + n, qi = r / a.per, hg = r - qi * a.per;
    const bool real = n < nrows;
    const int lim = real ? min(max(sw.len - sw.n + qi + 1, 0), sq.cap) : 0;
    const int lim_min = min(max(sw.len - sw.n + (rt * 16) / a.per + 1, 0), sq.cap);
    const int lim_max = min(max(sw.len - sw.n + (rt * 16 + nrows - 1) / a.per + 1, 0), sq.cap);

    // q: B operands, scaled by 2^e (and by 1/16 more where the code pair stays shifted).
    u32x4_t qf[L::ND];
    u32x4_t qs = {0u, 0u, 0u, 0u};
    float k_s, k_l;
    {
      const uint16_t* qp = a.q + (int64_t)(sw.first + qi) * a.q_ts + (int64_t)(h * a.per + hg) * a.q_hs + 8 * kq;
      half8_t qv[L::ND];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < L::ND; ++j) {
        qv[j] = (half8_t){0, 0, 0, 0, 0, 0, 0, 0};
        if (real) qv[j] = *(const half8_t*)(qp + 32 * j);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf((float)qv[j][i]));
      }
      top = column_max(top);
      const int e = top > 0.f && top <= 65504.f ? 6 - ilogbf(top) : 0;
      k_s = ldexpf(a.scale2, 24 - e);
      k_l = ldexpf(a.scale2, -e);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int j = g * (L::G / 32); j < (g + 1) * (L::G / 32); ++j) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = ldexpf((float)qv[j][i], e);
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
    float m = -INFINITY, l = 0.f;

    // This wave's tiles: positions 128 k + 32 w .. + 31 for k in [k0, k1).
    const int nt = k1 - k0;
    int pg = -1;  // lane 2 j + e: page of unit e of tile (32 jj + j)
    auto fetch_pages = [&](int j0) {
      const int j = j0 + (lane >> 1), u = 8 * (k0 + j) + 2 * w + (lane & 1);
      pg = j < nt && 16 * u < lim_max ? sq.page(s, u) : -1;
    };
    // Pages of tile j (of the fetched 32) into p0, p1, and its loads.
    UnitRegs<D, NG> cur[2], nxt[2];
    auto issue = [&](int j, UnitRegs<D, NG>(&d)[2], int (&p)[2]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        p[e] = __builtin_amdgcn_readlane(pg, 2 * (j & 31) + e);
        const int u = 8 * (k0 + j) + 2 * w + e;
        // a unit on no page is masked; its loads go to the first unit of the cache
        load_unit<D, NG>(p[e] < 0 ? a.cache : a.cache + unit_at(p[e], u, h, a.heads, sq.up_shift, L::bytes), lane,
                         d[e]);
      }
    };
    int pc[2] = {-1, -1}, pn[2] = {-1, -1};
    fetch_pages(0);
    issue(0, cur, pc);
    for (int j = 0; j < nt; ++j) {
      if (j + 1 < nt) {
        if (((j + 1) & 31) == 0) fetch_pages(j + 1);
        issue(j + 1, nxt, pn);
      }
      const int base = 128 * (k0 + j) + 32 * w;
      if (base < lim_max && (pc[0] >= 0 || pc[1] >= 0)) {
        float st[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) unit_scores<D, NG>(cur[e], qf, qs, k_s, k_l, st[e]);
        const bool edge = base + 32 > lim_min || pc[0] < 0 || pc[1] < 0;
        u32x4_t nan_seen = {0u, 0u, 0u, 0u};  // edge tiles: FP16 1 where a visible token's value group is NaN
        if (edge) {
          u32x4_t bad = {0u, 0u, 0u, 0u}, vis = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int pos = base + 16 * e + 4 * kq + i, hs = 16 * (i & 1);
              const bool sees = pos < lim && pc[e] >= 0;
              if (!sees) st[e][i] = -INFINITY;
              // Value statistics of tokens that no row sees may be anything: they become 0, and so do NaN
              // groups, whose NaN is added below only to the columns that see the token.
              const uint16_t vs = (uint16_t)(cur[e].vs[i / 2] >> hs), vl = (uint16_t)(cur[e].vs[2 + i / 2] >> hs);
              const bool held = pos < lim_max && pc[e] >= 0;
              const bool drop = !held || not_finite(vs) || not_finite(vl);
              if (drop) {
                cur[e].vs[i / 2] &= ~(0xFFFFu << hs);
                cur[e].vs[2 + i / 2] &= ~(0xFFFFu << hs);
              }
              if (held && drop) bad[2 * e + i / 2] |= 0x3C00u << hs;
              if (sees) vis[2 * e + i / 2] |= 0x3C00u << hs;
            }
          if (__ballot((bad[0] | bad[1] | bad[2] | bad[3]) != 0)) {
            const floatx4_t c = mfma(bad, vis, (floatx4_t){0.f, 0.f, 0.f, 0.f});  // per (dimension run, column)
#pragma unroll
            for (int i = 0; i < 4; ++i) nan_seen[i] = c[i] > 0.f;
          }
        }
        float top = st[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, st[i / 4][i % 4]);
        if (__ballot(top > m + 8.f)) {
          const float mn = fmaxf(m, column_max(top));
          const float f = mn == m ? 1.f : exp2f(m - mn);
          m = mn;
          l *= f;
#pragma unroll
          for (int j2 = 0; j2 < DL; ++j2) o[j2] *= f;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        u32x4_t pf;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = exp2f(st[e][i] - mu);
            l += p[i];
          }
          pf[2 * e] = pk_h(p[0], p[1]);
          pf[2 * e + 1] = pk_h(p[2], p[3]);
        }
        // Values: dword [tp][c] of unit e, nibble i -> dimension 4 c + i of tokens (2 tp, 2 tp + 1).
#pragma unroll
        for (int c = 0; c < L::NC; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u32x4_t av;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int tp = 0; tp < 2; ++tp) {
                const uint32_t wv = i < 2 ? cur[e].v[tp * L::NC + c] : cur[e].v[tp * L::NC + c] >> 8;
                const half2_t x = as_h2((i & 1) ? (wv & 0x00F000F0u) | 0x64006400u : (wv & 0x000F000Fu) | 0x64006400u);
                const _Float16 inv = (_Float16)((i & 1) ? 0.0625f : 1.f), off = (_Float16)((i & 1) ? -64.f : -1024.f);
                const half2_t q = x * (half2_t){inv, inv} + (half2_t){off, off};
                av[2 * e + tp] = as_u32(q * as_h2(cur[e].vs[tp]) + as_h2(cur[e].vs[2 + tp]));
              }
            o[4 * c + i] = mfma(av, pf, o[4 * c + i]);
          }
        }
        if (edge)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (nan_seen[i])
#pragma unroll
              for (int j2 = 0; j2 < DL; ++j2) o[j2][i] = NAN;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        cur[e] = nxt[e];
        pc[e] = pn[e];
      }
    }

    // The four waves meet.  o[j][i] is dimension (4 kq + i) DL + j of column n.
    l = column_sum(l);
    if (real) {
      if (kq == 0) {
        s_m[w][n] = m;
        s_l[w][n] = l;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < DL; j += 4)
          *(floatx4_t*)&s_o[w][n][(4 * kq + i) * DL + j] = (floatx4_t){o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]};
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == sw.nb;
    for (int x = threadIdx.x; x < nrows * (D / 4); x += 256) {
      const int row = x / (D / 4), d = 4 * (x - row * (D / 4));
      const float mx = fmaxf(fmaxf(s_m[0][row], s_m[1][row]), fmaxf(s_m[2][row], s_m[3][row]));
      const float mu = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      floatx4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = exp2f(s_m[u][row] - mu);
        sum += f * s_l[u][row];
        v += f * *(const floatx4_t*)&s_o[u][row][d];
      }
      if (whole) {
        const int rr = rt * 16 + row, i = rr / a.per;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const u32x2_t y = {pk_h(v[0] * inv, v[1] * inv), pk_h(v[2] * inv, v[3] * inv)};
        *(u32x2_t*)(a.out + (int64_t)(sw.first + i) * a.o_ts + (int64_t)(h * a.per + rr - i * a.per) * a.o_hs + d) = y;
      } else {
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (k0 > 0 ? 0 : 1)) * a.rows + row;
        *(floatx4_t*)(a.ws_o + slot * D + d) = v;
        if (d == 0) {
          a.ws_ml[2 * slot] = mx;
          a.ws_ml[2 * slot + 1] = sum;
        }
      }
    }
    __syncthreads();
    blk = 0;
    ++item;
  }
}

// One workgroup of D threads per (item, row of its tile): adds the item's
// partials in order and writes the row; rows of empty sequences become 0.
template <int D>
__global__ void __launch_bounds__(D)
k_qcache_join(AttendArgs a) {
  const int lane = threadIdx.x & 63;
  const Seqs& sq = a.sq;
  int total = 0, s = -1, item = 0, start = 0;  // start: first block of the sequence
  for (int s0 = 0, ibase = 0; s0 < sq.n_seq; s0 += 64) {
    int cb = 0, ci = 0;
    if (s0 + lane < sq.n_seq) {
      const SeqWork x = seq_work(a, s0 + lane);
      ci = x.items;
      cb = x.nb * x.items;
    }
    const int ib = wave_scan(cb), ii = wave_scan(ci);
    const uint64_t past = __ballot(ibase + ii > (int)blockIdx.x);
    if (s < 0 && past) {
      const int i = __builtin_ctzll(past);
      s = s0 + i;
      item = (int)blockIdx.x - (ibase + __shfl(ii, i) - __shfl(ci, i));
      start = total + __shfl(ib, i) - __shfl(cb, i);
    }
    ibase += __shfl(ii, 63);
    total += __shfl(ib, 63);
  }
  if (s < 0) return;
  const SeqWork sw = seq_work(a, s);
  const int rt = item / a.heads, h = item - rt * a.heads, row = blockIdx.y, rr = rt * 16 + row;
  if (rr >= sw.n * a.per) return;
  const int i = rr / a.per, d = threadIdx.x;
  uint16_t* y = a.out + (int64_t)(sw.first + i) * a.o_ts + (int64_t)(h * a.per + rr - i * a.per) * a.o_hs + d;
  if (sw.nb == 0) {
    *y = 0;
    return;
  }
  const int64_t x0 = start + (int64_t)item * sw.nb;
  const int grid = min(a.grid, total);
  const int ga = (int)(((x0 + 1) * grid - 1) / total), gb = (int)(((x0 + sw.nb) * grid - 1) / total);
  if (ga == gb) return;
  auto slot = [&](int g) { return ((int64_t)g * 2 + (g == ga ? 1 : 0)) * a.rows + row; };
  float mx = -INFINITY;
  for (int g = ga; g <= gb; ++g) mx = fmaxf(mx, a.ws_ml[2 * slot(g)]);
  const float mu = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, v = 0.f;
  for (int g = ga; g <= gb; ++g) {
    const float f = exp2f(a.ws_ml[2 * slot(g)] - mu);
    sum += f * a.ws_ml[2 * slot(g) + 1];
    v += f * a.ws_o[slot(g) * D + d];
  }
  *y = f2h(sum == 0.f ? 0.f : v / sum);
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
  const int per = 256 / (D / 8);
  hipLaunchKernelGGL((k_qcache_write<D, NG>), dim3((sq.n_tok + per - 1) / per, heads), dim3(256), 0, st, cache, sq, k, v,
                     heads);
  return hipGetLastError();
}
template <int D, int NG>
hipError_t launch_read(Dims<D, NG>, const uint8_t* cache, const Seqs& sq, const Rows& k, const Rows& v, int heads,
                       hipStream_t st) {
  const int per = 256 / (D / 8);
  hipLaunchKernelGGL((k_qcache_read<D, NG>), dim3((sq.n_tok + per - 1) / per, heads), dim3(256), 0, st, cache, sq, k, v,
                     heads);
  return hipGetLastError();
}

// The launch of an attention call: workgroups, partial rows per slot, and an
// upper bound of the items (row tiles times heads) for the join.
struct AttendPlan {
  int grid, rows;
  int64_t items;
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
  p.items = tiles * sh->n_heads;
  const int64_t cap = (int64_t)sq->max_pages * sh->page_size;
  const int64_t blocks = (cap + kBlock - 1) / kBlock;
  if (p.items > 0x7FFFFFFF || (blocks > 0 && p.items > 0x7FFFFFFF / blocks)) return QGEMV_ERR_UNSUPPORTED;
  if ((int64_t)sq->n_tok * per > 0x7FFFFFFF - 16) return QGEMV_ERR_UNSUPPORTED;
  const int64_t all = p.items * blocks;
  p.grid = all < 1 ? 1 : all < 1024 ? (int)all : 1024;
  p.rows = sq->q_start || per > 16 ? 16 : per;
  p.bytes = (size_t)p.grid * 2 * p.rows * (sh->head_dim + 2) * 4;
  return QGEMV_OK;
}

template <int D, int NG>
hipError_t launch_attend(Dims<D, NG>, const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
  hipLaunchKernelGGL((k_qcache_attend<D, NG>), dim3(p.grid), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_qcache_join<D>), dim3((uint32_t)p.items, p.rows), dim3(D), 0, st, a);
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
  return k->type == v->type ? QGEMV_OK : QGEMV_ERR_INVALID_ARG;
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
  if (!cache || (uintptr_t)cache % 256 || !std::isfinite(scale)) return QGEMV_ERR_INVALID_ARG;
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
  a.heads = shape->n_heads;
  a.per = n_q_heads / shape->n_heads;
  a.rows = p.rows;
  a.grid = p.grid;
  a.scale2 = scale * 1.4426950408889634f;
  return hip_status(by_shape(shape, [&](auto d) { return launch_attend(d, a, p, (hipStream_t)stream); }));
}

}  // extern "C"
