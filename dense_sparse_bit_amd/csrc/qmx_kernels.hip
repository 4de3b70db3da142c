// qmx_kernels.hip -- rows in MX blocks: quantising, values, plain arrays, and
// the product of two sets of blocks on the scaled MFMAs (include/qmx.h; storage
// in qmx_layout.h).

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/qmx.h"
#include "qgemv_epilogue_dev.h"
#include "qgemv_internal.h"
#include "qmx_blocks.h"
#include "qmx_layout.h"
#include "qmx_ring.h"

using namespace qmx_layout;
using namespace qmx_dev;

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float floatx16_t __attribute__((ext_vector_type(16)));
typedef float floatx1_t __attribute__((ext_vector_type(1)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Quantising, and the values back.
//
// A wave takes a chunk (16 rows x 128 columns).  In each of four steps 16 lanes
// take the 128 columns of a row, 8 columns a lane: rows move in contiguous 256
// (FP16) or 512 (fp32) bytes, four neighbouring lanes hold a block, and its
// largest value is two lane exchanges away.
// ---------------------------------------------------------------------------
template <bool F32>
__device__ __forceinline__ void load8(const void* x, int64_t e, float (&v)[8]) {
  if constexpr (F32) {
    const floatx4_t* p = (const floatx4_t*)((const float*)x + e);
    const floatx4_t a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const half8_t a = __builtin_bit_cast(half8_t, __builtin_nontemporal_load((const u32x4_t*)((const _Float16*)x + e)));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
  }
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(256)
k_mx_quantize(uint8_t* __restrict__ blocks, Geo g, const void* __restrict__ x, int64_t ldx, int clip, int total) {
  const int lane = threadIdx.x & 63;
  const int id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= total) return;
  const int tile = id / g.chunks, chunk = id - tile * g.chunks;
  const int c = lane & 15, col = 128 * chunk + 8 * c;
  uint8_t* to = blocks + tile * g.tile_bytes + (int64_t)chunk * (FMT ? 2048 : 1024);
  uint8_t* ex = blocks + g.exps + ((int64_t)tile * g.quads + (chunk >> 2)) * 256 + (chunk & 3);
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * tile + 4 * i + (lane >> 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
    if (row < g.rows && col < g.cols) load8<F32>(x, row * ldx + col, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + (lane >> 4);
    uint32_t w[2];
    const uint32_t byte = mx_quad<FMT>(v[i], clip, w);
    if (16 * tile + r >= g.rows) continue;
    if constexpr (FMT == kE2M1) *(uint32_t*)(to + lane_bytes<FMT>(r, c)) = w[0];
    else *(u32x2_t*)(to + lane_bytes<FMT>(r, c)) = (u32x2_t){w[0], w[1]};
    if ((c & 3) == 0) ex[4 * (16 * (c >> 2) + r)] = (uint8_t)byte;
  }
}

// N values of neighbouring codes.
template <int FMT, int N>
__device__ __forceinline__ void decode(uint64_t w, float step, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (FMT == kE2M1) {
      const uint32_t q = (uint32_t)w >> (4 * i), m = q & 7;
      // E2M1's bits in place of the top of an fp32's, times 2^126; 0.5 is the only subnormal
      const float a = m < 2 ? 0.5f * (float)m : __uint_as_float((m << 22) + (126u << 23));
      v[i] = (q & 8 ? -a : a) * step;
    } else {
      const uint32_t q = (uint32_t)(w >> (8 * i)), m = q & 127;
      const float a = m < 8 ? (float)m * 0.001953125f : m == 127 ? __uint_as_float(0x7FC00000u)
                                                                 : __uint_as_float((m << 20) + (120u << 23));
      v[i] = (q & 128 ? -a : a) * step;
    }
  }
}

// Rows leave 16 bytes a lane, lanes side by side: 8 columns of FP16, 4 of fp32 (8 in fp32, two stores with gaps: 8190 x 11008
// from E4M3 in 106 us, so 93).
template <int FMT, bool F32>
__global__ void __launch_bounds__(256)
k_mx_values(const uint8_t* __restrict__ blocks, Geo g, void* __restrict__ x, int64_t ldx, int total) {
  constexpr int N = F32 ? 4 : 8, H = 8 / N;  // columns of a lane and store, stores of a row
  const int lane = threadIdx.x & 63;
  const int id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= total) return;
  const int tile = id / g.chunks, chunk = id - tile * g.chunks;
  const uint8_t* from = blocks + tile * g.tile_bytes + (int64_t)chunk * (FMT ? 2048 : 1024);
  const uint8_t* ex = blocks + g.exps + ((int64_t)tile * g.quads + (chunk >> 2)) * 256 + (chunk & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + (lane >> 4), row = 16 * tile + r;
    if (row >= g.rows) return;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int c = 64 * h + N * (lane & 15), col = 128 * chunk + c;  // column in the chunk, and of all
      if (col >= g.cols) continue;
      const uint8_t* p = from + lane_bytes<FMT>(r, c >> 3);
      const float step = mx_step(ex[4 * (16 * (c >> 5) + r)]);
      float v[N];
      if constexpr (F32) {
        if constexpr (FMT == kE2M1) decode<FMT, N>(*(const uint16_t*)(p + (c & 4) / 2), step, v);
        else decode<FMT, N>(*(const uint32_t*)(p + (c & 4)), step, v);
        __builtin_nontemporal_store((floatx4_t){v[0], v[1], v[2], v[3]}, (floatx4_t*)((float*)x + row * ldx + col));
      } else {
        if constexpr (FMT == kE2M1) decode<FMT, N>(*(const uint32_t*)p, step, v);
        else decode<FMT, N>(*(const uint64_t*)p, step, v);
        half8_t y;
#pragma unroll
        for (int k = 0; k < N; ++k) y[k] = (_Float16)v[k];
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, y), (u32x4_t*)((_Float16*)x + row * ldx + col));
      }
    }
  }
}

// A lane moves one block: 16 or 32 bytes and its exponent byte.
template <int FMT, bool PACK>
__global__ void __launch_bounds__(256)
k_mx_plain(uint8_t* __restrict__ blocks, Geo g, uint8_t* __restrict__ codes, uint8_t* __restrict__ exps, int total) {
  constexpr int parts = FMT ? 2 : 1;
  const int lane = threadIdx.x & 63;
  const int id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= total) return;
  const int tile = id / g.chunks, chunk = id - tile * g.chunks;
  const int row = 16 * tile + (lane & 15), b = 4 * chunk + (lane >> 4), nb = g.cols / 32;
  const bool real = row < g.rows && b < nb;
  uint8_t* at = blocks + tile * g.tile_bytes + (int64_t)chunk * (1024 * parts);
  uint8_t* ex = blocks + g.exps + ((int64_t)tile * g.quads + (chunk >> 2)) * 256 + 4 * lane + (chunk & 3);
  if (!PACK && !real) return;
  const int64_t plain = ((int64_t)row * nb + b);
#pragma unroll
  for (int p = 0; p < parts; ++p) {
    u32x4_t* in = (u32x4_t*)(codes + plain * (16 * parts) + 16 * p);
    u32x4_t* bl = (u32x4_t*)(at + lane_bytes<FMT>(lane & 15, 4 * (lane >> 4) + 2 * p));
    if constexpr (PACK) *bl = real ? *in : (u32x4_t){0, 0, 0, 0};
    else *in = *bl;
  }
  if constexpr (PACK) *ex = real ? exps[plain] : 1;
  else exps[plain] = *ex;
}

// ---------------------------------------------------------------------------
// The product.  Weights are the A operand (16 features), activation rows the B
// operand (16 tokens): lane 16 q + n of a result holds features 4 q .. + 3 of
// token n, so a lane's outputs are neighbours in memory and a gated pair is in one
// lane.
// ---------------------------------------------------------------------------
struct Side {
  const uint8_t* codes;
  const uint8_t* exps;
  int64_t tile_bytes;
  int tiles;
};

// An operand of E4M3 elements in its upper and its lower eight binades.  The scaled MFMA adds E4M3 products with fewer bits
// than fp32 has below the largest: with all sixteen binades in one operand, sums came out up to 1e-4 of the largest
// product off (2e-5 of an output's 2-norm); eight at a time add up exactly.
template <int FMT>
struct Tokens {
  i32x8_t v;
};
template <>
struct Tokens<kE4M3> {
  i32x8_t v, lo;
};
template <int FMT>
__device__ __forceinline__ Tokens<FMT> tokens(i32x8_t x) {
  Tokens<FMT> t;
  if constexpr (FMT == kE2M1) {
    t.v = x;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = ((uint32_t)x[i] & 0x40404040u) >> 6;
      const uint32_t mask = (m << 8) - m;  // 0xFF where the top exponent bit is set
      t.v[i] = x[i] & (int)mask;
      t.lo[i] = x[i] & (int)~mask;
    }
  }
  return t;
}

template <int FMT, int J>
__device__ __forceinline__ floatx4_t mx_mfma(i32x8_t a, const Tokens<FMT>& b, floatx4_t c, int ea, int eb) {
  if constexpr (FMT == kE2M1) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b.v, c, 4, 4, J, ea, J, eb);
  } else {
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b.lo, c, 4, 0, J, ea, J, eb);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b.v, c, 4, 0, J, ea, J, eb);
  }
}

// The same of 32 features x 32 tokens and 64 columns.
template <int FMT, int J>
__device__ __forceinline__ floatx16_t mx_mfma32(i32x8_t a, const Tokens<FMT>& b, floatx16_t c, int ea, int eb) {
  if constexpr (FMT == kE2M1) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b.v, c, 4, 4, J, ea, J, eb);
  } else {
    c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b.lo, c, 4, 0, J, ea, J, eb);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b.v, c, 4, 0, J, ea, J, eb);
  }
}

// 2^t (1 + ln 2 lo), the power and its correction of t + lo in two parts.
__device__ __forceinline__ float exp2_parts(float t, float lo) {
  const float p = __builtin_amdgcn_exp2f(t);  // 1 ulp; results below 2^-126 are 0
  return p < INFINITY ? __builtin_fmaf(p, 0.6931471806f * lo, p) : p;
}
// v / (1 + e^-z); below z = -200 it is v / inf, above 200 v / 1.  Held on both sides: t of a z past fp32's largest / log2 e would be
// infinite, and its correction then NaN.
__device__ __forceinline__ float times_sigmoid(float v, float z) {
  constexpr float k1 = 1.442695041f, k2 = 1.925963033e-8f;  // log2 e
  const float x = -__builtin_amdgcn_fmed3f(z, -200.f, 200.f), t = x * k1;
  return v * __builtin_amdgcn_rcpf(1.f + exp2_parts(t, __builtin_fmaf(x, k2, __builtin_fmaf(x, k1, -t))));
}
// v erfc(-v / sqrt 2) / 2.  With x = |v| / sqrt 2, (1 + 2 x) e^(x^2) erfc x is smooth in q = (x - 2) / (x + 2) over all x
// (Shepherd and Laframboise 1981); the polynomial, a fit of degree 10, is within 6e-8, the result within 4e-7.
__device__ __forceinline__ float gelu_erf(float v) {
  constexpr float k1 = 0.7213475108f, k2 = 9.62981517e-9f;  // log2 e / 2
  constexpr float c[] = {0.000155460424f, -0.000183626486f, -0.00138272671f, 0.00104307686f, 0.00867822673f, -0.00794266723f,
                         -0.0542082563f, 0.164035827f, -0.166031525f, -0.0927630812f, 1.27697837f};
  const float a = fminf(__builtin_fabsf(v), 20.f), x = a * 0.7071067812f;
  const float q = __builtin_fmaf(-4.f, __builtin_amdgcn_rcpf(x + 2.f), 1.f);
  float r = c[0];
#pragma unroll
  for (int i = 1; i < 11; ++i) r = __builtin_fmaf(r, q, c[i]);
  const float h = a * a, l = __builtin_fmaf(a, a, -h), t = h * -k1;
  const float e = exp2_parts(t, __builtin_fmaf(l, -k1, __builtin_fmaf(h, -k2, __builtin_fmaf(h, -k1, -t))));
  const float tail = r * e * (0.5f * __builtin_amdgcn_rcpf(__builtin_fmaf(2.f, x, 1.f)));
  return v * (v < 0.f ? tail : 1.f - tail);
}

// N values activated under one look at the kind.  0.5 v (1 + tanh u) = v / (1 + e^-2u).  The forms above are short: the library's
// division, exp and erfc, 32 times over, are several KiB of instructions that a call fetches from memory (one row by 28672 x 8192
// with gelu_tanh 31.8 us, so 28.2), and tens of instructions an output (2048 rows by 22016 x 4096, none 122 us: gelu 174, so 152;
// silu 139, 130; on another card none 118, gelu 142, silu 122).
template <int N>
__device__ __forceinline__ void activate_all(int act, float (&v)[N]) {
  if (act == QGEMV_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = times_sigmoid(v[i], v[i]);
  } else if (act == QGEMV_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = times_sigmoid(v[i], v[i] * __builtin_fmaf(0.07135481627f, v[i] * v[i], 1.595769122f));
  } else if (act == QGEMV_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gelu_erf(v[i]);
  } else if (act == QGEMV_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // a NaN stays one
  }
}

// The lane's four features of one token.
__device__ __forceinline__ void put4(const EpiArg<true>& ep, int M, int T, int row, int t, floatx4_t s) {
  if (t >= T) return;
  float v[4], g[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ep.biased(s[i], min(row + i, M - 1));
  if (ep.gated) {
    g[0] = v[0], g[1] = v[2];
    activate_all(ep.act, g);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (row + 2 * i < M) ep.store(t, (row >> 1) + i, g[i] * v[2 * i + 1]);
  } else {
    activate_all(ep.act, v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row + i < M) ep.store(t, row + i, v[i]);
  }
}

// ---------------------------------------------------------------------------
// Few outputs: one token by any weights, or a few hundred by few features.  A workgroup takes RT tiles of features x NB
// tiles of tokens over all columns; its waves take the quads (512 columns) in turn, straight from
// memory into the operands' registers, and all of a quad's loads are on their way at once.  Their sums meet
// in LDS and are added in the waves' order.
//
// A CU takes in RT + NB KiB a chunk (E4M3: RT + 2 NB) for RT NB products, and the time goes with these once the weights' way
// from memory is not the longer one: 61 rows by 4096 x 11008 in 1 x 4 tiles 12.1 us, in 2 x 2, the tokens in two parts, 10.7
// (E4M3: 18.8, 14.8).  At some 50 GB/s a CU, 21 bytes a clock, what bounds it is no path's width but the loads' latency: a wave
// loads a quad, waits, multiplies, and only then loads its next one.
//
// ROWS 1, 2: x comes as FP16 or fp32 rows, kFusedRows at most, and a wave quantises its own
// quads' columns on the way: 8 columns a lane and token, the operands formed by way
// of LDS.  That saves the launch in front, and its 16 bits a value come from the L2.
// ---------------------------------------------------------------------------
template <int FMT, int RT, int NB>
constexpr int max_waves() {  // 16 have 128 registers each, 8 have 256
  return (RT + NB * (FMT ? 2 : 1)) * 16 + RT * NB * 4 > 100 ? 8 : 16;
}

constexpr int kFusedRows = 4;

template <int FMT>
struct QuadTokens {  // a wave's quantised quad: tokens' codes, then their exponents
  static constexpr int stride = FMT ? 528 : 272;  // bytes of a token, 16 of them for the banks
  static constexpr int exps = kFusedRows * stride;  // [block q][token] dwords
  static_assert(kFusedRows <= 16, "a tile");
  static constexpr int bytes = exps + 256;
};

template <int FMT, int RT, int NB, int ROWS>
__global__ void __launch_bounds__((64 * max_waves<FMT, RT, NB>()))
k_mx_stream(Side w, Side x, const void* rows, int64_t ldx, EpiArg<true> ep, int M, int T, int cols, int chunks, int quads, int parts) {
  constexpr int P = FMT ? 2 : 1;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6, n = lane & 15, kq = lane >> 4;
  // workgroups go to the eight XCDs in turn: those of the same features to one, whose L2 shares the weights
  const int seq = blockIdx.x >> 3, grp = seq / parts;
  const int a0 = (8 * grp + (blockIdx.x & 7)) * RT, b0 = (seq - grp * parts) * NB;
  if (a0 >= w.tiles) return;
  const uint8_t *pa[RT], *pb[NB];
  const int *ea[RT], *eb[NB];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t t = min(a0 + i, w.tiles - 1);
    pa[i] = w.codes + t * w.tile_bytes + 16 * lane;
    ea[i] = (const int*)(w.exps + t * quads * 256) + lane;
  }
  if constexpr (ROWS == 0) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      // tokens past the last read the last one's
      const int t = min(16 * (b0 + j) + n, T - 1);
      pb[j] = x.codes + (int64_t)(t >> 4) * x.tile_bytes + 256 * kq + 16 * (t & 15);
      eb[j] = (const int*)(x.exps + (int64_t)(t >> 4) * quads * 256) + 16 * kq + (t & 15);
    }
  }
  floatx4_t acc[RT][NB];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = (floatx4_t){0, 0, 0, 0};
  for (int q = wave; q < quads; q += waves) {
    // tokens first, which the L2 has sooner than memory the weights (22016 x 4096, 16 rows in E4M3: 13.0 us, last 13.4)
    int sb[NB];
    u32x4_t B[NB][4][P];
    if constexpr (ROWS == 0) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < P; ++e)
            B[j][c][e] = *(const u32x4_t*)(pb[j] + (int64_t)min(4 * q + c, chunks - 1) * (1024 * P) + 1024 * e);
        sb[j] = eb[j][q * 64];
      }
    }
    u32x4_t A[RT][4];
    int sa[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        A[i][c] = __builtin_nontemporal_load((const u32x4_t*)(pa[i] + (int64_t)min(4 * q + c, chunks - 1) * 1024));
      sa[i] = __builtin_nontemporal_load(ea[i] + q * 64);
    }
    if constexpr (ROWS != 0) {
      uint8_t* mine = lds + wave * QuadTokens<FMT>::bytes;
      const int col = 512 * q + 8 * lane;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 4
      for (int t = 0; t < T; ++t) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (col < cols) load8<ROWS == 2>(rows, t * ldx + col, v);
        uint32_t e[2];
        const uint32_t byte = mx_quad<FMT>(v, false, e);
        uint8_t* to = mine + t * QuadTokens<FMT>::stride;
        if constexpr (FMT == kE2M1) *(uint32_t*)(to + 4 * lane) = e[0];
        else *(u32x2_t*)(to + 8 * lane) = (u32x2_t){e[0], e[1]};
        // block b = lane / 4 of the quad: chunk b / 4, block b % 4
        if ((lane & 3) == 0) mine[QuadTokens<FMT>::exps + 64 * ((lane >> 2) & 3) + 4 * t + (lane >> 4)] = (uint8_t)byte;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const int t = min(n, T - 1);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < P; ++e)
          B[0][c][e] = *(const u32x4_t*)(mine + t * QuadTokens<FMT>::stride + 64 * P * c + 64 * e + 16 * kq);
      sb[0] = *(const int*)(mine + QuadTokens<FMT>::exps + 64 * kq + 4 * t);
    }
    auto step = [&](auto J) {
      constexpr int c = decltype(J)::value;
      if (4 * q + c >= chunks) return;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        i32x8_t b = {};
#pragma unroll
        for (int e = 0; e < 4 * P; ++e) b[e] = (int)B[j][c][e / 4][e % 4];
        const Tokens<FMT> tk = tokens<FMT>(b);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const i32x8_t a = {(int)A[i][c][0], (int)A[i][c][1], (int)A[i][c][2], (int)A[i][c][3], 0, 0, 0, 0};
          acc[i][j] = mx_mfma<FMT, c>(a, tk, acc[i][j], sa[i], sb[j]);
        }
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
  // [wave][tile][token tile][lane]
  floatx4_t* sums = (floatx4_t*)lds;
  if constexpr (ROWS != 0) __syncthreads();  // all waves are done with their tokens
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) sums[((wave * RT + i) * NB + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int at = wave; at < RT * NB; at += waves) {
    floatx4_t v = sums[at * 64 + lane];
    for (int k = 1; k < waves; ++k) v += sums[(k * RT * NB + at) * 64 + lane];
    put4(ep, M, T, (a0 + at / NB) * 16 + 4 * kq, (b0 + at % NB) * 16 + n, v);
  }
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup of four waves takes 64 AT features x 64 BT tokens, a wave
// a quarter of them, 32 AT x 32 BT, in AT BT results of sixteen registers.
//
// 32x32x64 MFMAs: with E2M1 on both sides they run at 6.2 to 6.7 PFLOP/s on random
// operands in registers (9.8 on zeros: the card's power decides), 16x16x128 at 4.4
// to 5.1.  Their operand of 32 rows and half a chunk is 256 contiguous bytes of two tiles each.
//
// Chunks move from memory into LDS past the registers, S steps of 128 columns
// ahead, as they are: a KiB a wave instruction; a wave's read of an operand is a KiB too,
// without bank conflicts.  Operands are read from LDS half a chunk ahead.  One
// barrier a chunk: behind it the next chunk has landed for all waves, and the place of the
// one whose operands all waves hold is free.
//
// 8192 rows by 28672 x 8192 among such calls: E2M1 900 to 920 us (4.2 PFLOP/s; MFMAs busy for 60 % of the cycles, at the 1.7 GHz
// that the card's power leaves of 2.4); 2048 rows 237 to 248, in E4M3 560 to 583, twice the MFMAs and their operands' split.  Alone,
// the caches clean, 917, 253 and 590; behind 256 MiB of writes, whose lines have to leave first, 1069, 285 and 698.
// Two workgroups a CU hide each other's waits: one of 256 x 256 outputs 959 us where two took 940, one that stays for all its
// tiles 970 (900); rings of 8 to 10 stages, and each workgroup's columns from another start, are no faster.
// ---------------------------------------------------------------------------
typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ rsrc_t resource(const uint8_t* p, int64_t bytes) {
  const uint32_t n = bytes > 0xFFFFFFF0ll ? 0xFFFFFFF0u : (uint32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, (int)n, 0x00020000);
}
__device__ __forceinline__ void to_lds(rsrc_t r, uint8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ int load_dword(rsrc_t r, int voff, int soff) {
  return (int)__builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
}
// s_waitcnt vmcnt(N) alone.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkm() { __builtin_amdgcn_s_waitcnt(0xC07F); }
__device__ __forceinline__ void wave_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Whether a lane's eight outputs (four when gated) can be stored, and their residuals loaded, 16 bytes or the whole at a time.
struct Whole {
  bool y, residual;
};

template <class V>
__device__ __forceinline__ void put_typed(void* y, int f32, int64_t e, V v) {
  constexpr int n = sizeof(V) / 4;
  if (f32) {
    *(V*)((float*)y + e) = v;
  } else {
    typedef _Float16 hv __attribute__((ext_vector_type(n)));
    *(hv*)((_Float16*)y + e) = __builtin_convertvector(v, hv);
  }
}

// A wave's 16 AT features x 16 NT tokens, at `s` in LDS token by token (stride 16 AT + 4), to y: a lane takes eight
// features of a token, U tokens at a time so that their reads and stores overlap.
template <int AT, int NT>
__device__ __forceinline__ void put_tile(const EpiArg<true>& ep, int M, int T, int row0, int t0, const float* s, int lane,
                                         Whole whole) {
  constexpr int LT = 2 * AT, RT = 64 / LT;  // lanes of a token, tokens of a round
  constexpr int U = 4;
  const int f = 8 * (lane % LT), row = row0 + f;
  if (row >= M) return;
  float bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = ep.bias ? ep.load(ep.bias, ep.bias32, min(row + i, M - 1)) : 0.f;
  const int mo = ep.gated ? M >> 1 : M, col = ep.gated ? row >> 1 : row;
  const int n = min(ep.gated ? 4 : 8, mo - col);
  const bool full = n == (ep.gated ? 4 : 8), full_y = full && whole.y, full_r = full && whole.residual;
#pragma unroll 1
  for (int i0 = lane / LT; i0 < 16 * NT && t0 + i0 < T; i0 += U * RT) {
    float g[U * 8];  // features, or gates
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* at = s + min(i0 + u * RT, 16 * NT - 1) * (16 * AT + 4) + f;
      const floatx4_t a = *(const floatx4_t*)at, b = *(const floatx4_t*)(at + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[8 * u + i] = a[i] + bias[i], g[8 * u + 4 + i] = b[i] + bias[4 + i];
    }
    if (ep.gated) {
      float h[U * 4];
#pragma unroll
      for (int i = 0; i < U * 4; ++i) h[i] = g[2 * i];
      activate_all(ep.act, h);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[8 * u + i] = h[4 * u + i] * g[8 * u + 2 * i + 1];
    } else {
      activate_all(ep.act, g);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RT, t = t0 + i;
      if (i >= 16 * NT || t >= T) continue;
      const int64_t e = t * ep.ldy + col, er = t * ep.ldr + col;
      if (ep.residual && full_r) {
        float r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (ep.res32) {
          const floatx4_t* from = (const floatx4_t*)((const float*)ep.residual + er);
          const floatx4_t x = from[0], z = ep.gated ? x : from[1];
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = x[k], r[4 + k] = z[k];
        } else if (ep.gated) {
          const half4_t x = *(const half4_t*)((const _Float16*)ep.residual + er);
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = (float)x[k];
        } else {
          const half8_t x = *(const half8_t*)((const _Float16*)ep.residual + er);
#pragma unroll
          for (int k = 0; k < 8; ++k) r[k] = (float)x[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) g[8 * u + k] += r[k];
      } else if (ep.residual) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < n) g[8 * u + k] += ep.load(ep.residual, ep.res32, er + k);
      }
      const floatx4_t a = {g[8 * u], g[8 * u + 1], g[8 * u + 2], g[8 * u + 3]};
      const floatx4_t b = {g[8 * u + 4], g[8 * u + 5], g[8 * u + 6], g[8 * u + 7]};
      if (full_y && ep.gated) {
        put_typed(ep.y, ep.y32, e, a);
      } else if (full_y && ep.y32) {
        put_typed(ep.y, 1, e, a);
        put_typed(ep.y, 1, e + 4, b);
      } else if (full_y) {
        *(half8_t*)((_Float16*)ep.y + e) = __builtin_convertvector(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7), half8_t);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < n) put_typed(ep.y, ep.y32, e + k, (floatx1_t){g[8 * u + k]});
      }
    }
  }
}

// The order of a half chunk's instructions: an LDS read (and, with VM, a copy) between every few MFMAs.  Left to itself the
// compiler moves the reads down to their use, and waits for each.
template <int READS, int MFMAS, int VM>
__device__ __forceinline__ void spread() {
  constexpr int per = MFMAS >= READS ? MFMAS / READS : 1;
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if constexpr (VM) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x8, per, 0);
  }
}

// Workgroups go to the eight XCDs in turn.  Each XCD takes a contiguous part of the tiles, in an order that walks four token
// tiles and then on to the next features: its 32 CUs are at work on some 4 x 8 tiles, whose operands its L2
// shares.
__device__ __forceinline__ void tile_of(int id, int tiles_a, int tiles_b, int& ta, int& tb) {
  const int n = tiles_a * tiles_b, q = n >> 3, r = n & 7, xcd = id & 7;
  const int t = xcd * q + min(xcd, r) + (id >> 3);
  const int per = 4 * tiles_a, grp = t / per, in = t - grp * per, width = min(4, tiles_b - 4 * grp);
  ta = in / width;
  tb = 4 * grp + in - ta * width;
}

template <int FMT, int AT, int BT, int S, int WG>
__global__ void __launch_bounds__(256, WG)
k_mx_tile(Side w, Side x, EpiArg<true> ep, int M, int T, int chunks, int quads, int tiles_a, int tiles_b, Whole whole) {
  constexpr int P = FMT ? 2 : 1;               // KiB of a token chunk
  constexpr int CA = 4 * AT, CB = 4 * BT * P;  // KiB of a stage
  constexpr int NL = (CA + CB) / 4;            // copies of a wave and stage
  constexpr int H = BT > 1 ? 2 : 1;            // the results leave by way of LDS in H parts
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int ta, tb;
  tile_of(blockIdx.x, tiles_a, tiles_b, ta, tb);
  const int wa = wave & 1, wb = wave >> 1;
  const int a0 = ta * 4 * AT, b0 = tb * 4 * BT;  // first tiles of 16
  const rsrc_t ra = resource(w.codes + a0 * w.tile_bytes, (w.tiles - a0) * w.tile_bytes);
  const rsrc_t rb = resource(x.codes + b0 * x.tile_bytes, (x.tiles - b0) * x.tile_bytes);
  // the wave's copies: NL consecutive KiB of the stage; tiles past the last are the last again
  int voff[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int c = wave * NL + i;
    voff[i] = c < CA ? min(c, w.tiles - 1 - a0) * (int)w.tile_bytes
                     : min((c - CA) / P, x.tiles - 1 - b0) * (int)x.tile_bytes + (c - CA) % P * 1024;
    voff[i] += 16 * lane;
  }
  auto stage = [&](int c) {
    uint8_t* to = lds + (c % S) * ((CA + CB) * 1024) + wave * (NL * 1024);
    const int cc = min(c, chunks - 1);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      if (wave * NL + i < CA) to_lds(ra, to + 1024 * i, voff[i], cc * 1024);
      else to_lds(rb, to + 1024 * i, voff[i], cc * (1024 * P));
    }
  };
  floatx16_t acc[AT][BT];
#pragma unroll
  for (int i = 0; i < AT; ++i)
#pragma unroll
    for (int j = 0; j < BT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // Lane 32 g + n of an operand holds row n of two tiles; its blocks are g and 2 + g of a chunk.
  const int tile = (lane >> 4) & 1, place = 16 * (lane & 15) + 256 * (lane >> 5);
  const rsrc_t xa = resource(w.exps + (int64_t)a0 * quads * 256, (int64_t)(w.tiles - a0) * quads * 256);
  const rsrc_t xb = resource(x.exps + (int64_t)b0 * quads * 256, (int64_t)(x.tiles - b0) * quads * 256);
  int oa[AT], ob[BT];
#pragma unroll
  for (int i = 0; i < AT; ++i) oa[i] = min(2 * (wa * AT + i) + tile, w.tiles - 1 - a0) * quads * 256 + (place >> 2);
#pragma unroll
  for (int j = 0; j < BT; ++j) ob[j] = min(2 * (wb * BT + j) + tile, x.tiles - 1 - b0) * quads * 256 + (place >> 2);
  int sa[2][AT], sb[2][BT], na[2][AT], nb[2][BT];
  auto exponents = [&](int q) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < AT; ++i) na[h][i] = load_dword(xa, oa[i] + 128 * h, q * 256);
#pragma unroll
      for (int j = 0; j < BT; ++j) nb[h][j] = load_dword(xb, ob[j] + 128 * h, q * 256);
    }
  };
  auto next_exponents = [&] {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < AT; ++i) sa[h][i] = na[h][i];
#pragma unroll
      for (int j = 0; j < BT; ++j) sb[h][j] = nb[h][j];
    }
  };
  u32x4_t fa[2][AT], fb[2][BT][P];
  const uint8_t* my_a = lds + (2 * wa * AT + tile) * 1024 + place;
  const uint8_t* my_b = lds + (CA + (2 * wb * BT + tile) * P) * 1024 + place;
  auto read = [&](int c, auto HH) {
    constexpr int h = decltype(HH)::value;
    const int at = (c % S) * ((CA + CB) * 1024);
#pragma unroll
    for (int i = 0; i < AT; ++i) fa[h][i] = *(const u32x4_t*)(my_a + at + 2048 * i + 512 * h);
#pragma unroll
    for (int j = 0; j < BT; ++j) {
      // E4M3: columns 16 g .. and 32 + 16 g .. of part h
      const uint8_t* p = my_b + at + 2048 * P * j + (P == 1 ? 512 : 1024) * h;
#pragma unroll
      for (int e = 0; e < P; ++e) fb[h][j][e] = *(const u32x4_t*)(p + 512 * e);
    }
  };
  auto multiply = [&](auto HH, auto J) {
    constexpr int h = decltype(HH)::value, jj = decltype(J)::value;
#pragma unroll
    for (int j = 0; j < BT; ++j) {
      i32x8_t b = {};
#pragma unroll
      for (int e = 0; e < 4 * P; ++e) b[e] = (int)fb[h][j][e / 4][e % 4];
      const Tokens<FMT> tk = tokens<FMT>(b);
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const u32x4_t v = fa[h][i];
        const i32x8_t a = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        acc[i][j] = mx_mfma32<FMT, jj>(a, tk, acc[i][j], sa[h][i], sb[h][j]);
      }
    }
  };
  typedef std::integral_constant<int, 0> I0;
  typedef std::integral_constant<int, 1> I1;
  typedef std::integral_constant<int, 2> I2;
  typedef std::integral_constant<int, 3> I3;
  // more: another quad follows, and its exponents are loaded.
  auto step = [&](auto J, int q, auto more) {
    constexpr int jj = decltype(J)::value;
    const int c = 4 * q + jj;
    __builtin_amdgcn_sched_barrier(0);
    read(c, I1{});
    multiply(I0{}, J);
    spread<AT + BT * P, AT * BT * P, 0>();
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<qmx_ring::may_be_on_the_way(S, NL, more ? 2 * (AT + BT) : 0, jj)>();  // the next chunk has landed
    wait_lgkm();  // the chunk's operands are in registers, its place is free for all behind the barrier
    wave_barrier();
    stage(c + S);
    if constexpr (jj == 0 && more) exponents(min(q + 1, quads - 1));
    read(c + 1, I0{});
    multiply(I1{}, J);
    spread<AT + BT * P, AT * BT * P, 1>();
  };
  exponents(0);
#pragma unroll
  for (int c = 0; c < S; ++c) stage(c);
  wait_vm<(S - 1) * NL>();
  wave_barrier();
  read(0, I0{});
  const int full = chunks >> 2, left = chunks & 3;
  for (int q = 0; q < full; ++q) {
    next_exponents();
    step(I0{}, q, std::true_type{});
    step(I1{}, q, std::true_type{});
    step(I2{}, q, std::true_type{});
    step(I3{}, q, std::true_type{});
  }
  if (left) {
    next_exponents();
    step(I0{}, full, std::false_type{});
    if (left > 1) step(I1{}, full, std::false_type{});
    if (left > 2) step(I2{}, full, std::false_type{});
  }
  wait_vm<0>();  // copies past the end
  wait_lgkm();
  wave_barrier();
  // Lane 32 g + n of a result holds features 8 u + 4 g .. + 3, u = 0 .. 3, of token n.
  float* mine = (float*)lds + wave * (32 * BT / H * (32 * AT + 4));
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int j = 0; j < BT / H; ++j)
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const floatx16_t& r = acc[i][h * (BT / H) + j];
          *(floatx4_t*)(mine + (32 * j + (lane & 31)) * (32 * AT + 4) + 32 * i + 8 * u + 4 * (lane >> 5)) =
              (floatx4_t){r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]};
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    put_tile<2 * AT, 2 * BT / H>(ep, M, T, (a0 + 2 * wa * AT) * 16, (b0 + 2 * wb * BT + h * (2 * BT / H)) * 16, mine, lane, whole);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// ---- host side ----------------------------------------------------------------
int hip_status(hipError_t e) {
  if (e == hipSuccess) return QGEMV_OK;
  qgemv_set_hip_error((int)e);
  return QGEMV_ERR_HIP;
}

int check_shape(const qmx_shape* s) {
  if (!s) return QGEMV_ERR_INVALID_ARG;
  if (s->rows < 0 || s->cols < 1) return QGEMV_ERR_INVALID_ARG;
  if (s->rows > kMaxRows || s->cols > kMaxCols || s->cols % 32) return QGEMV_ERR_UNSUPPORTED;
  if (s->format != QMX_E2M1 && s->format != QMX_E4M3) return QGEMV_ERR_UNSUPPORTED;
  const Geo g = geo(s->rows, s->cols, s->format);
  // a wave a chunk, and fewer than 2^32 threads a launch
  if ((int64_t)g.tiles * g.chunks > (1 << 26) - 4) return QGEMV_ERR_UNSUPPORTED;
  return QGEMV_OK;
}

int check_rows(const void* x, int type, int64_t ldx) {
  if (!x || (uintptr_t)x % 16 || ldx % 8) return QGEMV_ERR_INVALID_ARG;
  if (type != QGEMV_F16 && type != QGEMV_F32) return QGEMV_ERR_UNSUPPORTED;
  return QGEMV_OK;
}

bool bad_blocks(const void* p) { return !p || (uintptr_t)p % 256; }

Side side(const void* blocks, const Geo& g) {
  return Side{(const uint8_t*)blocks, (const uint8_t*)blocks + g.exps, g.tile_bytes, g.tiles};
}

hipError_t launch_quantize(const Geo& g, void* blocks, const void* x, int type, int64_t ldx, int clip, hipStream_t st) {
  const int total = g.tiles * g.chunks;
  auto go = [&](auto k) { hipLaunchKernelGGL(k, dim3((total + 3) / 4), dim3(256), 0, st, (uint8_t*)blocks, g, x, ldx, clip, total); };
  if (g.fmt == QMX_E2M1) type == QGEMV_F32 ? go(k_mx_quantize<kE2M1, true>) : go(k_mx_quantize<kE2M1, false>);
  else type == QGEMV_F32 ? go(k_mx_quantize<kE4M3, true>) : go(k_mx_quantize<kE4M3, false>);
  return hipGetLastError();
}

// Rows that the stream kernel quantises on the way: every workgroup does so for itself, where a launch in front takes 3 us (and
// as much of the host's time).  us, weights from memory, E2M1 | E4M3 rows:
//   4096 x 4096    1 row 5.4 | 6.0    4 rows  6.9 |  7.6    16 rows (two launches)  9.5 | 10.6
//   28672 x 8192   1 row 23.9 | 25.6  4 rows 25.6 | 27.5    16 rows (two launches) 29.8 | 31.3
// From some 8 rows on the launch is the shorter way.  us, E2M1, on the way | two launches:
//   4096 x 4096    5 rows  6.9 |  7.5   8 rows  9.0 |  8.2   16 rows 12.3 |  9.4
//   28672 x 8192                        8 rows 29.9 | 29.7   16 rows 40.0 | 31.5
bool fused_rows(int T, int x_type) { return x_type != QMX_IN_BLOCKS && T <= kFusedRows; }

struct RunPlan {
  Geo gw, gx;
  size_t bytes;  // workspace: x in blocks
};

int run_plan(const qmx_shape* w, const qmx_input* x, const qgemv_epilogue* e, RunPlan& p) {
  int st = check_shape(w);
  if (st) return st;
  if (!x || !e || w->rows < 1) return QGEMV_ERR_INVALID_ARG;
  if (w->format != QMX_E2M1) return QGEMV_ERR_UNSUPPORTED;
  const qmx_shape xs = {x->rows, w->cols, x->format};
  if ((st = check_shape(&xs))) return st;
  if (x->x_type != QMX_IN_BLOCKS && x->x_type != QGEMV_F16 && x->x_type != QGEMV_F32) return QGEMV_ERR_UNSUPPORTED;
  p.gw = geo(w->rows, w->cols, w->format);
  p.gx = geo(x->rows, w->cols, x->format);
  // the smallest tiles' workgroups, fewer than 2^32 threads a launch
  if ((int64_t)((p.gw.tiles + 3) / 4) * ((p.gx.tiles + 3) / 4) >= 1 << 24) return QGEMV_ERR_UNSUPPORTED;
  p.bytes = x->x_type == QMX_IN_BLOCKS || fused_rows(x->rows, x->x_type) ? 0 : (size_t)p.gx.bytes;
  return QGEMV_OK;
}

Whole whole_rows(const EpiArg<true>& ep) {
  auto whole = [&](const void* p, int64_t ld, int f32) {
    const int n = ep.gated || f32 ? 4 : 8, size = f32 ? 4 : 2;
    return ld % n == 0 && (uintptr_t)p % (n * size) == 0;
  };
  return Whole{whole(ep.y, ep.ldy, ep.y32), whole(ep.residual, ep.ldr, ep.res32)};
}

constexpr int kLdsBytes = 160 * 1024;

template <int FMT, int AT, int BT, int S, int WG>
hipError_t launch_tile(const RunPlan& p, const Side& a, const Side& b, const EpiArg<true>& ep, hipStream_t st) {
  constexpr int ring = S * (4 * AT + 4 * BT * (FMT ? 2 : 1)) * 1024, out = 4 * (BT > 1 ? 16 * BT : 32) * (32 * AT + 4) * 4;
  constexpr int lds = ring > out ? ring : out;
  const int na = (a.tiles + 4 * AT - 1) / (4 * AT), nb = (b.tiles + 4 * BT - 1) / (4 * BT);
  auto k = k_mx_tile<FMT, AT, BT, S, WG>;
  // once per instantiation (thread-safe static initialisation)
  static const hipError_t attr = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(k, dim3(na * nb), dim3(256), lds, st, a, b, ep, p.gw.rows, p.gx.rows, p.gw.chunks, p.gw.quads, na, nb,
                     whole_rows(ep));
  return hipGetLastError();
}

template <int FMT, int RT, int NB, int ROWS>
hipError_t launch_stream(const RunPlan& p, const Side& a, const Side& b, const EpiArg<true>& ep, const qmx_input* x, hipStream_t st) {
  // as many waves as share the quads evenly
  constexpr int most = max_waves<FMT, RT, NB>();
  const int rounds = (p.gw.quads + most - 1) / most, waves = (p.gw.quads + rounds - 1) / rounds;
  const int sums = waves * RT * NB * 1024, tokens = ROWS ? waves * QuadTokens<FMT>::bytes : 0;
  const int lds = sums > tokens ? sums : tokens;
  const int groups = ((a.tiles + RT - 1) / RT + 7) / 8, parts = ROWS ? 1 : (b.tiles + NB - 1) / NB;
  auto k = k_mx_stream<FMT, RT, NB, ROWS>;
  static const hipError_t attr = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(k, dim3(8 * groups * parts), dim3(64 * waves), lds, st, a, b, x->data, x->ldx, ep, p.gw.rows,
                     p.gx.rows, p.gw.cols, p.gw.chunks, p.gw.quads, parts);
  return hipGetLastError();
}

// Tiles of features a workgroup takes: as few as let the card hold all workgroups at once, counted as sixteen waves a CU; a second
// round costs a whole round's time, and many tiles a workgroup little, since tokens are read once for all of them.  us, 16 rows:
//   256 tiles x 4096 columns, E2M1    1 tile  5.5   2 tiles  6.3   3 tiles  7.2
//   1376 x 4096, E4M3                 2 tiles 15.4  3 tiles 13.8   4 tiles 17.2   7 tiles 14.1
//   1792 x 8192, E4M3                 2 tiles 36.6  3 tiles 33.7   4 tiles 29.7   7 tiles 28.1
// The count is not so for kernels of more than 128 registers (max_waves: 7 tiles, and 4 in E4M3), of which a CU holds eight
// waves, and 5 and 6 tiles, which take 7, are not built.  What that costs: 1792 x 4096 in E4M3 17.6 us by the rule's 4 tiles, 16.1
// by 7; 1280 x 8192 by the rule's 7 for 5 tiles 23.4 us in E2M1 and 21.8 in E4M3, by 5 19.8 and 20.5.
template <int FMT, int ROWS>
hipError_t stream_by_tiles(const RunPlan& p, const Side& a, const Side& b, const EpiArg<true>& ep, const qmx_input* x,
                           hipStream_t st) {
  const int at_once = 256 * (p.gw.quads >= 16 ? 1 : 16 / p.gw.quads), rt = (a.tiles + at_once - 1) / at_once;
  if (rt <= 1) return launch_stream<FMT, 1, 1, ROWS>(p, a, b, ep, x, st);
  if (rt <= 2) return launch_stream<FMT, 2, 1, ROWS>(p, a, b, ep, x, st);
  if (rt <= 3) return launch_stream<FMT, 3, 1, ROWS>(p, a, b, ep, x, st);
  if (rt <= 4) return launch_stream<FMT, 4, 1, ROWS>(p, a, b, ep, x, st);
  return launch_stream<FMT, 7, 1, ROWS>(p, a, b, ep, x, st);
}

// Kernel and tiles of the least time by a model, in us.
//
// The stream kernel: 2.8 for the call, then as many times as workgroups are a CU what their operands take, KiB by KiB, or
// the weights' way from memory at 4.4 TB/s.  Past 4096 workgroups it is out of the question.
//
// The tile kernel: `call`, and as many times as workgroups are a CU `end` and `chunk` a chunk, or `alone` a chunk, which one
// workgroup takes whose CU waits for its copies.
//
// Fits to 17 to 4096 rows by 1024 x 4096 to 28672 x 8192 with weights from memory (202 products in two formats, each by up to ten
// of these shapes): the choice is 0.5 % slower than the fastest on average, 15 % at most.  us, stream | tile, the best tiles of each:
//   E2M1   64 rows  4096 x 11008: 10.6 | 19.5    8192 x 8192: 13.0 | 16.2   22016 x 4096: 20.8 | 13.6
//         256 rows  1024 x  4096:  6.1 |  8.3    4096 x 4096: 13.5 |  8.7
//   E4M3   64 rows  4096 x 11008: 14.8 | 35.8    8192 x 8192: 17.1 | 28.3   22016 x 4096: 27.7 | 19.5
//         256 rows  1024 x  4096:  7.5 | 16.2    4096 x 4096: 17.7 | 16.7
struct TileCost {
  int features, tokens;
  float call, alone, chunk, end;
};
struct Choice {
  int kernel;  // 0: stream, RT = a, NB = b; 1: tile, shape a
  int a, b;
};
template <int FMT>
Choice best_choice(int M, int T, int chunks) {
  static const TileCost e2m1[] = {{64, 64, 4.0f, 0.17f, 0.13f, 0.7f}, {128, 64, 4.0f, 0.235f, 0.205f, 0.9f},
                                  {128, 128, 4.0f, 0.32f, 0.28f, 1.6f}, {128, 256, 3.6f, 0.5f, 0.51f, 2.8f}};
  static const TileCost e4m3[] = {{64, 64, 4.5f, 0.375f, 0.27f, 0.6f}, {128, 64, 4.6f, 0.43f, 0.41f, 0.2f},
                                  {256, 128, 5.8f, 1.2f, 1.2f, 1.5f}};
  auto of_cu = [&](int64_t features, int64_t tokens) {
    const int64_t n = ((M + features - 1) / features) * ((T + tokens - 1) / tokens);
    return (float)((n + 255) / 256);
  };
  Choice best = {1, 0, 0};
  float least = 0.f;
  for (int i = 0; i < (FMT ? 3 : 4); ++i) {
    const TileCost& c = (FMT ? e4m3 : e2m1)[i];
    const float share = of_cu(c.features, c.tokens) * (chunks * c.chunk + c.end), alone = chunks * c.alone;
    const float t = c.call + (share > alone ? share : alone);
    if (i == 0 || t < least) least = t, best = {1, i, 0};
  }
  for (int rt = 1; rt <= 4; ++rt)
    for (int nb = 1; nb <= 2; ++nb) {
      const float n = of_cu(16 * rt, 16 * nb);
      if (n > 16.f) continue;
      const float operands = n * (rt + (FMT ? 2 : 1) * nb) * (0.2f + 0.0204f * chunks);
      const float weights = (float)M * chunks * (68.f / 4.4e6f);
      const float t = 2.8f + (operands > weights ? operands : weights);
      if (t < least) least = t, best = {0, rt, nb};
    }
  return best;
}

template <int FMT>
hipError_t launch_product(const RunPlan& p, const Side& a, const Side& b, const EpiArg<true>& ep, const qmx_input* x,
                          hipStream_t st) {
  const int M = p.gw.rows, T = p.gx.rows;
  if (fused_rows(T, x->x_type))
    return x->x_type == QGEMV_F32 ? stream_by_tiles<FMT, 2>(p, a, b, ep, x, st) : stream_by_tiles<FMT, 1>(p, a, b, ep, x, st);
  // 16 rows are the weights' way from memory, which the stream kernel's loads take past the caches.  28672 x 8192, E2M1, 1 row, us,
  // stream | tile: 25.9 | 24.6 among such calls, but 26.5 | 47 where the caches hold lines that have to be written back first;
  // 22016 x 4096 11.8 | 12.7; E4M3, 16 rows 26.7 | 33
  if (T <= 16) return stream_by_tiles<FMT, 0>(p, a, b, ep, x, st);
  const Choice c = best_choice<FMT>(M, T, p.gw.chunks);
  if (c.kernel == 0) {
    switch (2 * c.a + c.b) {
      case 3: return launch_stream<FMT, 1, 1, 0>(p, a, b, ep, x, st);
      case 4: return launch_stream<FMT, 1, 2, 0>(p, a, b, ep, x, st);
      case 5: return launch_stream<FMT, 2, 1, 0>(p, a, b, ep, x, st);
      case 6: return launch_stream<FMT, 2, 2, 0>(p, a, b, ep, x, st);
      case 7: return launch_stream<FMT, 3, 1, 0>(p, a, b, ep, x, st);
      case 8: return launch_stream<FMT, 3, 2, 0>(p, a, b, ep, x, st);
      case 9: return launch_stream<FMT, 4, 1, 0>(p, a, b, ep, x, st);
      default: return launch_stream<FMT, 4, 2, 0>(p, a, b, ep, x, st);
    }
  }
  if (c.a == 0) return launch_tile<FMT, 1, 1, FMT ? 5 : 8, 2>(p, a, b, ep, st);
  if (c.a == 1) return launch_tile<FMT, 2, 1, FMT ? 4 : 5, 2>(p, a, b, ep, st);
  if constexpr (FMT == kE4M3) {
    return launch_tile<FMT, 4, 2, 2, 2>(p, a, b, ep, st);
  } else {
    if (c.a == 2) return launch_tile<FMT, 2, 2, 4, 2>(p, a, b, ep, st);
    return launch_tile<FMT, 2, 4, 3, 2>(p, a, b, ep, st);
  }
}

}  // namespace

extern "C" {

int qmx_bytes(const qmx_shape* shape, size_t* bytes) {
  const int st = check_shape(shape);
  if (st) return st;
  if (!bytes) return QGEMV_ERR_INVALID_ARG;
  *bytes = (size_t)geo(shape->rows, shape->cols, shape->format).bytes;
  return QGEMV_OK;
}

int qmx_quantize(const qmx_shape* shape, void* blocks, const void* x, int32_t x_type, int64_t ldx, int32_t clip,
                 void* stream) {
  int st = check_shape(shape);
  if (st || shape->rows == 0) return st;
  if (bad_blocks(blocks)) return QGEMV_ERR_INVALID_ARG;
  if ((st = check_rows(x, x_type, ldx))) return st;
  return hip_status(launch_quantize(geo(shape->rows, shape->cols, shape->format), blocks, x, x_type, ldx, clip != 0,
                                    (hipStream_t)stream));
}

int qmx_values(const qmx_shape* shape, const void* blocks, void* x, int32_t x_type, int64_t ldx, void* stream) {
  int st = check_shape(shape);
  if (st || shape->rows == 0) return st;
  if (bad_blocks(blocks)) return QGEMV_ERR_INVALID_ARG;
  if ((st = check_rows(x, x_type, ldx))) return st;
  if (shape->rows > 1 && ldx < shape->cols) return QGEMV_ERR_INVALID_ARG;
  const Geo g = geo(shape->rows, shape->cols, shape->format);
  const int total = g.tiles * g.chunks;
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, dim3((total + 3) / 4), dim3(256), 0, (hipStream_t)stream, (const uint8_t*)blocks, g, x, ldx, total);
  };
  if (g.fmt == QMX_E2M1) x_type == QGEMV_F32 ? go(k_mx_values<kE2M1, true>) : go(k_mx_values<kE2M1, false>);
  else x_type == QGEMV_F32 ? go(k_mx_values<kE4M3, true>) : go(k_mx_values<kE4M3, false>);
  return hip_status(hipGetLastError());
}

static int plain(const qmx_shape* shape, const void* blocks, const void* codes, const void* exponents, bool pack,
                 void* stream) {
  const int st = check_shape(shape);
  if (st || shape->rows == 0) return st;
  if (bad_blocks(blocks) || !codes || (uintptr_t)codes % 16 || !exponents) return QGEMV_ERR_INVALID_ARG;
  const Geo g = geo(shape->rows, shape->cols, shape->format);
  const int total = g.tiles * g.chunks;
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, dim3((total + 3) / 4), dim3(256), 0, (hipStream_t)stream, (uint8_t*)blocks, g, (uint8_t*)codes,
                       (uint8_t*)exponents, total);
  };
  if (g.fmt == QMX_E2M1) pack ? go(k_mx_plain<kE2M1, true>) : go(k_mx_plain<kE2M1, false>);
  else pack ? go(k_mx_plain<kE4M3, true>) : go(k_mx_plain<kE4M3, false>);
  return hip_status(hipGetLastError());
}

int qmx_pack(const qmx_shape* shape, void* blocks, const void* codes, const void* exponents, void* stream) {
  return plain(shape, blocks, codes, exponents, true, stream);
}

int qmx_unpack(const qmx_shape* shape, const void* blocks, void* codes, void* exponents, void* stream) {
  return plain(shape, blocks, codes, exponents, false, stream);
}

int qmx_run_ws(const qmx_shape* w, const qmx_input* x, const qgemv_epilogue* e, size_t* bytes) {
  RunPlan p;
  const int st = run_plan(w, x, e, p);
  if (st) return st;
  if (!bytes) return QGEMV_ERR_INVALID_ARG;
  *bytes = p.bytes;
  return QGEMV_OK;
}

int qmx_run(const qmx_shape* w, const void* w_blocks, const qmx_input* x, void* y, const qgemv_epilogue* e, void* ws,
            size_t ws_bytes, void* stream) {
  RunPlan p;
  int st = run_plan(w, x, e, p);
  if (st || x->rows == 0) return st;
  if (bad_blocks(w_blocks) || !y) return QGEMV_ERR_INVALID_ARG;
  EpiArg<true> ep;
  if ((st = fill_epilogue(w->rows, y, e, ep))) return st;
  // the residual at y: each lane then has to store where it loaded
  if (ep.residual == y && (ep.res32 != ep.y32 || (x->rows > 1 && ep.ldr != ep.ldy))) return QGEMV_ERR_INVALID_ARG;
  const void* xb = x->data;
  if (x->x_type == QMX_IN_BLOCKS) {
    if (bad_blocks(xb)) return QGEMV_ERR_INVALID_ARG;
  } else if ((st = check_rows(xb, x->x_type, x->ldx))) {
    return st;
  }
  if (p.bytes > 0 && (!ws || (uintptr_t)ws % 256)) return QGEMV_ERR_INVALID_ARG;
  if (ws_bytes < p.bytes) return QGEMV_ERR_SIZE;
  const hipStream_t s = (hipStream_t)stream;
  if (p.bytes > 0) {
    const hipError_t er = launch_quantize(p.gx, ws, xb, x->x_type, x->ldx, 0, s);
    if (er != hipSuccess) return hip_status(er);
    xb = ws;
  }
  const Side a = side(w_blocks, p.gw), b = side(xb, p.gx);
  return hip_status(p.gx.fmt == QMX_E2M1 ? launch_product<kE2M1>(p, a, b, ep, x, s) : launch_product<kE4M3>(p, a, b, ep, x, s));
}
}  // extern "C"
