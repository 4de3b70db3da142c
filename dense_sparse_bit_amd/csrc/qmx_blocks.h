// qmx_blocks.h -- MX blocks on the device: a block's power of two and its
// elements (include/qmx.h, storage in qmx_layout.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmx_dev {

constexpr int kE2M1 = 0, kE4M3 = 1;

// Exponent byte of a block from the bits of its largest magnitude (255: not finite).  6 = 1.5 2^2, 448 = 1.75 2^8.
template <int FMT>
__device__ __forceinline__ uint32_t mx_exponent(uint32_t top, bool clip) {
  constexpr int emax = FMT == kE2M1 ? 2 : 8;
  constexpr uint32_t over = FMT == kE2M1 ? 0x400000u : 0x600000u;
  int b = (int)(top >> 23) - emax;
  if (!clip && (top & 0x7FFFFFu) > over) ++b;
  return top >= 0x7F800000u ? 255u : (uint32_t)max(b, 1);
}
// 2^-e as a factor: exact, since 1 <= byte <= 253 makes it a normal number.  A NaN block's elements are zeros.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == 255 ? 0.f : __uint_as_float((254u - byte) << 23);
}
// The value of an exponent byte.
__device__ __forceinline__ float mx_step(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// Byte offset in a chunk of the 8 elements of row r (of 16), columns 8 c .. + 7 of the chunk.
template <int FMT>
__device__ __forceinline__ int lane_bytes(int r, int c) {
  return FMT == kE2M1 ? 16 * (16 * (c >> 2) + r) + 4 * (c & 3) : 1024 * (c >> 3) + 16 * (16 * ((c >> 1) & 3) + r) + 8 * (c & 1);
}

// Four values times 2^-e in E4M3.  The conversion rounds to nearest even; what lies above the largest is held at it
// beforehand.
__device__ __forceinline__ uint32_t mx_four_e4m3(float a, float b, float c, float d) {
  auto in = [](float v) { return __builtin_amdgcn_fmed3f(v, -448.f, 448.f); };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(in(a), in(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(in(c), in(d), w, true);
}
// Eight values times 2^-e in E2M1: nearest even, saturating.
__device__ __forceinline__ uint32_t mx_eight_e2m1(const float* v) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.f, 3);
}

// The largest |v| of a quad of neighbouring lanes, as bits (order of magnitudes, not finite at the top).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false));  // i ^ 1
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, false));  // i ^ 2
}

// A quad of neighbouring lanes holds a block, 8 values each: the lane's elements (one dword of E2M1, two of E4M3) and
// the block's byte.
template <int FMT>
__device__ __forceinline__ uint32_t mx_quad(const float (&v)[8], bool clip, uint32_t (&w)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const uint32_t byte = mx_exponent<FMT>(quad_max(top), clip);
  const float inv = mx_inverse(byte);
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = byte == 255 ? 0.f : v[i] * inv;
  if constexpr (FMT == kE2M1) {
    w[0] = mx_eight_e2m1(u);
  } else {
    w[0] = mx_four_e4m3(u[0], u[1], u[2], u[3]);
    w[1] = mx_four_e4m3(u[4], u[5], u[6], u[7]);
  }
  return byte;
}

}  // namespace qmx_dev
