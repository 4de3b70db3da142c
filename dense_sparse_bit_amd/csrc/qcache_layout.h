// qcache_layout.h -- the 4-bit key/value cache as the kernels hold it.
//
// cache = [page][head][unit of 16 tokens].  A unit holds the keys and values
// of 16 consecutive positions of one head, with D = head_dim dimensions in
// NG = D / group groups (halves are FP16):
//
//   offset            bytes
//   0                 8 D     key codes     [lane 64][D/32 dwords]
//   8 D               8 D     value codes   [lane 64][D/32 dwords]
//   16 D              32 NG   key steps s   [kq 4][NG][4 tokens] halves
//   16 D + 32 NG      32 NG   key lowests   [16 tokens][NG] halves
//   16 D + 64 NG      64 NG   value stats   [kq 4][NG][s of 4 tokens, lo of 4 tokens] halves
//
// Key codes are the A operands of the score product K q (16x16x32 MFMAs, rows
// = tokens): lane 16 kq + t holds token t, and its dword g the dimensions
// 32 g + 8 kq .. + 7, one A operand of step g.  Dimension 2 i + e of the eight
// sits in nibble i + 4 e, so (w >> 4 i) & 0x000f000f is the pair (2i, 2i + 1).
//
// Value codes are the A operands of V^T p (rows = dimensions, the MFMA's K
// axis = tokens): lane 16 kq + m holds tokens 4 kq .. + 3 and dimensions
// m D/16 .. + D/16 - 1; its dword [tp][c] (tp = 0, 1; c = 0 .. D/64 - 1) the
// token pair 4 kq + 2 tp + e and the dimensions m D/16 + 4 c + i, in nibble
// i + 4 e, so (w >> 4 i) & 0x000f000f is one dimension of two tokens.  The
// tokens 4 kq .. + 3 are also those whose scores lane 16 kq + n of the score
// product's result holds, so the weights go into the second product without
// leaving their lanes.
//
// A token's codes are whole dwords (keys) or 16-bit halves of dwords (values):
// writing one token touches no other token's bytes.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qcache_layout {

constexpr int kUnit = 16;    // tokens of a unit
constexpr int kBlock = 128;  // tokens a workgroup of four waves takes at a time

template <int D, int NG>
struct Geo {
  static constexpr int G = D / NG;
  static constexpr int ND = D / 32;  // dwords of a lane, score-product steps
  static constexpr int NC = D / 64;  // dwords of a lane and token pair
  static constexpr int off_v = 8 * D;
  static constexpr int off_ks = 16 * D;
  static constexpr int off_kl = 16 * D + 32 * NG;
  static constexpr int off_vs = 16 * D + 64 * NG;
  static constexpr int bytes = 16 * D + 128 * NG;
};

inline size_t unit_bytes(int D, int G) { return 16 * (size_t)D + 128 * (size_t)(D / G); }

}  // namespace qcache_layout
