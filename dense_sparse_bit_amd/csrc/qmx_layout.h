// qmx_layout.h -- rows in MX blocks as the kernels hold them.
//
// Rows form tiles of 16, columns chunks of 128 (the last one padded with zeros).
// A chunk of a tile is one operand of a 16x16x128 scaled MFMA, as its 64 lanes
// take it:
//
//   E2M1   lane 16 q + r holds columns 32 q .. + 31 of row r: one MX block
//   E4M3   lane 16 q + r holds columns 16 q .. + 15 (part 0) and 64 + 16 q .. + 15 (part 1) of row r
//
//   codes      [tile][chunk][part][lane 64][16 bytes]   1 part for E2M1, 2 for E4M3
//   exponents  [tile][quad of 4 chunks][lane 64][4 bytes]   lane 16 q + r: block q of row r; byte j: chunk 4 quad + j
//
// So a wave's load of an operand is one contiguous KiB, also by way of LDS, and
// one dword a lane holds the exponents of four MFMAs, whose instruction
// selects the byte.  Rows past the last are whatever the memory held; columns
// past the last are zeros with exponent byte 1.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qmx_layout {

constexpr int kMaxRows = 1 << 26;
constexpr int kMaxCols = 1 << 20;

struct Geo {
  int rows, cols, fmt;
  int tiles, chunks, quads;
  int64_t tile_bytes;  // codes of a tile
  int64_t exps;        // offset of the exponents
  int64_t bytes;
};

inline Geo geo(int rows, int cols, int fmt) {
  Geo g;
  g.rows = rows, g.cols = cols, g.fmt = fmt;
  g.tiles = (rows + 15) / 16;
  g.chunks = (cols + 127) / 128;
  g.quads = (g.chunks + 3) / 4;
  g.tile_bytes = (int64_t)g.chunks * (fmt ? 2048 : 1024);
  g.exps = g.tiles * g.tile_bytes;
  g.bytes = g.exps + (int64_t)g.tiles * g.quads * 256;
  return g;
}

}  // namespace qmx_layout
