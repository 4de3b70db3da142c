// qnorm_sums.h -- where the sums over a row's waves lie in LDS.
//
// For a sum each wave writes its part, one barrier follows, and every wave reads
// all parts.  A fast wave may be at the next sum while a slow one still reads the
// last, with no barrier between the two, so consecutive sums lie in different
// halves; the next but one is behind a barrier that the slow wave has passed. The halves
// are counted in bytes, since the sums of one row may be of different types.
#pragma once

namespace qnorm_sums {

constexpr int kWaves = 16;         // of a row, at most
constexpr int kHalf = kWaves * 8;  // bytes of a sum: parts of up to 64 bits
constexpr int kBytes = 2 * kHalf;

// Byte offset of the sum that follows the one at `at`; 0 before the first.
constexpr int next(int at) { return at ^ kHalf; }

}  // namespace qnorm_sums
