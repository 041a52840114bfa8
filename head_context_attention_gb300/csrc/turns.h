// turns.h -- frequencies as fractions of a turn in 64-bit fixed point.
//
// An angle position * inv_freq in turns, modulo 1, is the product modulo 2^64 of
// the position and turn_fraction(inv_freq): exact but for the fraction's own
// error, which the position multiplies.  That is the rounding of inv_freq / (2 pi)
// in a double, below 2^-52 of inv_freq, and the cut at 64 bits, below 2^-64 turn:
//   |position| (|inv_freq| 2^-52 + 2 pi 2^-64) radians.
// The top 32 bits as fp32 half turns add 2 pi 2^-32 and pi 2^-25, below 2^-23.
#pragma once

#include <stdint.h>

#include <cmath>

namespace loong {

// inv_freq / (2 pi) modulo 1.  A negative frequency is the other sense of its
// positive one: taking the fraction of a small negative number in a double would
// leave it 53 bits of a turn.
inline uint64_t turn_fraction(double inv_freq) {
  double t = std::fabs(inv_freq) / 6.283185307179586476925;
  t -= std::floor(t);
  const double hi = std::floor(t * 4294967296.0);
  const double lo = (t * 4294967296.0 - hi) * 4294967296.0;  // exact: powers of two
  const uint64_t f = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo);
  return inv_freq < 0 ? 0 - f : f;
}

}  // namespace loong
