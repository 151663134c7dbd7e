// rope_rates.h -- the rotary embedding's rates as 64-bit fractions of a turn
// (host code).
#pragma once
#include <math.h>
#include <stdint.h>

namespace oq {

// Turns per position of each pair, theta^(-2 i / size) / 2 pi <= 1 / 2 pi
// (theta >= 1), in units of 2^-64, and the pair's axis.  Exponentials for
// every 16th pair, a product a pair between, for a small part of the
// exponentials' time.
//
// Error in units of 2^-64, with rates below 0.16 2^64 and extended precision
// (a half step of 0.125 there, functions to one step of theirs): 15 products
// 15 x 0.125; the ratio's own error, at most 2^-64 / r, grows with the number
// of products j as j r^(j-1): 15 x 0.16; the exponential, its argument and the
// unit 0.16 x (2 + 3 x 0.37 + 3); the rounding to whole units 0.5: together
// below 6.  At a position of 2^31 that is 6 x 2^-33 of a turn, with the
// kernel's rounding of the fraction (2^-33) below 2^-30.  (The largest found
// over 14 theta from 1 to 1e12 and every size to 504: 2.4 units, 2^-31.2.)
inline void rope_rates(double theta, int axes, const int *axis_dims, uint64_t *freq, uint8_t *axis) {
  int j = 0;
  const long double log_theta = logl((long double)theta), unit64 = 0x1p64L / (2 * acosl(-1.0L));
  for (int i = 0; i < axes; i++) {
    if (axis_dims[i] == 0) continue;
    const long double rate = log_theta / axis_dims[i], ratio = expl(-2 * rate);
    long double f = unit64;
    for (int k = 0; k < axis_dims[i]; k += 2, j++) {
      if (k % 32 == 0) f = expl(-k * rate) * unit64;
      freq[j] = (uint64_t)(int64_t)(f + 0.5L);
      axis[j] = (uint8_t)i;
      f *= ratio;
    }
  }
}

}  // namespace oq
