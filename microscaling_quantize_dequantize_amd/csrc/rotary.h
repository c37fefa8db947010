// Rotary positions on the device: the angle of a pair and its sine and cosine.
#pragma once

#include "launch.h"

namespace mx {

enum RotaryLayout { ROTARY_HALF = 0, ROTARY_INTERLEAVED = 1 };

// The position that turns a pair of a token; zero on an axis that there is not.  AXES: the pairs have axes.
template <bool AXES>
__device__ __forceinline__ double position_of(const Positions &p, int64_t token, int pair) {
  if constexpr (!AXES) return (double)p.at[token];
  const int axis = p.axes[pair];
  return (unsigned)axis < (unsigned)p.count ? (double)p.at[axis * p.stride + token] : 0.0;
}

// Sine and cosine of an angle in radians, in fp64.
//
// The angle of a far position (2^20 and beyond) has to be reduced before it
// is rounded: n = rint(a / (pi/2)), r = a - n pi/2 with pi/2 in two parts
// whose products with n are exact inside the fused multiply-adds, so r is
// within 2^-53 of the reduced angle for every |a| < 2^50.  On [-pi/4, pi/4]
// the Taylor series to r^15 and r^16 leave less than 2^-54.  fp64
// multiply-adds run at the rate of fp32 ones here (64 lanes a clock a CU),
// and a pair's values serve every head of its token.
__device__ __forceinline__ void sine_cosine(double a, double &s, double &c) {
  const double n = __builtin_rint(a * 0x1.45f306dc9c883p-1);
  double r = __builtin_fma(-n, 0x1.921fb54442d18p+0, a);
  r = __builtin_fma(-n, 0x1.1a62633145c07p-54, r);
  const double z = r * r;
  double ps = -1.0 / 1307674368000.0;
  ps = __builtin_fma(ps, z, 1.0 / 6227020800.0);
  ps = __builtin_fma(ps, z, -1.0 / 39916800.0);
  ps = __builtin_fma(ps, z, 1.0 / 362880.0);
  ps = __builtin_fma(ps, z, -1.0 / 5040.0);
  ps = __builtin_fma(ps, z, 1.0 / 120.0);
  ps = __builtin_fma(ps, z, -1.0 / 6.0);
  const double sr = __builtin_fma(ps * z, r, r);
  double pc = 1.0 / 20922789888000.0;
  pc = __builtin_fma(pc, z, -1.0 / 87178291200.0);
  pc = __builtin_fma(pc, z, 1.0 / 479001600.0);
  pc = __builtin_fma(pc, z, -1.0 / 3628800.0);
  pc = __builtin_fma(pc, z, 1.0 / 40320.0);
  pc = __builtin_fma(pc, z, -1.0 / 720.0);
  pc = __builtin_fma(pc, z, 1.0 / 24.0);
  pc = __builtin_fma(pc, z, -0.5);
  const double cr = __builtin_fma(pc, z, 1.0);
  // the quarter turn, n mod 4: odd ones exchange the two, and two of the four negate each
  const int q = (int)(n - 4.0 * __builtin_floor(n * 0.25));
  const double ss = (q & 1) ? cr : sr, cc = (q & 1) ? sr : cr;
  s = (q & 2) ? -ss : ss;
  c = ((q + 1) & 2) ? -cc : cc;
}

}  // namespace mx
