// rotary.h -- the cosine and sine of a position's angles, in 64 bits.
//
// A far position's angle has no digits left in 32 bits (10^6 radians: 0.06), and a key that goes into 8 or
// 4 bits is decided at borders that its exact value may be next to.  The angle is reduced by whole quarter
// turns, pi / 2 taken in two parts (106 bits) so that a product of up to 2^50 quarters loses nothing, and
// the rest within +-pi / 4 goes through the Taylor series of sine and cosine, whose next terms, x^17 / 17!
// and x^18 / 18!, are below 2^-54 there.
#pragma once

#include "common.h"

namespace kmi {

// What a launch needs of the rotation.
struct RotaryView {
  const double *freqs;
  double factor;             // times cosine and sine
  double sign;               // of the angles
  int32_t pairs;
  bool interleaved;
};

__device__ __forceinline__ void turn_by(double angle, double *c, double *s) {
  const double k = __builtin_rint(angle * 0.63661977236758134308);     // 2 / pi
  double r = __builtin_fma(-k, 1.57079632679489661923, angle);         // pi / 2, and the rest of it
  r = __builtin_fma(-k, 6.12323399573676588613e-17, r);
  const double z = r * r;
  double p = -1.0 / 1307674368000.0;                                   // 15!
  p = __builtin_fma(p, z, 1.0 / 6227020800.0);
  p = __builtin_fma(p, z, -1.0 / 39916800.0);
  p = __builtin_fma(p, z, 1.0 / 362880.0);
  p = __builtin_fma(p, z, -1.0 / 5040.0);
  p = __builtin_fma(p, z, 1.0 / 120.0);
  p = __builtin_fma(p, z, -1.0 / 6.0);
  const double sn = __builtin_fma(p * z, r, r);
  double q = 1.0 / 20922789888000.0;                                   // 16!
  q = __builtin_fma(q, z, -1.0 / 87178291200.0);
  q = __builtin_fma(q, z, 1.0 / 479001600.0);
  q = __builtin_fma(q, z, -1.0 / 3628800.0);
  q = __builtin_fma(q, z, 1.0 / 40320.0);
  q = __builtin_fma(q, z, -1.0 / 720.0);
  q = __builtin_fma(q, z, 1.0 / 24.0);
  q = __builtin_fma(q, z, -0.5);
  const double cs = __builtin_fma(q, z, 1.0);
  const int turns = (int)(k - 4.0 * __builtin_floor(k * 0.25));        // quarters, 0 .. 3
  const bool odd = turns & 1;
  *c = odd ? sn : cs;
  *s = odd ? cs : sn;
  if (turns == 1 || turns == 2) *c = -*c;
  if (turns >= 2) *s = -*s;
}

// factor (cos, sin) of pair i at a position.
__device__ __forceinline__ double2 rotation(const RotaryView &v, int position, int i) {
  double c, s;
  turn_by(v.sign * ((double)position * v.freqs[i]), &c, &s);
  return make_double2(c * v.factor, s * v.factor);
}

}  // namespace kmi
