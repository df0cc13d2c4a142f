// fa_angle.h - angles of the position rotation: the fraction of a turn per
// position in 64-bit fixed point, and cosine and sine of its product with a
// position.  Plain arithmetic on integers and floats, so that the host's compiler
// takes it too.
#pragma once

#include <cmath>

#ifdef __CUDACC__
#define FA_ANGLE_FN __host__ __device__ __forceinline__
#else
#define FA_ANGLE_FN inline
#endif

namespace fa {

namespace rope {

// x mod 1 in units of 2^-64, x >= 0.
FA_ANGLE_FN unsigned long long fraction(double x) {
  x -= floor(x);
  const double hi = floor(x * 4294967296.0);  // two steps: a double holds 53 bits
  const double lo = (x * 4294967296.0 - hi) * 4294967296.0;
  return (static_cast<unsigned long long>(hi) << 32) + static_cast<unsigned long long>(lo);
}
// Turns per position: f / (2 pi).  1 / (2 pi) is taken as 29 bits, whose product
// with the 24 bits of f is exact, and a remainder.  A frequency that is no finite
// number has no turn: it is NO_TURN, and the one finite fraction of that value (2^-64
// of a turn, 2^-33 after 2^31 positions) is taken as none.
constexpr unsigned long long NO_TURN = 1;
FA_ANGLE_FN unsigned long long turns(float f) {
  const double x = fabs(static_cast<double>(f));
  if (!(x <= 3.5e38)) return NO_TURN;  // past the largest float: infinite, or NaN
  unsigned long long t = fraction(x * 0.15915494272485375) + fraction(x * 3.6704158172530464e-10);
  if (f < 0.f) t = 0ull - t;
  return t == NO_TURN ? 0 : t;
}

// cos and sin of position * frequency: the product's fraction of a turn, its
// nearest quarter turn, and the Taylor series about it to the ninth and eighth
// power (|theta| <= pi / 4: remainders 1.8e-9 and 2.5e-8).
FA_ANGLE_FN void turn(int pos, unsigned long long f, float& c, float& s) {
  // sums wrap around the turn, so they are formed without a sign
  const unsigned frac =
      static_cast<unsigned>((static_cast<unsigned long long>(static_cast<long long>(pos)) * f) >> 32);
  const int quarter = static_cast<int>(frac + (1u << 29)) >> 30;  // -2 .. 1, two of them the half turn
  const float th = static_cast<float>(static_cast<int>(frac - (static_cast<unsigned>(quarter) << 30))) *
                   1.4629180792671596e-9f;                        // 2 pi / 2^32
  const float x = th * th;
  const float si = fmaf(th * x, fmaf(x, fmaf(x, fmaf(x, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f),
                                     -1.6666667e-1f), th);
  const float co = fmaf(x, fmaf(x, fmaf(x, fmaf(x, 2.4801587e-5f, -1.3888889e-3f), 4.1666667e-2f), -0.5f),
                        1.f);
  const bool swap = (quarter & 1) != 0;
  c = swap ? si : co;
  s = swap ? co : si;
  if (((quarter + 1) & 2) != 0) c = -c;          // quarters 1 and 2
  if ((quarter & 2) != 0) s = -s;                // quarters 2 and 3
  if (f == NO_TURN) c = s = NAN;
}

}  // namespace rope

}  // namespace fa
