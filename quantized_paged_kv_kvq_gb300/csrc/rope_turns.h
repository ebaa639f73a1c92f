// Host side of the rotation tables: the turns per position of every pair, as 64-bit
// fractions of a turn (kvq_rope_kind has the formulas).
//
// A position p multiplies the fraction's error by p, up to 2^31, and the table's
// entries are to stay within 3e-7: a float64 theta (2^-53 of it, twice or three times
// over) moves the angle by 3.6e-7 there (base 1.298, 2 of 4 elements).  So the
// fractions are made in pairs of float64 whose sum is the value (105 bits or so) and
// rounded once, to 2^-65 turns: at p = 2^31 some 4e-10 radians.
#pragma once

#include <math.h>
#include <stdint.h>

#include "../../include/kvq.h"
#include "kvq_internal.h"

namespace kvq {

// A number as the unevaluated sum of two float64, |lo| <= ulp(hi) / 2.  Sums and
// products by their exact errors (Dekker, Knuth).
struct Wide {
  double hi, lo;
};
inline Wide wide_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
inline Wide add(Wide a, Wide b) {
  const Wide s = wide_sum(a.hi, b.hi);
  return wide_sum(s.hi, s.lo + (a.lo + b.lo));
}
inline Wide mul(Wide a, Wide b) {
  const double p = a.hi * b.hi;
  return wide_sum(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
inline Wide neg(Wide a) { return {-a.hi, -a.lo}; }
inline Wide div(Wide a, Wide b) {
  const Wide q = {a.hi / b.hi, 0.0};
  const Wide r = add(a, neg(mul(q, b)));
  return add(q, {r.hi / b.hi, 0.0});
}
inline Wide clamp01(Wide a) { return a.hi < 0.0 ? Wide{0.0, 0.0} : a.hi >= 1.0 ? Wide{1.0, 0.0} : a; }

// x^(-1/m): the float64 root, and one Newton step on y^m x = 1.
inline Wide root(double x, int m) {
  const double y = pow(x, -1.0 / m);
  Wide p = {x, 0.0}, square = {y, 0.0};
  for (int e = m; e > 0; e >>= 1) {  // x y^m
    if (e & 1) p = mul(p, square);
    square = mul(square, square);
  }
  const double off = ((p.hi - 1.0) + p.lo) / m;
  return fabs(off) < 1e-9 ? wide_sum(y, -y * off) : Wide{y, 0.0};  // else y^m left float64's range
}

// The turns (of 2^64) of every pair; false where one turns more than 2^24 times a
// position (a factor below 2^-24 or so), which leaves no fraction to keep.
inline bool rope_turns(int rot_dim, double base, const kvq_rope_scaling& sc, RopeTurns* turns) {
  const double two_pi = 6.283185307179586476925;
  const Wide turns_per_radian = div({1.0, 0.0}, {two_pi, 2.449293598294706355e-16});  // 1 / (2 pi)
  // theta_i = ratio^i
  Wide ratio = root(base, rot_dim / 2);
  if (sc.kind == KVQ_ROPE_NTK) ratio = mul(ratio, root(sc.factor, (rot_dim - 2) / 2));
  double from = 0.0, to = 0.0;  // YARN's ramp
  if (sc.kind == KVQ_ROPE_YARN) {
    auto pair_of = [&](double n) {
      return rot_dim * log(sc.original_len / (two_pi * n)) / (2.0 * log(base));
    };
    from = fmax(floor(pair_of(sc.high)), 0.0);
    to = fmin(ceil(pair_of(sc.low)), rot_dim - 1.0);
  }
  const Wide one = {1.0, 0.0}, factor = {sc.factor, 0.0};
  Wide theta = one;
  for (int i = 0; i < kMaxRopePairs; ++i) {
    turns->t[i] = 0;
    if (i >= rot_dim / 2) continue;
    Wide x = mul(theta, turns_per_radian);
    if (sc.kind == KVQ_ROPE_LINEAR) x = div(x, factor);
    if (sc.kind == KVQ_ROPE_YARN || sc.kind == KVQ_ROPE_BANDS) {
      Wide slow;  // the part divided by the factor
      if (sc.kind == KVQ_ROPE_YARN) {
        slow = clamp01(div(wide_sum(i, -from), {fmax(to - from, 0.001), 0.0}));
      } else {
        const Wide whole = mul(x, {sc.original_len, 0.0});  // turns within the original length
        slow = add(one, neg(clamp01(div(add(whole, {-sc.low, 0.0}), wide_sum(sc.high, -sc.low)))));
      }
      x = add(mul(div(x, factor), slow), mul(x, add(one, neg(slow))));
    }
    if (!(fabs(x.hi) <= 0x1p24)) return false;
    // whole turns change nothing: what is left is in [-1/2, 1/2], and 1/2 is -1/2
    double part = x.hi - rint(x.hi);
    if (part >= 0.5) part -= 1.0;
    const double top = floor(ldexp(part, 64));
    const double rest = (ldexp(part, 64) - top) + ldexp(x.lo, 64);
    turns->t[i] = static_cast<unsigned long long>(static_cast<int64_t>(top)) +
                  static_cast<unsigned long long>(llrint(rest));
    theta = mul(theta, ratio);
  }
  return true;
}

}  // namespace kvq
