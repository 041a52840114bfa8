// score_cap.h -- the constants of scores capped by a hyperbolic tangent (softcap.cuh).
//
// tanh(inv s) / inv, inv = scale / cap, by odd polynomials s (1 + y a(y)), y = (inv s)^2,
// a(y) fitted for the least greatest absolute error of the tangent (iterated weighted
// least squares): up to |inv s| = 1 degree 11, off by at most 3.3e-7 (below three half
// steps of fp32 next to 1), up to 1/2 degree 7, 2.0e-7.  The powers of inv are in the
// coefficients.
#pragma once

#include <cmath>

namespace loong {

struct ScoreCap {
  float inv = 0.f;  // scale / cap; 0: no cap
  float rinv = 0.f;
  float limit = 0.f, half = 0.f;  // |s| up to which the polynomials hold
  float c[5] = {}, h[3] = {};     // theirs: of s^2, s^4, ..
};

// scale and cap as the entry points let them through (2^-24 .. 2^24 and 2^-20 ..
// 2^20).  The coefficients have to be normal numbers: the highest is about 2^-8
// inv^10, so below inv = 2^-11 it may be lost, where it does not count up to a
// quarter, below 2^-14 the next as well, and the polynomial is not used.
inline ScoreCap make_score_cap(float scale, float cap) {
  ScoreCap r;
  if (!(cap > 0.f)) return r;
  constexpr double a[5] = {-0.33328669672829153, 0.1327561340237302, -0.05142530563209422, 0.01653276431015356,
                           -0.0029830620753639016};
  constexpr double half[3] = {-0.33326460635391786, 0.1318586029707108, -0.04422924520882877};
  const double inv = static_cast<double>(scale) / cap;
  r.inv = static_cast<float>(inv);
  r.rinv = static_cast<float>(1.0 / inv);
  const double most = inv > 2048.0 ? 0.0 : inv > 0x1p-11 ? 1.0 : inv > 0x1p-14 ? 0.25 : 0.0;
  r.limit = static_cast<float>(most / inv);
  r.half = static_cast<float>(std::fmin(0.5, most) / inv);
  double p = 1.0;
  for (int i = 0; i < 5; ++i) {
    p *= inv * inv;
    r.c[i] = most > 0.0 ? static_cast<float>(a[i] * p) : 0.f;
    if (i < 3) r.h[i] = most > 0.0 ? static_cast<float>(half[i] * p) : 0.f;
  }
  return r;
}

}  // namespace loong
