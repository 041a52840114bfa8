// score_cap.h -- the constants of scores capped by a hyperbolic tangent (softcap.cuh).
//
// tanh(inv s) / inv, inv = scale / cap, by odd polynomials s (1 + y a(y)), y = (inv s)^2,
// a(y) fitted for the least greatest absolute error of the tangent (iterated weighted
// least squares): up to |inv s| = 1 degree 11, off by at most 3.3e-7 (below three half
// steps of fp32 next to 1), up to 1/2 degree 7, 2.0e-7.  The powers of inv are in the
// coefficients.  Relative to the tangent that is 1.3 * 2^-20 and 1.05 * 2^-20 at most, the
// first terms being next to exact: within 2^-19 of itself however far below the cap a
// score lies, and under a cap far above the scores they are the uncapped ones.
// The exponential, 1 - 2 / (1 + e^2x), is off by up to 2^-21 for small x as well, that
// much of the cap: 3.1e-5 of a logit at a cap of 64.  Under larger ones it is for |x| above
// 1/2 alone, with the shorter polynomial beside it.
#pragma once

#include <math.h>

#include <cmath>

namespace loong {

struct ScoreCap {
  float inv = 0.f;  // scale / cap; 0: no cap
  float rinv = 0.f;
  bool near = false;              // beyond the polynomials: scores below the cap's half by the shorter one
  float limit = 0.f, half = 0.f;  // |s| up to which the polynomials hold
  float c[5] = {}, h[3] = {};     // theirs: of s^2, s^4, ..
};

// The shorter polynomial's coefficients, of x = inv s.
constexpr float kTanhHalf[3] = {-0.33326460635391786f, 0.1318586029707108f, -0.04422924520882877f};

// What the entry points let through: no cap (0), or caps of 2^-20 .. 2^20 and scales, where
// given, of 2^-24 .. 2^24.  A capped logit is at most the cap; up to 2^20 the softmax's
// reference, rounded to 24 bits, is off by at most 2^-3 in log2 units, which fp16 P has
// room for.
inline bool score_cap_fits(float scale, float cap) {
  const bool scale_fits = !(scale > 0.f) || (scale >= 0x1p-24f && scale <= 0x1p24f);
  return !(cap > 0.f) || (cap >= 0x1p-20f && cap <= 0x1p20f && scale_fits);
}

// The coefficients that count have to be normal numbers: the longer polynomial's
// highest is about 2^-8 inv^10, so it is for inv above 2^-11, the shorter one's 2^-5
// inv^6, above 2^-20.  Below, s (1 - y / 3) is left, to which the next term adds less than
// 2^-26 up to |x| = 2^-6.  Above inv = 2^11 inv^10 may pass the largest number.
inline ScoreCap make_score_cap(float scale, float cap) {
  ScoreCap r;
  if (!(cap > 0.f)) return r;
  constexpr double a[5] = {-0.33328669672829153, 0.1327561340237302, -0.05142530563209422, 0.01653276431015356,
                           -0.0029830620753639016};
  const double inv = static_cast<double>(scale) / cap;
  r.inv = static_cast<float>(inv);
  r.rinv = static_cast<float>(1.0 / inv);
  r.near = cap > 64.f;
  if (inv > 2048.0) return r;
  const bool longer = inv > 0x1p-11;
  const double half = inv > 0x1p-20 ? 0.5 : 0x1p-6;
  r.half = static_cast<float>(half / inv);
  r.limit = static_cast<float>((longer ? 1.0 : half) / inv);
  double p = 1.0;
  for (int i = 0; i < 5; ++i) {
    p *= inv * inv;
    if (i < 3) r.h[i] = static_cast<float>(kTanhHalf[i] * p);
    r.c[i] = longer ? static_cast<float>(a[i] * p) : i < 3 ? r.h[i] : 0.f;
  }
  return r;
}

// One score beyond the polynomials' reach, or beside one that is: by the exponential;
// NEAR: below |x| = 1/2 by the shorter polynomial, formed in x, as inv may be anything.
// Exp2 and Rcp: the caller's 2^a and 1 / a.
template <bool NEAR, typename Exp2, typename Rcp>
#ifdef __CUDACC__
__host__ __device__
#endif
inline float cap_far_score(float s, const ScoreCap& cap, Exp2&& exp2_of, Rcp&& reciprocal) {
  constexpr float log2e2 = 2.8853900817779268f;  // 2 log2 e
  const float x = s * cap.inv;
  if (!NEAR) return fmaf(-2.f * cap.rinv, reciprocal(1.f + exp2_of(x * log2e2)), cap.rinv);
  const float y = x * x, near = fmaf(s, y * fmaf(y, fmaf(y, kTanhHalf[2], kTanhHalf[1]), kTanhHalf[0]), s);
  const float far = fmaf(-2.f * cap.rinv, reciprocal(1.f + exp2_of(fabsf(x) * log2e2)), cap.rinv);
  return fabsf(x) <= 0.5f ? near : copysignf(far, s);
}

}  // namespace loong
