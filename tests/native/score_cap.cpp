// Host check of the capped scores' polynomials: in fp32, for scales and caps from
// one end of what the entry points take to the other, within their bounds of the
// tangent up to their limits.  Compiled by tests/test_score_cap.py.
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include "score_cap.h"

using namespace loong;

template <int N>
static float poly(float s, const float (&c)[N]) {
  const float y = s * s;
  float p = c[N - 1];
  for (int i = N - 2; i >= 0; --i) p = std::fma(y, p, c[i]);
  return std::fma(s, y * p, s);
}

int main() {
  long checked = 0, bad = 0;
  double worst = 0;
  for (int es = -24; es <= 24; es += 2)
    for (int ec = -20; ec <= 20; ec += 2)
      for (double f : {1.0, 1.3, 1.9}) {
        const float scale = static_cast<float>(std::ldexp(f, es)), cap = static_cast<float>(std::ldexp(2.0 - 0.5 * f, ec));
        const ScoreCap c = make_score_cap(scale, cap);
        const double inv = static_cast<double>(scale) / cap;
        if (!(c.half <= c.limit) || !std::isfinite(c.limit)) ++bad;
        for (int i = -1000; i <= 1000; ++i) {
          for (int far = 0; far < 2; ++far) {
            const float s = static_cast<float>((far ? c.limit : c.half) * (i / 1000.0));
            const double got = inv * (far ? poly(s, c.c) : poly(s, c.h)), want = std::tanh(inv * s);
            // the fit's error, and roundings of at most 1 in fp32
            const double err = std::fabs(got - want);
            worst = std::fmax(worst, err);
            if (!(err <= (far ? 3.3e-7 : 2.0e-7) + 4 * 5.97e-8 * std::fabs(want))) ++bad;
            ++checked;
          }
        }
      }
  std::printf("%ld values checked, %ld outside, worst %.3g\n", checked, bad, worst);
  return bad ? 1 : 0;
}
