// Host check of the capped scores in every form that a kernel may take: in fp32, for
// scales and caps from one end of what the entry points take to the other, each form
// within 2^-19 of the exact score itself (the exponential alone, under caps up to 64, 2^-21
// of the cap), however far below the cap the score lies.  Compiled by tests/test_mask_paged_corrections.py.
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
  int flip = 0;
  // off by the instructions' bounds (exponential 2^-22, reciprocal 2^-23), either way
  auto off = [&](double v, double by) { return static_cast<float>(v * (1.0 + (++flip & 2 ? by : -by))); };
  for (int es = -24; es <= 24; es += 2)
    for (int ec = -20; ec <= 20; ec += 2)
      for (double f : {1.0, 1.3, 1.9}) {
        const float scale = static_cast<float>(std::ldexp(f, es));
        const float cap = static_cast<float>(std::ldexp(2.0 - 0.5 * f, ec));
        const ScoreCap c = make_score_cap(scale, cap);
        const double inv = static_cast<double>(scale) / cap;
        // |x| from 2^-30 to 2^7, both signs
        for (int i = 0; i < 37 * 40; ++i) {
          const float s = static_cast<float>((i & 1 ? -1 : 1) * std::exp2(-30 + i / 40.0) / inv);
          if (!std::isfinite(s) || std::fabs(s) < 1e-30f) continue;
          const double want = std::tanh(inv * s) / inv;
          auto look = [&](float got, double own) {
            const double err = std::fabs(got - want);
            if (own > 0) worst = std::fmax(worst, err / std::fabs(want));
            if (!(err <= own * std::fabs(want) || (own == 0 && cap <= 64)) || !(err * inv <= 0x1p-21)) ++bad;
            ++checked;
          };
          auto e = [&](float a) { return off(std::exp2(static_cast<double>(a)), 0x1p-22); };
          auto r = [&](float a) {
            ++flip;
            return off(1.0 / a, 0x1p-23);
          };
          if (c.near)
            look(cap_far_score<true>(s, c, e, r), 0x1p-19);
          else
            look(cap_far_score<false>(s, c, e, r), 0);
          if (std::fabs(s) <= c.half) look(poly(s, c.h), 0x1p-19);
          if (std::fabs(s) <= c.limit) look(poly(s, c.c), 0x1p-19);
        }
        // scores of the size that attention has are the uncapped ones under a large cap
        const float s = 8.f / scale;
        if (cap >= 0x1p19f && !(std::fabs(s) <= c.half)) ++bad;
      }
  std::printf("%ld values checked, %ld outside, worst %.3g of 2^-19\n", checked, bad, worst * 0x1p19);
  return bad ? 1 : 0;
}
