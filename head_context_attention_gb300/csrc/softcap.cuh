// softcap.cuh -- scores capped by a hyperbolic tangent: the attention kernels'
// logit is cap * tanh(scale q.k / cap).
//
// A raw score s (the product of the matrix instructions) becomes t = tanh(x), x =
// s * scale / cap, and the rest of a kernel goes on with t where it had s, its
// factor cap * log2 e where it had scale * log2 e.  What counts is the absolute
// error of t: times the cap it is the logit's.
//
// |x| <= 1 takes an odd polynomial of degree 11, x (1 + y a(y)), y = x^2, a(y) fitted
// on [0, 1] for the least greatest error of the whole (iterated weighted least
// squares): 3.3e-7, below three half steps of fp32 next to 1.  Scores are formed in
// pairs, so it costs four instructions a score, on the pipes that the exponentials
// leave free.  A warp whose scores pass 1 takes 1 - 2 / (1 + e^2x), two more special
// functions a score, off by at most 4e-7.
#pragma once

#include "ptx.cuh"

namespace loong {

constexpr float kTanhA1 = -0.33328669672829153f, kTanhA2 = 0.1327561340237302f, kTanhA3 = -0.05142530563209422f,
                kTanhA4 = 0.01653276431015356f, kTanhA5 = -0.0029830620753639016f;

// max(|a|, |b|, |c|) in one instruction (sm_100 family).
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// x[0 .. N) becomes tanh(x * inv), inv = scale / cap (32-bit words that hold
// floats; N a multiple of 4).  The warp's lanes call it together.
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], float inv) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    m0 = fmax3_abs(m0, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    m1 = fmax3_abs(m1, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
  }
  if (__all_sync(0xffffffffu, fmaxf(m0, m1) * inv <= 1.f)) {
    const float2 iv = make_float2(inv, inv);
    auto pair = [](float c) { return make_float2(c, c); };
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 x = __fmul2_rn(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), iv);
      const float2 y = __fmul2_rn(x, x);
      float2 p = __ffma2_rn(y, pair(kTanhA5), pair(kTanhA4));
      p = __ffma2_rn(y, p, pair(kTanhA3));
      p = __ffma2_rn(y, p, pair(kTanhA2));
      p = __ffma2_rn(y, p, pair(kTanhA1));
      p = __ffma2_rn(y, p, pair(1.f));
      p = __fmul2_rn(x, p);
      s[i] = __float_as_uint(p.x);
      s[i + 1] = __float_as_uint(p.y);
    }
  } else {
    const float k = inv * 2.8853900817779268f;  // 2 log2 e
#pragma unroll
    for (int i = 0; i < N; ++i)
      s[i] = __float_as_uint(1.f - __fdividef(2.f, 1.f + fast_exp2(__uint_as_float(s[i]) * k)));
  }
}

}  // namespace loong
