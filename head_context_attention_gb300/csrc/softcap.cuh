// softcap.cuh -- scores capped by a hyperbolic tangent: the attention kernels'
// logit is cap * tanh(scale q.k / cap).
//
// A raw score s (the product of the matrix instructions) becomes s' = tanh(inv s) /
// inv, inv = scale / cap, and the rest of a kernel goes on with s' where it had s.
// It is within 2^-19 of itself, or 2^-21 of a cap of up to 64 (score_cap.h): the cap may be
// far above the scores.
//
// Scores within the polynomials' reach (score_cap.h) are formed in pairs: 7 paired
// operations for two scores up to |inv s| = 1, 5 up to 1/2, where most are.  The fp32 pipe
// takes 14 and 10 cycles for them and 6 for exponentials and sums, the matrix instructions 16
// for both products at head dimension 128, so it is not a pipe's rate that the cap costs
// (cap_tile).  (A third polynomial up to 1/4: 4 % for the forward where
// scores stay there, 3 % against it elsewhere and in the backward.)  A warp whose scores
// pass 1 takes 1 - 2 / (1 + e^2x), two more special functions a score, and under caps above
// 64 the shorter polynomial for those of them below 1/2.  (For every cap: 12 % for the
// forward where scores pass it, 20 % for a chunk over pages, and 2 to 3 % for the backward
// everywhere.)
#pragma once

#include "ptx.cuh"
#include "score_cap.h"

namespace loong {

// max(|a|, |b|, |c|) in one instruction (sm_100 family).
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One score where the polynomials do not reach (score_cap.h).
template <bool NEAR>
__device__ __forceinline__ float cap_score(float s, const ScoreCap& cap) {
  return cap_far_score<NEAR>(s, cap, [](float a) { return fast_exp2(a); }, [](float a) { return fast_rcp(a); });
}

// s (1 + y (c[0] + y (c[1] + ..))), y = s^2, of s[0 .. N), N a multiple of 8.
template <int N, int C>
__device__ __forceinline__ void cap_polynomial(uint32_t (&s)[N], const float (&c)[C]) {
  auto pair = [](float v) { return make_float2(v, v); };
  constexpr int W = 4;  // pairs side by side (8 and 16: as fast)
#pragma unroll
  for (int i = 0; i < N; i += 2 * W) {
    float2 x[W], y[W], p[W];
#pragma unroll
    for (int u = 0; u < W; ++u) {
      x[u] = make_float2(__uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
      y[u] = __fmul2_rn(x[u], x[u]);
    }
#pragma unroll
    for (int u = 0; u < W; ++u) p[u] = __ffma2_rn(y[u], pair(c[C - 1]), pair(c[C - 2]));
#pragma unroll
    for (int k = C - 3; k >= 0; --k)
#pragma unroll
      for (int u = 0; u < W; ++u) p[u] = __ffma2_rn(y[u], p[u], pair(c[k]));
#pragma unroll
    for (int u = 0; u < W; ++u) p[u] = __fmul2_rn(y[u], p[u]);
#pragma unroll
    for (int u = 0; u < W; ++u) {
      x[u] = __ffma2_rn(x[u], p[u], x[u]);
      s[i + 2 * u] = __float_as_uint(x[u].x);
      s[i + 2 * u + 1] = __float_as_uint(x[u].y);
    }
  }
}

// Scores s[0 .. N) (32-bit words that hold floats; N a multiple of 8) capped.  The
// warp's lanes call it together; which form they take goes by the lanes that count
// and all of their scores, so those that are not seen are 0.
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], const ScoreCap& cap, bool counts = true) {
  float m[4] = {};
#pragma unroll
  for (int i = 0; i < N; i += 8)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      m[u] = fmax3_abs(m[u], __uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
  const float most = counts ? fmaxf(fmax3_abs(m[0], m[1], m[2]), m[3]) : 0.f;
  if (__all_sync(0xffffffffu, most <= cap.half)) {
    cap_polynomial(s, cap.h);
  } else if (__all_sync(0xffffffffu, most <= cap.limit)) {
    cap_polynomial(s, cap.c);
  } else if (!cap.near) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __float_as_uint(cap_score<false>(__uint_as_float(s[i]), cap));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __float_as_uint(cap_score<true>(__uint_as_float(s[i]), cap));
  }
}

// The 128 scores of a lane's row in tensor memory, from column address t on, capped
// where they are, before the softmax reads them, N at a time.  A loop, because the
// code of a tile in one piece, the polynomial of 64 pairs and the other form of the
// tangent beside it in front of the exponentials, did not fit the instruction cache:
// forward of 32 + 8 heads of 128, 16K tokens, scores of deviation 3, 3.03-3.81 ms by how
// it was arranged, as a loop 2.56, with the shorter polynomial beside the longer 2.32
// (without a cap, on the same scores, 1.57), on blocks that stay 2.24.  What is left is a chain:
// a warp takes its 32 rows of a tile through cap, exponentials and packing by itself, two
// such warps a scheduler, and a slot's next scores wait for it.  The polynomials lengthen it by
// 1,280 cycles for two slots (0.58 ms) and the way through tensor memory as well (0.24), while
// no pipe is full: the matrix instructions take 2,048 cycles for the two slots, 40 % of the
// time, the fp32 pipe is busy about as long.  Four more warps for the cap alone, 2.63: the
// softmax warps then have 176 registers for 216, and every tile one more barrier on its way.
// masked: seen(c) has a bit for each of columns c .. c + 31.
template <int N, typename Seen>
__device__ __forceinline__ void cap_tile(uint32_t t, const ScoreCap& cap, bool counts, bool masked, Seen&& seen) {
#pragma unroll 1
  for (int cb = 0; cb < 128; cb += N) {
    uint32_t s[N / 32][32], x[N];
#pragma unroll
    for (int u = 0; u < N / 32; ++u) tmem_ld32(t + cb + u * 32, s[u]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = s[i / 32][i % 32];
    if (masked) {
#pragma unroll
      for (int u = 0; u < N / 32; ++u) {
        const uint32_t bits = seen(cb + u * 32);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(bits >> i & 1)) x[u * 32 + i] = 0;
      }
    }
    cap_scores(x, cap, counts);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i / 32][i % 32] = x[i];
#pragma unroll
    for (int u = 0; u < N / 32; ++u) tmem_st32(t + cb + u * 32, s[u]);
  }
  tmem_wait_st();
}

}  // namespace loong
