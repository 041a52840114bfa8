// fastdiv.cuh -- unsigned division by a divisor fixed for the launch, n < 2^31:
// the multiply-and-shift method of Granlund and Montgomery ("Division by
// Invariant Integers using Multiplication", 1994), with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, so that n / d = (umulhi(m, n) + n) >> l.
#pragma once

#include <stdint.h>

namespace loong {

struct FastDiv {
  uint32_t d, m, l;
};

inline FastDiv make_fastdiv(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.l = 0;
  while ((1ull << f.l) < d) ++f.l;
  f.m = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.l) - d)) / d + 1);
  return f;
}

__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) {
  return (__umulhi(f.m, n) + n) >> f.l;
}

}  // namespace loong
