// v16.cuh -- V as the forward's P V product reads it, V * 2^-e in fp16 with e
// from max |V| (v16_shift, ptx.cuh): the pieces of its conversion.
#pragma once

#include "ptx.cuh"

namespace loong {

// max |x| of 8 bf16 values, as the upper half of a float's bit pattern.  With
// the sign cleared, bf16 bit patterns order like the values they encode.
__device__ __forceinline__ unsigned v16_absmax(const uint4& x) {
  const unsigned w[4] = {x.x, x.y, x.z, x.w};
  unsigned m = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) m = max(m, max(w[u] & 0x7FFFu, (w[u] >> 16) & 0x7FFFu));
  return m;
}

__device__ __forceinline__ float v16_factor(unsigned amax) {
  return __int_as_float((127 - v16_shift(amax)) << 23);  // 2^-e, -100 <= e <= 114
}

__device__ __forceinline__ uint4 v16_scaled(const uint4& x, float f) {
  const unsigned w[4] = {x.x, x.y, x.z, x.w};
  unsigned y[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    y[u] = pack_f16(__uint_as_float(w[u] << 16) * f, __uint_as_float(w[u] & 0xFFFF0000u) * f);
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// The whole conversion by one block of THREADS: max |V| into *amax (a float's
// bit pattern) and the copy.
template <int THREADS>
__device__ __forceinline__ void block_v_to_f16(const uint4* __restrict__ in, uint4* __restrict__ out,
                                               unsigned* __restrict__ amax, int nvec) {
  __shared__ unsigned warp_max[THREADS / 32];
  constexpr int U = 8;  // loads in flight per thread
  unsigned m = 0;
  for (int i0 = threadIdx.x; i0 < nvec; i0 += THREADS * U) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      x[k] = i0 + k * THREADS < nvec ? __ldg(in + i0 + k * THREADS) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < U; ++k) m = max(m, v16_absmax(x[k]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = max(m, warp_max[w]);
  if (threadIdx.x == 0) *amax = m << 16;
  const float f = v16_factor(m << 16);
  for (int i0 = threadIdx.x; i0 < nvec; i0 += THREADS * U) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      x[k] = i0 + k * THREADS < nvec ? __ldg(in + i0 + k * THREADS) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i0 + k * THREADS < nvec) out[i0 + k * THREADS] = v16_scaled(x[k], f);
  }
}

}  // namespace loong
