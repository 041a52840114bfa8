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

// Values that are not finite, of bf16 pairs: 0xFFFF in their halves.
__device__ __forceinline__ unsigned bf16x2_not_finite(unsigned w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}
// The vector with 0 in their place; `bad` collects whether there were any.
__device__ __forceinline__ uint4 v16_finite(uint4 x, unsigned& bad) {
  const uint4 m = make_uint4(bf16x2_not_finite(x.x), bf16x2_not_finite(x.y), bf16x2_not_finite(x.z),
                             bf16x2_not_finite(x.w));
  bad |= m.x | m.y | m.z | m.w;
  return make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
}

// The whole conversion by one block of THREADS: max |V| into *amax (a float's
// bit pattern) and the copy.
// FINITE: values that are not finite are left out of the maximum and 0 in the
// copy, and amax[1] tells whether there were any.
template <int THREADS, bool FINITE = false>
__device__ __forceinline__ void block_v_to_f16(const uint4* __restrict__ in, uint4* __restrict__ out,
                                               unsigned* __restrict__ amax, int nvec) {
  __shared__ unsigned warp_max[THREADS / 32];
  constexpr int U = 8;  // loads in flight per thread
  unsigned m = 0, bad = 0;
  for (int i0 = threadIdx.x; i0 < nvec; i0 += THREADS * U) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      x[k] = i0 + k * THREADS < nvec ? __ldg(in + i0 + k * THREADS) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < U; ++k) m = max(m, v16_absmax(FINITE ? v16_finite(x[k], bad) : x[k]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  if constexpr (FINITE)
    bad = __syncthreads_or(bad != 0);
  else
    __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = max(m, warp_max[w]);
  if (threadIdx.x == 0) *amax = m << 16;
  if (FINITE && threadIdx.x == 0) amax[1] = bad;
  const float f = v16_factor(m << 16);
  for (int i0 = threadIdx.x; i0 < nvec; i0 += THREADS * U) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      x[k] = i0 + k * THREADS < nvec ? __ldg(in + i0 + k * THREADS) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i0 + k * THREADS < nvec) out[i0 + k * THREADS] = v16_scaled(FINITE ? v16_finite(x[k], bad) : x[k], f);
  }
}

// The conversion by many blocks, in two launches: every block's share of max |V|,
// then the copy, whose blocks take the maximum of the shares each.
// 16K tokens of 32 + 8 heads of 128: 11.6 us for V's 34 MB, 11.8 us for the
// copy (cold); memory's latency, in launches this short.
struct VArgs {
  const uint4* v;
  uint4* v16;
  unsigned* amax;    // the bit pattern of max |V|; FINITE: and, after it, whether V holds values that are not finite
  unsigned* shares;  // [max_blocks]
  int64_t vecs;
  int max_blocks;  // 0: one block converts V
};

// V of at most this many vectors of 8 is converted by one block, in the launch
// that prepares the rest, else by two launches.  The forward of heads of 64 with a
// bias, one block and two launches: 1,600 vectors 17.1 and 20.8 us, 4,096 21.0 and
// 23.0, 6,144 23.1 and 24.7, 8,192 25.1 and 25.2, 12,288 29.2 and 27.1.
constexpr int64_t kBlockV = 8192;

// Maximum over the block of every thread's m, in every thread.
template <int THREADS>
__device__ __forceinline__ unsigned block_max(unsigned m) {
  __shared__ unsigned warp_max[THREADS / 32];
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = max(m, warp_max[w]);
  return m;
}

// Block `id`'s part of the launch before the copy (one block: all of it).
// FINITE: bit 15 of a share says that it met a value that is not finite.
template <int THREADS, bool FINITE = false>
__device__ __forceinline__ void v16_first_launch(const VArgs& v, int id) {
  if (v.max_blocks == 0) {
    block_v_to_f16<THREADS, FINITE>(v.v, v.v16, v.amax, static_cast<int>(v.vecs));
    return;
  }
  constexpr int U = 4;  // loads in flight per thread
  const int64_t i1 = v.vecs * (id + 1) / v.max_blocks;
  unsigned m = 0, bad = 0;
  for (int64_t i = v.vecs * id / v.max_blocks + threadIdx.x; i < i1; i += THREADS * U) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) x[k] = i + k * THREADS < i1 ? __ldg(v.v + i + k * THREADS) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < U; ++k) m = max(m, v16_absmax(FINITE ? v16_finite(x[k], bad) : x[k]));
  }
  m = block_max<THREADS>(m);
  if constexpr (FINITE) m |= __syncthreads_or(bad != 0) ? 0x8000u : 0u;
  if (threadIdx.x == 0) v.shares[id] = m;
}

// V's fp16 form from the shares' maxima, and max |V| for the attention kernel.
template <int THREADS, bool FINITE = false>
__device__ __forceinline__ void v16_copy(const VArgs& v) {
  unsigned m = 0, bad = 0;
  for (int i = threadIdx.x; i < v.max_blocks; i += THREADS) {
    const unsigned s = v.shares[i];
    m = max(m, FINITE ? s & 0x7FFFu : s);
    bad |= s & 0x8000u;
  }
  m = block_max<THREADS>(m) << 16;
  if constexpr (FINITE) bad = __syncthreads_or(bad != 0);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *v.amax = m;
    if (FINITE) v.amax[1] = bad;
  }
  const float f = v16_factor(m);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * THREADS;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < v.vecs; i += stride) {
    const uint4 x = __ldg(v.v + i);
    v.v16[i] = v16_scaled(FINITE ? v16_finite(x, bad) : x, f);
  }
}

}  // namespace loong
