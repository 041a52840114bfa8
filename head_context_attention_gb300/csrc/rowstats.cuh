// rowstats.cuh -- the backward's row statistics, a block's share.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "ring.cuh"

namespace loong {

constexpr int kRowStatsThreads = 256;
constexpr float kRowStatsLog2e = 1.4426950408889634f;

struct RowStatsArgs {
  const __nv_bfloat16 *o, *o_res, *dout;  // o_res may be null
  const float* lse;
  float *lse2, *dstat;
  int64_t rows, stat_len;
  int S, hq, blk, blk_pad;
  Layout lay;
  unsigned* err;
};

// Backward row statistics (see stat_row_len): for row (b, s, h) of O and dO
// (read where `lay` keeps them), D = sum_d dO*O in fp32 and LSE*log2(e),
// written at the padded position of token s.  With o_res, O is taken as
// O + O_res (exact in fp32: the residual holds the next 8 bits).  16 threads
// per row of 128 bf16 (8 elements each), 8 for d = 64.  Block bx
// of nx covers consecutive tokens of head h of sequence b, so a thread finds
// its token and part by shifts; only the layout map and the block position
// divide (32-bit).  With a bias the statistics hold -LSE*log2(e).
template <int D, bool BIAS>
__device__ __forceinline__ void rowstats_block(const RowStatsArgs& a, int bx, int nx, int h, int b) {
  constexpr int TPR = D / 8;                   // threads per row
  constexpr int RPB = kRowStatsThreads / TPR;  // rows (tokens) per block and pass
  const int part = threadIdx.x % TPR;
  const int lane_row = (threadIdx.x & 31) / TPR;  // this lane's row within its warp
  const int64_t bh = static_cast<int64_t>(b) * a.hq + h;
  // The loop runs per warp (lanes leave together) so the shuffles below see
  // every lane; TPR divides 32, so a row's lanes are all live or all idle.
  const int64_t step = static_cast<int64_t>(nx) * RPB;
  for (int64_t s = static_cast<int64_t>(bx) * RPB + threadIdx.x / TPR; s - lane_row < a.S; s += step) {
    const bool live = s < a.S;
    float acc = 0.f;
    bool row_ok = true;
    if (live) {
      const int64_t off = a.lay.vec(b, s, h, a.hq) * D;
      // checked build: the row's O / dO vectors lie inside the tensors
      row_ok = in_bounds(off >= 0 && off + D <= a.rows * D, a.err);
      if (row_ok) {
        const uint4 ov = __ldg(reinterpret_cast<const uint4*>(a.o + off) + part);
        const uint4 gv = __ldg(reinterpret_cast<const uint4*>(a.dout + off) + part);
        const uint4 rv = a.o_res ? __ldg(reinterpret_cast<const uint4*>(a.o_res + off) + part) : make_uint4(0, 0, 0, 0);
        const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&ov);
        const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&gv);
        const __nv_bfloat162* r2 = reinterpret_cast<const __nv_bfloat162*>(&rv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 fa = __bfloat1622float2(a2[e]);
          const float2 fr = __bfloat1622float2(r2[e]);
          const float2 fb = __bfloat1622float2(b2[e]);
          acc = fmaf(fa.x + fr.x, fb.x, acc);
          acc = fmaf(fa.y + fr.y, fb.y, acc);
        }
      }
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (live && part == 0 && row_ok) {
      const int si = static_cast<int>(s);  // s < S < 2^31
      const int blk_i = si / a.blk;
      const int64_t pos = bh * a.stat_len + static_cast<int64_t>(blk_i) * a.blk_pad + (si - blk_i * a.blk);
      if (in_bounds(pos >= 0 && pos < (bh + 1) * a.stat_len, a.err)) {
        a.dstat[pos] = acc;
        const float l = __ldg(a.lse + bh * a.S + s);
        if constexpr (BIAS)  // a row that a bias of -inf left nothing: its P must come out 0
          a.lse2[pos] = l == -INFINITY ? l : -(l * kRowStatsLog2e);
        else
          a.lse2[pos] = l * kRowStatsLog2e;
      }
    }
  }
}

}  // namespace loong
