// mask_attn.cu -- ring attention in which every query sees a range of keys of its
// own and scores may be capped: the entry points and the launches in front of the
// attention kernels (the scores themselves in attn_fwd.cu, attn_bwd.cu).
//
//   z_ij = cap tanh(scale q_i.k_j / cap), over begin_i <= j < end_i (and j <= i, causal)
//   P = softmax(z), O = P V;  dS = P (dP - D) (1 - (z / cap)^2)
//
// A range covers what training on long sequences masks with: packed documents,
// prefixes, windows, padding.  The attention kernels visit only the tiles that some
// row sees, so before them every 128-row query tile's ranges are summed up (16 bytes
// for 128 * 8), in the launch that prepares V or the row statistics anyway.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "rowstats.cuh"
#include "v16.cuh"

namespace loong {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1216;                  // of a launch that strides over its data: 8 per SM
constexpr int kSms = 152;                         // workspace sizes do not ask the device
constexpr int64_t kMaxSeqlen = int64_t{1} << 30;  // a tile past the last token still has a 32-bit number

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Blocks of a launch that strides over n threads' work.
unsigned blocks_for(int64_t n) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((n + kThreads - 1) / kThreads, kMaxBlocks)));
}

struct TileArgs {
  MaskView m;
  RingGeom g;
  int S;
  int64_t count;  // B * nblocks * ntile
};

// The ranges of query tile x (of B * nblocks * ntile), by a warp.
__device__ __forceinline__ void sum_tile(const TileArgs& a, int64_t x) {
  const int lane = threadIdx.x & 31;
  const int per_seq = a.g.nblocks * a.g.ntile;
  const int b = static_cast<int>(x / per_seq);
  const int i = static_cast<int>(x - static_cast<int64_t>(b) * per_seq);
  const int bq = i / a.g.ntile;
  const int t0 = bq * a.g.blk + (i - bq * a.g.ntile) * kTile;
  const int t1 = min(t0 + kTile, (bq + 1) * a.g.blk);
  int first = 0x7fffffff, last = 0, all_from = 0, all_to = 0x7fffffff;
#pragma unroll
  for (int u = 0; u < kTile / 32; ++u) {
    const int t = t0 + u * 32 + lane;
    if (t < t1) {
      const int2 r = mask_range(a.m, b, t, a.S, a.g.causal);
      const bool some = r.x < r.y;
      first = min(first, some ? r.x : 0x7fffffff);
      last = max(last, r.y);
      all_from = max(all_from, some ? r.x : 0x7fffffff);
      all_to = min(all_to, r.y);
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  all_from = __reduce_max_sync(0xffffffffu, all_from);
  all_to = __reduce_min_sync(0xffffffffu, all_to);
  if (lane == 0) const_cast<int4*>(a.m.tiles)[x] = make_int4(first, last, all_from, all_to);
}

// Before the forward, in one launch: V's part of it (v16.cuh; its blocks come
// first), then 8 tiles a block.
__global__ void __launch_bounds__(kThreads) mask_fwd_prep_kernel(const __grid_constant__ TileArgs a,
                                                                 const __grid_constant__ VArgs v) {
  next_launch_go();
  const int id = static_cast<int>(blockIdx.x) - max(v.max_blocks, 1);
  if (id < 0) {
    v16_first_launch<kThreads, true>(v, blockIdx.x);
    return;
  }
  if (id == 0 && threadIdx.x == 0) *a.m.counter = 0;
  const int64_t x = static_cast<int64_t>(id) * (kThreads / 32) + threadIdx.x / 32;
  if (x < a.count) sum_tile(a, x);
}

__global__ void __launch_bounds__(kThreads) mask_v16_kernel(const __grid_constant__ VArgs v) {
  next_launch_go();
  previous_launch_wait();
  v16_copy<kThreads, true>(v);
}

// Before the backward, in one launch, a block for a query tile of a head: dQ's
// accumulator cleared, the row statistics (rowstats.cuh), and whether the tile has
// rows for the backward's producer to clear: those whose dO or LSE is not finite (so
// is their LSE among the statistics, which hold -LSE and -D: NaN, but infinite for a
// row that sees no key), and
// with a cap, which leaves infinite scores finite, those whose Q is not; and,
// where the tile ends inside the block of 128, any not finite among the rows behind
// it, which the copies bring in as well.  Head 0's blocks sum the tile's ranges up.
// Bound by memory: O, its residual and dO (with a cap Q) in, the accumulator out; 16K
// tokens of 32 heads of 128 98 us, 640 MB, 82 % of DRAM's peak (ncu).
struct BwdPrepArgs {
  TileArgs tiles;
  RowStatsArgs r;
  const __nv_bfloat16* q;
  float* dq_acc;
  uint8_t* bad;
};
template <int D>
__global__ void __launch_bounds__(kThreads) mask_bwd_prep_kernel(const __grid_constant__ BwdPrepArgs a) {
  next_launch_go();
  constexpr int TPR = D / 8, RPP = kThreads / TPR;  // threads of a row, rows of a pass
  const RowStatsArgs& r = a.r;
  const RingGeom& g = a.tiles.g;
  const int h = blockIdx.y, b = blockIdx.z;
  const int bq = blockIdx.x / g.ntile, qi = blockIdx.x - bq * g.ntile;
  const int t0 = bq * g.blk + qi * kTile, len = min(kTile, (bq + 1) * g.blk - t0);
  const int part = threadIdx.x % TPR;
  int hc;
  const int64_t row0 = r.lay.view_row(b, t0, h, r.hq, hc);
  const int heads = r.lay.view_heads(r.hq);
  const int64_t rows = r.lay.view_rows(gridDim.z), bh = static_cast<int64_t>(b) * r.hq + h;
  const int64_t stat0 = bh * r.stat_len + static_cast<int64_t>(bq) * r.blk_pad + qi * kTile;
  bool mark = false;
#pragma unroll
  for (int p = 0; p < kTile / RPP; ++p) {
    const int row = p * RPP + threadIdx.x / TPR;
    const int64_t at = ((row0 + row) * heads + hc) * D + part * 8;
    const bool there = row0 + row < rows;
    float acc = 0.f;
    unsigned bad = 0;
    if (row < len) {
      if (in_bounds(there, r.err)) {
        const uint4 ov = __ldg(reinterpret_cast<const uint4*>(r.o + at));
        const uint4 gv = __ldg(reinterpret_cast<const uint4*>(r.dout + at));
        const uint4 rv = r.o_res ? __ldg(reinterpret_cast<const uint4*>(r.o_res + at)) : make_uint4(0, 0, 0, 0);
        float4* dq = reinterpret_cast<float4*>(a.dq_acc + at);
        dq[0] = dq[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        v16_finite(gv, bad);
        if (a.tiles.m.cap.inv > 0.f) v16_finite(__ldg(reinterpret_cast<const uint4*>(a.q + at)), bad);
        const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(&ov);
        const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&gv);
        const __nv_bfloat162* r2 = reinterpret_cast<const __nv_bfloat162*>(&rv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 fo = __bfloat1622float2(o2[e]);
          const float2 fr = __bfloat1622float2(r2[e]);
          const float2 fg = __bfloat1622float2(g2[e]);
          acc = fmaf(fo.x + fr.x, fg.x, acc);
          acc = fmaf(fo.y + fr.y, fg.y, acc);
        }
      }
    } else if (there) {
      v16_finite(__ldg(reinterpret_cast<const uint4*>(a.q + at)), bad);
      v16_finite(__ldg(reinterpret_cast<const uint4*>(r.dout + at)), bad);
    }
    mark |= bad != 0;
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) {
      acc += __shfl_xor_sync(0xffffffffu, acc, off);
      bad |= __shfl_xor_sync(0xffffffffu, bad, off);
    }
    if (part == 0 && row < len) {
      const int64_t pos = stat0 + row;
      if (in_bounds(pos >= 0 && pos < (bh + 1) * r.stat_len, r.err)) {
        float l = __ldg(r.lse + bh * r.S + t0 + row);
        if (bad || !(l < INFINITY)) l = __int_as_float(0x7fffffff);
        r.dstat[pos] = -acc;
        r.lse2[pos] = -l * kRowStatsLog2e;
        mark |= !(fabsf(l) < INFINITY);
      }
    }
  }
  const int any = __syncthreads_or(mark);
  if (threadIdx.x == 0) a.bad[bh * g.nblocks * g.ntile + blockIdx.x] = any != 0;
  if (h == 0 && threadIdx.x < 32) sum_tile(a.tiles, static_cast<int64_t>(b) * g.nblocks * g.ntile + blockIdx.x);
}

// After the backward, where the query heads of a group went to several blocks: dQ
// rounded, and the blocks' parts of dK and dV added up, in the order of the heads, and
// rounded.
struct FinishArgs {
  const float4 *dq_acc, *dk_parts, *dv_parts;
  uint4 *dq, *dk, *dv;
  int64_t q_vecs, kv_vecs;  // of 8 elements
  int splits;
};
__global__ void __launch_bounds__(kThreads) mask_finish_kernel(const __grid_constant__ FinishArgs a) {
  auto pack = [](float4 x, float4 y) {
    return make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  };
  auto add = [](float4 x, float4 y) { return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < a.q_vecs + 2 * a.kv_vecs;
       i += stride) {
    if (i < a.q_vecs) {
      a.dq[i] = pack(a.dq_acc[2 * i], a.dq_acc[2 * i + 1]);
      continue;
    }
    const bool v = i >= a.q_vecs + a.kv_vecs;
    const int64_t j = i - a.q_vecs - (v ? a.kv_vecs : 0);
    const float4* parts = v ? a.dv_parts : a.dk_parts;
    float4 x = parts[2 * j], y = parts[2 * j + 1];
    for (int s = 1; s < a.splits; ++s) {
      x = add(x, parts[2 * (s * a.kv_vecs + j)]);
      y = add(y, parts[2 * (s * a.kv_vecs + j) + 1]);
    }
    (v ? a.dv : a.dk)[j] = pack(x, y);
  }
}

int check_mask(const loong_attn_desc* d, const loong_attn_mask* m) {
  int st = loong_attn_check(d);
  if (st != LOONG_OK) return st;
  if (!m || !std::isfinite(m->score_cap) || m->score_cap < 0.f) return LOONG_ERR_INVALID_ARG;
  if (d->seqlen > kMaxSeqlen || d->hq > 65535 || d->batch > 65535) return LOONG_ERR_UNSUPPORTED;
  return score_cap_fits(d->softmax_scale, m->score_cap) ? LOONG_OK : LOONG_ERR_UNSUPPORTED;
}

// In FUSED mode the walks do not follow the ring, so where the layout does not either
// the sequence is one block: its tiles are of 128 tokens but for the last one, whatever
// the ring's blocks (2 x 1990 tokens in 10 blocks of 199, 6 + 3 heads of 64: 16 tiles a
// sequence for 20; 320 tokens in 16 blocks: 3 for 16).
loong_attn_desc one_block(loong_attn_desc d) {
  if (d.mode == LOONG_MODE_FUSED && d.layout == LOONG_LAYOUT_NATURAL) {
    d.hp = d.cp = d.ring_inner = d.ring_outer = 1;
    d.placement = LOONG_PLACEMENT_CONTIGUOUS;
  }
  return d;
}

// The workspace: the plain pass's first, then the tiles' sums and, forward, the
// shares of max |V|, backward, the marks of the query tiles.
struct MaskWs {
  size_t tiles, shares, counter, bad, dk_parts, dv_parts, total;
  int64_t count;
  int splits, per_split;
};
MaskWs mask_ws(const loong_attn_desc& d, int pass) {
  const RingGeom g = ring_geom(d);
  MaskWs w{};
  w.count = d.batch * static_cast<int64_t>(g.nblocks) * g.ntile;
  size_t at = up256(loong_attn_workspace_size(&d, pass));
  w.tiles = at;
  at += up256(static_cast<size_t>(w.count) * sizeof(int4));
  if (pass == 0) {
    w.shares = at;
    at += up256(kMaxBlocks * 4);
    w.counter = at;
    at += up256(4);
  } else {
    w.bad = at;
    at += up256(static_cast<size_t>(w.count) * d.hq);
    // Query heads of a group per block: as many blocks as SMs, where key tiles are fewer.
    // Training passes on the device, one block a key tile and several: 1K tokens of 4 + 2
    // heads of 64 59 and 49 us, 858 of 30 + 5 of 128 123 and 82, 162 in six ring blocks of
    // 56 + 7 of 64 173 and 101, twice 1990 of 6 + 3 of 64 139 and 116.
    const int group = d.hq / d.hkv;
    const int64_t blocks = w.count * d.hkv;
    const int most = d.mode == LOONG_MODE_FUSED ? static_cast<int>(std::max<int64_t>(1, kSms / blocks)) : 1;
    w.per_split = (group + std::min(most, group) - 1) / std::min(most, group);
    w.splits = (group + w.per_split - 1) / w.per_split;
    if (w.splits > 1) {
      const size_t part = up256(static_cast<size_t>(w.splits) * d.batch * d.seqlen * d.hkv * d.head_dim * 4);
      w.dk_parts = at;
      w.dv_parts = at + part;
      at += 2 * part;
    }
  }
  w.total = at;
  return w;
}

TileArgs tile_args(const loong_attn_desc& d, const loong_attn_mask& m, const MaskWs& w, uint8_t* base) {
  TileArgs a;
  a.m.range = reinterpret_cast<const int2*>(m.key_range);
  a.m.tiles = reinterpret_cast<const int4*>(base + w.tiles);
  const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / std::sqrt(static_cast<float>(d.head_dim));
  a.m.cap = make_score_cap(scale, m.score_cap);
  a.g = ring_geom(d);
  a.S = static_cast<int>(d.seqlen);
  a.count = w.count;
  return a;
}

}  // namespace

}  // namespace loong

using namespace loong;

extern "C" {

int loong_attn_mask_check(const loong_attn_desc* d, const loong_attn_mask* mask) { return check_mask(d, mask); }

size_t loong_attn_mask_workspace_size(const loong_attn_desc* d, const loong_attn_mask* mask, int pass) {
  if (check_mask(d, mask) != LOONG_OK || (pass != 0 && pass != 1)) return 0;
  return mask_ws(one_block(*d), pass).total;
}

int loong_attn_mask_fwd(const loong_attn_desc* desc, const loong_attn_mask* mask, const void* q, const void* k,
                        const void* v, void* o, float* lse, void* o_res, void* ws, size_t ws_bytes,
                        loong_stream_t stream_) {
  NvtxRange range("loong_attn_mask_fwd");
  int st = check_mask(desc, mask);
  if (st != LOONG_OK) return st;
  const loong_attn_desc one = one_block(*desc), *d = &one;
  const void* ptrs[] = {q, k, v, o, lse};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 16)) return LOONG_ERR_INVALID_ARG;
  if (!aligned(o_res, 16) || !aligned(mask->key_range, 8)) return LOONG_ERR_INVALID_ARG;
  const MaskWs w = mask_ws(*d, 0);
  if (!ws || ws_bytes < w.total || !aligned(ws, 16)) return LOONG_ERR_WORKSPACE;
  if ((st = device_ready()) != LOONG_OK) return st;
  for (const void* p : ptrs)
    if (!on_device(p)) return LOONG_ERR_INVALID_ARG;
  if (!on_device(ws) || (o_res && !on_device(o_res)) || (mask->key_range && !on_device(mask->key_range)))
    return LOONG_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* base = static_cast<uint8_t*>(ws);
  TileArgs a = tile_args(*d, *mask, w, base);
  a.m.v = static_cast<const __nv_bfloat16*>(v);
  a.m.counter = reinterpret_cast<int*>(base + w.counter);
  const FwdWsLayout L = fwd_ws_layout(*d);
  VArgs va;
  va.v = static_cast<const uint4*>(v);
  va.v16 = reinterpret_cast<uint4*>(base + L.v16);
  va.amax = reinterpret_cast<unsigned*>(base + L.amax);
  va.shares = reinterpret_cast<unsigned*>(base + w.shares);
  va.vecs = d->batch * d->seqlen * d->hkv * d->head_dim / 8;
  va.max_blocks = va.vecs <= kBlockV ? 0 : static_cast<int>(blocks_for(va.vecs / 2));
  const int64_t tile_blocks = (w.count + kThreads / 32 - 1) / (kThreads / 32);
  mask_fwd_prep_kernel<<<static_cast<unsigned>(std::max(va.max_blocks, 1) + tile_blocks), kThreads, 0, stream>>>(a, va);
  if ((st = check_launch()) != LOONG_OK) return st;
  if (va.max_blocks > 0) {
    st = launch_dependent(mask_v16_kernel, dim3(blocks_for(va.vecs)), kThreads, 0, stream, va);
    if (st != LOONG_OK) return st;
  }
  return run_attn_fwd(*d, q, k, v, o, lse, o_res, ws, stream, nullptr, &a.m);
}

int loong_attn_mask_bwd(const loong_attn_desc* desc, const loong_attn_mask* mask, const void* q, const void* k,
                        const void* v, const void* o, const void* o_res, const float* lse, const void* dout, void* dq,
                        void* dk, void* dv, void* ws, size_t ws_bytes, loong_stream_t stream_) {
  NvtxRange range("loong_attn_mask_bwd");
  int st = check_mask(desc, mask);
  if (st != LOONG_OK) return st;
  const loong_attn_desc one = one_block(*desc), *d = &one;
  const void* ptrs[] = {q, k, v, o, lse, dout, dq, dk, dv};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 16)) return LOONG_ERR_INVALID_ARG;
  if (!aligned(o_res, 16) || !aligned(mask->key_range, 8)) return LOONG_ERR_INVALID_ARG;
  const MaskWs w = mask_ws(*d, 1);
  if (!ws || ws_bytes < w.total || !aligned(ws, 16)) return LOONG_ERR_WORKSPACE;
  if ((st = device_ready()) != LOONG_OK) return st;
  for (const void* p : ptrs)
    if (!on_device(p)) return LOONG_ERR_INVALID_ARG;
  if (!on_device(ws) || (o_res && !on_device(o_res)) || (mask->key_range && !on_device(mask->key_range)))
    return LOONG_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const BwdWsLayout L = bwd_ws_layout(*d);
  BwdPrepArgs a;
  a.tiles = tile_args(*d, *mask, w, base);
  int passes;
  if ((st = rowstats_args(*d, o, o_res, dout, lse, reinterpret_cast<float*>(base + L.stats), &a.r, &passes)) !=
      LOONG_OK)
    return st;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.dq_acc = reinterpret_cast<float*>(base + L.dq_acc);
  a.bad = base + w.bad;
  const RingGeom& g = a.tiles.g;
  const dim3 grid(static_cast<unsigned>(g.nblocks * g.ntile), static_cast<unsigned>(d->hq),
                  static_cast<unsigned>(d->batch));
  if (d->head_dim == 128)
    mask_bwd_prep_kernel<128><<<grid, kThreads, 0, stream>>>(a);
  else
    mask_bwd_prep_kernel<64><<<grid, kThreads, 0, stream>>>(a);
  if ((st = check_launch()) != LOONG_OK) return st;
  MaskView& m = a.tiles.m;
  m.bad = a.bad;
  m.splits = w.splits;
  m.per_split = w.per_split;
  m.dk_parts = reinterpret_cast<float*>(base + w.dk_parts);
  m.dv_parts = reinterpret_cast<float*>(base + w.dv_parts);
  st = run_attn_bwd(*d, q, k, v, o, o_res, lse, dout, dq, dk, dv, ws, stream, nullptr, nullptr, &m);
  if (st != LOONG_OK || w.splits == 1) return st;
  FinishArgs f;
  f.dq_acc = reinterpret_cast<const float4*>(a.dq_acc);
  f.dk_parts = reinterpret_cast<const float4*>(m.dk_parts);
  f.dv_parts = reinterpret_cast<const float4*>(m.dv_parts);
  f.dq = static_cast<uint4*>(dq);
  f.dk = static_cast<uint4*>(dk);
  f.dv = static_cast<uint4*>(dv);
  f.q_vecs = d->batch * d->seqlen * d->hq * d->head_dim / 8;
  f.kv_vecs = d->batch * d->seqlen * d->hkv * d->head_dim / 8;
  f.splits = w.splits;
  mask_finish_kernel<<<blocks_for(f.q_vecs + 2 * f.kv_vecs), kThreads, 0, stream>>>(f);
  return check_launch();
}

}  // extern "C"
