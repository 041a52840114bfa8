// rel_bias.cu -- ring attention with a learned bias of the distance q - k, in
// buckets: the entry points, the bias by distance that the attention kernels
// read, and the sum of the bias gradient's parts.
//
//   logit_ij = scale q_i . k_j + table[bucket(i - j)][head]
//   dtable[t][head] = sum over i, j with bucket(i - j) = t of dS_ij
//
// bucket() is piecewise constant in the distance.  It is expanded once per call
// into the bias of every distance (in units of the unscaled score, so that a
// score takes it with one add) and the distance's interval; the attention
// kernels decide from the interval at a tile's two extreme distances whether
// the whole tile shares one value.  The expansion is hq * S words against
// hq * S^2 / 2 scores.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "rowstats.cuh"
#include "v16.cuh"

namespace loong {

namespace {

constexpr int kMaxIntervals = 256;
constexpr int kMaxBuckets = 256;
constexpr int kThreads = 256;
// The finite values a bias may have.  From -kBound down it masks, as -inf does,
// from kBound up it is as +inf: a softmax reference of that size, rounded to 24
// bits, is off by up to 2^-3 in log2 units, which fp16 P still has room for (its
// bound 2^15 is half of what fp16 holds).  Divided by the smallest scale accepted
// it is finite.
constexpr float kBound = 1048576.f;  // 2^20
constexpr float kMinScale = 5.9604645e-8f;        // 2^-24
constexpr int64_t kMaxSeqlen = int64_t{1} << 29;  // places fit 32 bits
constexpr int kSumSplits = 64;
constexpr int kMaxBlocks = 1216;  // of a launch that strides over its data: 8 per SM

struct BucketMap {
  int intervals;
  int bounds[kMaxIntervals - 1];
  uint8_t bucket[kMaxIntervals];
};

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// What a block needs to expand the bias.
struct ExpandArgs {
  BucketMap m;
  const __nv_bfloat16* table;
  int hq;
  float inv_scale;
  BiasView out;
};

// One thread per distance: its interval and its pieces' by binary search, then
// the bias of heads by, by + ny, ...; consecutive threads write consecutive
// words.
__device__ __forceinline__ void expand_block(const ExpandArgs& a, int bx, int by, int ny) {
  const BucketMap& m = a.m;
  const BiasView& out = a.out;
  __shared__ int bounds[kMaxIntervals];
  __shared__ uint8_t bucket[kMaxIntervals];
  for (int i = threadIdx.x; i < m.intervals; i += kThreads) {
    bounds[i] = i + 1 < m.intervals ? m.bounds[i] : 0x7fffffff;
    bucket[i] = m.bucket[i];
  }
  __syncthreads();
  const int64_t i = static_cast<int64_t>(bx) * kThreads + threadIdx.x;
  if (i >= out.len) return;
  const int n = static_cast<int>(i) - out.off;
  auto interval_of = [&](int d) {  // the number of bounds <= d
    int lo = 0, hi = m.intervals - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (bounds[mid] <= d)
        lo = mid + 1;
      else
        hi = mid;
    }
    return lo;
  };
  const int at = interval_of(n);
  if (by == 0) {
    const_cast<uint8_t*>(out.interval)[i] = static_cast<uint8_t>(at);
    auto code = [&](int reach) {
      const int lo = interval_of(n - reach), hi = interval_of(n + reach);
      const int kind = min(hi - lo, static_cast<int>(kPieceMixed));
      return PieceCode::make(kind, lo, kind == kPieceStep ? n - bounds[lo] : 0);
    };
    const_cast<int*>(out.piece)[i] = code(31);
    const_cast<int*>(out.tile)[i] = code(127);
  }
  const __nv_bfloat16* row = a.table + static_cast<int64_t>(bucket[at]) * a.hq;
  float* lut = const_cast<float*>(out.lut);
  for (int h = by; h < a.hq; h += ny) {
    const float v = __bfloat162float(row[h]);
    lut[h * out.len + i] = v <= -kBound ? -INFINITY : v >= kBound ? INFINITY : v * a.inv_scale;
  }
}

// Before the forward, in one launch: nx x ny blocks expand the bias, the rest
// work on V (v16.cuh): one block brings a short V into its fp16 form (whole); else
// max_blocks blocks take the maximum of |V| of a share each, for v16_kernel.
__global__ void __launch_bounds__(kThreads) fwd_prep_kernel(const __grid_constant__ ExpandArgs a, int nx, int ny,
                                                            const __grid_constant__ VArgs v) {
  // V's blocks, the longer ones, come first
  const int id = static_cast<int>(blockIdx.x) - max(v.max_blocks, 1);
  if (id >= 0) {
    const int by = id / nx;
    expand_block(a, id - by * nx, by, ny);
    return;
  }
  v16_first_launch<kThreads>(v, blockIdx.x);
}

__global__ void __launch_bounds__(kThreads) v16_kernel(const __grid_constant__ VArgs v) { v16_copy<kThreads>(v); }

// 16-byte words cleared by the whole grid.
__device__ __forceinline__ void clear(uint4* p, int64_t n, int64_t id, int64_t threads) {
  for (int64_t i = id; i < n; i += threads) p[i] = make_uint4(0, 0, 0, 0);
}

// Before the backward, in one launch: dQ's accumulator and the gradient's parts
// and tickets cleared, the row statistics (blockIdx.x < passes), and the bias
// expanded (the other blocks of sequence 0, a head each).  Bound by memory: 16K
// tokens of 32 heads of 128 112 us, 672 MB (6.0 TB/s).
struct ClearArgs {
  uint4 *dq_acc, *parts;
  int64_t dq_vecs, part_vecs;
};
template <int D>
__global__ void __launch_bounds__(kThreads) bwd_prep_kernel(const __grid_constant__ ExpandArgs a,
                                                            const __grid_constant__ RowStatsArgs r, int passes,
                                                            const __grid_constant__ ClearArgs c) {
  static_assert(kThreads == kRowStatsThreads, "one block size");
  const int64_t block = (static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t id = block * kThreads + threadIdx.x;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * gridDim.y * gridDim.z * kThreads;
  clear(c.dq_acc, c.dq_vecs, id, threads);
  clear(c.parts, c.part_vecs, id, threads);
  if (static_cast<int>(blockIdx.x) < passes)
    rowstats_block<D, true>(r, blockIdx.x, passes, blockIdx.y, blockIdx.z);
  else if (blockIdx.z == 0)
    expand_block(a, static_cast<int>(blockIdx.x) - passes, blockIdx.y, gridDim.y);
}

// Sum of the backward's parts over warps, key tiles and sequences, in a fixed
// order: block (head, split) adds its share of the (sequence, key tile) pairs,
// `lots` threads per interval, in 32 bits over a pair's warps and in 64 beyond;
// the last block of a head to finish (tickets, cleared by bwd_prep_kernel) adds
// the splits' sums and then the intervals of every bucket.
struct SumArgs {
  BucketMap m;
  const float* part;
  int64_t pairs;
  int nkt, hkv, group, splits, buckets;
  double* sums;
  unsigned* ticket;
  __nv_bfloat16* dtable;
};
__device__ __forceinline__ void dbias_sum_block(const SumArgs& a, int h, int split) {
  __shared__ bool last;
  __shared__ double by_interval[kMaxIntervals], shares[kThreads];
  const int hq = a.hkv * a.group;
  const int kvh = h / a.group, g = h - kvh * a.group;
  const int ni = a.m.intervals;
  const int64_t width = static_cast<int64_t>(a.group) * ni;
  const int lots = kThreads / ni;  // ni <= kThreads
  const int lot = threadIdx.x / ni, ivl = threadIdx.x - lot * ni;
  const bool mine = lot < lots;
  // the lots' shares of an interval, in the order of the lots
  auto add_shares = [&](double s) {
    if (mine) shares[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x < ni) {
      double t = 0.0;
      for (int l = 0; l < lots; ++l) t += shares[l * ni + threadIdx.x];
      by_interval[threadIdx.x] = t;
    }
    __syncthreads();
  };
  const int64_t j0 = a.pairs * split / a.splits, j1 = a.pairs * (split + 1) / a.splits;
  double acc = 0.0;
  if (mine) {
    for (int64_t j = j0; j < j1; ++j) {
      const int64_t b = j / a.nkt;
      const float* p = a.part + ((b * a.hkv + kvh) * a.nkt + (j - b * a.nkt)) * kBwdComputeWarps * width + g * ni + ivl;
      float s = 0.f;
#pragma unroll 4
      for (int w = lot; w < kBwdComputeWarps; w += lots) s += __ldg(p + w * width);
      acc += static_cast<double>(s);
    }
  }
  add_shares(acc);
  if (threadIdx.x < ni) a.sums[(static_cast<int64_t>(split) * hq + h) * ni + threadIdx.x] = by_interval[threadIdx.x];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.ticket + h, 1u) == static_cast<unsigned>(a.splits) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  acc = 0.0;
  if (mine) {
#pragma unroll 4
    for (int sp = lot; sp < a.splits; sp += lots)
      acc += __ldcg(a.sums + (static_cast<int64_t>(sp) * hq + h) * ni + ivl);
  }
  add_shares(acc);
  for (int t = threadIdx.x; t < a.buckets; t += kThreads) {
    double s = 0.0;
    for (int i = 0; i < ni; ++i)
      if (a.m.bucket[i] == t) s += by_interval[i];
    a.dtable[static_cast<int64_t>(t) * hq + h] = __float2bfloat16_rn(static_cast<float>(s));
  }
}

// After the backward, in one launch: the table's gradient (blocks of a split and
// head) and dQ rounded to bf16 (the rest).  Bound by memory: 16K tokens of 32
// heads of 128 70 us, 403 MB (5.7 TB/s).
__global__ void __launch_bounds__(kThreads) bwd_finish_kernel(const __grid_constant__ SumArgs a,
                                                              const float4* __restrict__ dq_acc,
                                                              uint4* __restrict__ dq, int64_t dq_vecs) {
  const int hq = a.hkv * a.group, sum_blocks = hq * a.splits;
  const int bid = static_cast<int>(blockIdx.x);
  if (bid < sum_blocks) {
    dbias_sum_block(a, bid % hq, bid / hq);
    return;
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x - sum_blocks) * kThreads;
  for (int64_t i = static_cast<int64_t>(bid - sum_blocks) * kThreads + threadIdx.x; i < dq_vecs; i += stride) {
    const float4 x = dq_acc[2 * i], y = dq_acc[2 * i + 1];
    dq[i] = make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
}

int check_bias(const loong_attn_desc* d, const loong_rel_bias* b) {
  int st = loong_attn_check(d);
  if (st != LOONG_OK) return st;
  if (!b) return LOONG_ERR_INVALID_ARG;
  if (b->num_buckets < 1 || b->num_buckets > kMaxBuckets || b->num_bounds < 0 || b->num_bounds >= kMaxIntervals)
    return LOONG_ERR_INVALID_ARG;
  if (b->num_bounds > 0 && !b->bounds) return LOONG_ERR_INVALID_ARG;
  for (int i = 1; i < b->num_bounds; ++i)
    if (b->bounds[i] <= b->bounds[i - 1]) return LOONG_ERR_INVALID_ARG;
  for (int i = 0; i <= b->num_bounds; ++i) {
    const int t = b->bucket_of ? b->bucket_of[i] : i;
    if (t < 0 || t >= b->num_buckets) return LOONG_ERR_INVALID_ARG;
  }
  if (d->seqlen > kMaxSeqlen) return LOONG_ERR_UNSUPPORTED;
  if (d->softmax_scale > 0.f && d->softmax_scale < kMinScale) return LOONG_ERR_UNSUPPORTED;
  return LOONG_OK;
}

BucketMap bucket_map(const loong_rel_bias& b) {
  BucketMap m{};
  m.intervals = b.num_bounds + 1;
  for (int i = 0; i < b.num_bounds; ++i) m.bounds[i] = b.bounds[i];
  for (int i = 0; i < m.intervals; ++i) m.bucket[i] = static_cast<uint8_t>(b.bucket_of ? b.bucket_of[i] : i);
  return m;
}

// The workspace: the plain pass's first, then the bias by distance and, for the
// backward, the gradient's parts and their sums.
struct BiasWs {
  size_t lut, interval, piece, tile, vmax, part, ticket, sums, total;
  size_t clear_bytes;  // the backward's parts and tickets, from `part` on
  int off;
  int64_t len;
};

BiasWs bias_ws(const loong_attn_desc& d, const loong_rel_bias& b, int pass) {
  BiasWs w{};
  // a tile's distances reach 127 past the first and the last token's, a pair of
  // tiles' first one another 128 (causal: where only the second sees the keys)
  w.off = static_cast<int>(d.causal ? 256 : d.seqlen + 128);
  w.len = w.off + d.seqlen + 128;
  size_t at = up256(loong_attn_workspace_size(&d, pass));
  w.lut = at;
  at += up256(static_cast<size_t>(d.hq) * w.len * 4);
  w.interval = at;
  at += up256(static_cast<size_t>(w.len));
  w.piece = at;
  at += up256(static_cast<size_t>(w.len) * 4);
  w.tile = at;
  at += up256(static_cast<size_t>(w.len) * 4);
  if (pass == 0) {
    w.vmax = at;
    at += up256(kMaxBlocks * 4);
  } else {
    const size_t width = static_cast<size_t>(d.hq / d.hkv) * (b.num_bounds + 1);
    w.part = at;
    at += up256(static_cast<size_t>(bwd_blocks(d)) * kBwdComputeWarps * width * 4);
    w.ticket = at;
    at += up256(static_cast<size_t>(d.hq) * 4);
    w.clear_bytes = at - w.part;
    w.sums = at;
    at += up256(static_cast<size_t>(kSumSplits) * d.hkv * width * 8);
  }
  w.total = at;
  return w;
}

ExpandArgs expand_args(const loong_attn_desc& d, const loong_rel_bias& b, const BiasWs& w, void* ws) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / std::sqrt(static_cast<float>(d.head_dim));
  ExpandArgs a;
  a.m = bucket_map(b);
  a.table = static_cast<const __nv_bfloat16*>(b.table);
  a.hq = d.hq;
  a.inv_scale = 1.0f / scale;
  a.out.lut = reinterpret_cast<float*>(base + w.lut);
  a.out.interval = base + w.interval;
  a.out.piece = reinterpret_cast<int*>(base + w.piece);
  a.out.tile = reinterpret_cast<int*>(base + w.tile);
  a.out.len = w.len;
  a.out.off = w.off;
  a.out.intervals = a.m.intervals;
  return a;
}

int64_t expand_blocks(const BiasWs& w) { return (w.len + kThreads - 1) / kThreads; }

// At most `cap` blocks for n threads' work.
int64_t blocks_for(int64_t n, int64_t cap) {
  return std::max<int64_t>(1, std::min<int64_t>((n + kThreads - 1) / kThreads, cap));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace loong

using namespace loong;

extern "C" {

int loong_rel_bias_check(const loong_attn_desc* d, const loong_rel_bias* bias) { return check_bias(d, bias); }

size_t loong_attn_bias_workspace_size(const loong_attn_desc* d, const loong_rel_bias* bias, int pass) {
  if (check_bias(d, bias) != LOONG_OK || (pass != 0 && pass != 1)) return 0;
  return bias_ws(*d, *bias, pass).total;
}

int loong_attn_bias_fwd(const loong_attn_desc* d, const loong_rel_bias* bias, const void* q, const void* k,
                        const void* v, void* o, float* lse, void* o_res, void* ws, size_t ws_bytes,
                        loong_stream_t stream_) {
  NvtxRange range("loong_attn_bias_fwd");
  int st = check_bias(d, bias);
  if (st != LOONG_OK) return st;
  const void* ptrs[] = {q, k, v, o, lse};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 16)) return LOONG_ERR_INVALID_ARG;
  if (!aligned(o_res, 16) || !bias->table || !aligned(bias->table, 2)) return LOONG_ERR_INVALID_ARG;
  const BiasWs w = bias_ws(*d, *bias, 0);
  if (!ws || ws_bytes < w.total || !aligned(ws, 16)) return LOONG_ERR_WORKSPACE;
  if ((st = device_ready()) != LOONG_OK) return st;
  for (const void* p : ptrs)
    if (!on_device(p)) return LOONG_ERR_INVALID_ARG;
  if (!on_device(ws) || !on_device(bias->table) || (o_res && !on_device(o_res))) return LOONG_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const ExpandArgs a = expand_args(*d, *bias, w, ws);
  // short sequences spread the heads over blocks as well
  const int64_t nx = expand_blocks(w);
  const int64_t ny = std::max<int64_t>(1, std::min<int64_t>(d->hq, 608 / nx));
  uint8_t* base = static_cast<uint8_t*>(ws);
  const FwdWsLayout L = fwd_ws_layout(*d);
  VArgs va;
  va.v = static_cast<const uint4*>(v);
  va.v16 = reinterpret_cast<uint4*>(base + L.v16);
  va.amax = reinterpret_cast<unsigned*>(base + L.amax);
  va.shares = reinterpret_cast<unsigned*>(base + w.vmax);
  va.vecs = d->batch * d->seqlen * d->hkv * d->head_dim / 8;
  va.max_blocks = va.vecs <= kBlockV ? 0 : static_cast<int>(blocks_for(va.vecs / 2, kMaxBlocks));
  fwd_prep_kernel<<<static_cast<unsigned>(std::max(va.max_blocks, 1) + nx * ny), kThreads, 0, stream>>>(
      a, static_cast<int>(nx), static_cast<int>(ny), va);
  if ((st = check_launch()) != LOONG_OK) return st;
  if (va.max_blocks > 0) {
    v16_kernel<<<static_cast<unsigned>(blocks_for(va.vecs, kMaxBlocks)), kThreads, 0, stream>>>(va);
    if ((st = check_launch()) != LOONG_OK) return st;
  }
  return run_attn_fwd(*d, q, k, v, o, lse, o_res, ws, stream, &a.out);
}

int loong_attn_bias_bwd(const loong_attn_desc* d, const loong_rel_bias* bias, const void* q, const void* k,
                        const void* v, const void* o, const void* o_res, const float* lse, const void* dout, void* dq,
                        void* dk, void* dv, void* dtable, void* ws, size_t ws_bytes, loong_stream_t stream_) {
  NvtxRange range("loong_attn_bias_bwd");
  int st = check_bias(d, bias);
  if (st != LOONG_OK) return st;
  const void* ptrs[] = {q, k, v, o, lse, dout, dq, dk, dv};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 16)) return LOONG_ERR_INVALID_ARG;
  const void* tables[] = {bias->table, dtable};
  for (const void* p : tables)
    if (!p || !aligned(p, 2)) return LOONG_ERR_INVALID_ARG;
  if (!aligned(o_res, 16)) return LOONG_ERR_INVALID_ARG;
  const BiasWs w = bias_ws(*d, *bias, 1);
  if (!ws || ws_bytes < w.total || !aligned(ws, 16)) return LOONG_ERR_WORKSPACE;
  if ((st = device_ready()) != LOONG_OK) return st;
  for (const void* p : ptrs)
    if (!on_device(p)) return LOONG_ERR_INVALID_ARG;
  for (const void* p : tables)
    if (!on_device(p)) return LOONG_ERR_INVALID_ARG;
  if (!on_device(ws) || (o_res && !on_device(o_res))) return LOONG_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const ExpandArgs a = expand_args(*d, *bias, w, ws);
  const BwdWsLayout L = bwd_ws_layout(*d);
  RowStatsArgs r;
  int passes;
  if ((st = rowstats_args(*d, o, o_res, dout, lse, reinterpret_cast<float*>(base + L.stats), &r, &passes)) != LOONG_OK)
    return st;
  const int64_t dq_vecs = d->batch * d->seqlen * d->hq * d->head_dim / 8;  // of 8 elements
  ClearArgs c;
  c.dq_acc = reinterpret_cast<uint4*>(base + L.dq_acc);
  c.dq_vecs = 2 * dq_vecs;
  c.parts = reinterpret_cast<uint4*>(base + w.part);
  c.part_vecs = static_cast<int64_t>(w.clear_bytes / 16);
  const dim3 prep(static_cast<unsigned>(passes + expand_blocks(w)), static_cast<unsigned>(d->hq),
                  static_cast<unsigned>(d->batch));
  if (d->head_dim == 128)
    bwd_prep_kernel<128><<<prep, kThreads, 0, stream>>>(a, r, passes, c);
  else
    bwd_prep_kernel<64><<<prep, kThreads, 0, stream>>>(a, r, passes, c);
  if ((st = check_launch()) != LOONG_OK) return st;
  SumArgs s;
  s.m = a.m;
  s.part = reinterpret_cast<const float*>(base + w.part);
  if ((st = run_attn_bwd(*d, q, k, v, o, o_res, lse, dout, dq, dk, dv, ws, stream, &a.out,
                         reinterpret_cast<float*>(base + w.part))) != LOONG_OK)
    return st;
  const RingGeom g = ring_geom(*d);
  s.group = d->hq / d->hkv;
  s.hkv = d->hkv;
  s.nkt = g.nblocks * g.ntile;
  s.pairs = d->batch * s.nkt;
  // about 1,200 blocks, a pair each at least
  s.splits = static_cast<int>(std::min({int64_t{kSumSplits}, s.pairs, std::max<int64_t>(1, 1216 / d->hq)}));
  s.buckets = bias->num_buckets;
  s.sums = reinterpret_cast<double*>(base + w.sums);
  s.ticket = reinterpret_cast<unsigned*>(base + w.ticket);
  s.dtable = static_cast<__nv_bfloat16*>(dtable);
  bwd_finish_kernel<<<static_cast<unsigned>(d->hq * s.splits + blocks_for(dq_vecs, kMaxBlocks)), kThreads, 0, stream>>>(
      s, reinterpret_cast<const float4*>(c.dq_acc), static_cast<uint4*>(dq), dq_vecs);
  return check_launch();
}

}  // extern "C"
