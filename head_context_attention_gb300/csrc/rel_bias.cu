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
#include "v16.cuh"

namespace loong {

namespace {

constexpr int kMaxIntervals = 256;
constexpr int kMaxBuckets = 256;
constexpr int kThreads = 256;
// The finite values a bias may have.  From -kBound down it masks, as -inf does,
// from kBound up it is as +inf: a softmax reference of that size, rounded to 24
// bits, is off by up to 2^-3 in log2 units, which fp16 P still has room for (its
// bound 2^15 is half of what fp16 holds), and a score beside it has 3 bits left.
// Divided by the smallest scale accepted it is finite.
constexpr float kBound = 1048576.f;  // 2^20
constexpr float kMinScale = 5.9604645e-8f;             // 2^-24
constexpr int64_t kMaxSeqlen = int64_t{1} << 29;       // places fit 32 bits
constexpr int kSumSplits = 64;
// V of at most this many vectors of 8 is converted by one block, beside the
// expansion, else by two launches.  The forward of heads of 64, one block and two
// launches: 1,600 vectors 17.1 and 20.8 us, 4,096 21.0 and 23.0, 6,144 23.1 and
// 24.7, 8,192 25.1 and 25.2, 12,288 29.2 and 27.1.
constexpr int64_t kBlockV = 8192;

struct BucketMap {
  int intervals;
  int bounds[kMaxIntervals - 1];
  uint8_t bucket[kMaxIntervals];
};

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// One thread per distance: its interval and its pieces' by binary search, then
// the bias of heads blockIdx.y, blockIdx.y + gridDim.y, ...; consecutive threads
// write consecutive words.  The same launch clears the words that the pass adds
// into: max |V| (forward), the gradient's parts and tickets (backward).  A short
// forward's V (v_vecs vectors of 8) is also brought into its fp16 form here, by
// the last column's first block alone: max |V| and the copy are two launches
// otherwise, each longer than the work.
__global__ void __launch_bounds__(kThreads) expand_kernel(const __grid_constant__ BucketMap m,
                                                          const __nv_bfloat16* __restrict__ table, int hq,
                                                          float inv_scale, BiasView out,
                                                          uint4* __restrict__ zero, int64_t zero_vecs,
                                                          const uint4* __restrict__ v, uint4* __restrict__ v16,
                                                          unsigned* __restrict__ amax, int v_vecs) {
  if (v_vecs > 0 && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) block_v_to_f16<kThreads>(v, v16, amax, v_vecs);
    return;
  }
  const int64_t nthreads = static_cast<int64_t>(gridDim.x) * gridDim.y * kThreads;
  for (int64_t z = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + threadIdx.x; z < zero_vecs;
       z += nthreads)
    zero[z] = make_uint4(0, 0, 0, 0);
  __shared__ int bounds[kMaxIntervals];
  __shared__ uint8_t bucket[kMaxIntervals];
  for (int i = threadIdx.x; i < m.intervals; i += kThreads) {
    bounds[i] = i + 1 < m.intervals ? m.bounds[i] : 0x7fffffff;
    bucket[i] = m.bucket[i];
  }
  __syncthreads();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
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
  if (blockIdx.y == 0) {
    const_cast<uint8_t*>(out.interval)[i] = static_cast<uint8_t>(at);
    auto code = [&](int reach) {
      const int lo = interval_of(n - reach), hi = interval_of(n + reach);
      const int kind = min(hi - lo, static_cast<int>(kPieceMixed));
      return PieceCode::make(kind, lo, kind == kPieceStep ? n - bounds[lo] : 0);
    };
    const_cast<int*>(out.piece)[i] = code(31);
    const_cast<int*>(out.tile)[i] = code(127);
  }
  const __nv_bfloat16* row = table + static_cast<int64_t>(bucket[at]) * hq;
  float* lut = const_cast<float*>(out.lut);
  for (int h = blockIdx.y; h < hq; h += gridDim.y) {
    const float v = __bfloat162float(row[h]);
    lut[h * out.len + i] = v <= -kBound ? -INFINITY : v >= kBound ? INFINITY : v * inv_scale;
  }
}

// Sum of the backward's parts over warps, key tiles and sequences, in a fixed
// order: block (head, split) adds its share of the (sequence, key tile) pairs,
// `lots` threads per interval, in 32 bits over a pair's warps and in 64 beyond;
// the last block of a head to finish (tickets, cleared by expand_kernel) adds the
// splits' sums and then the intervals of every bucket.
__global__ void __launch_bounds__(kThreads) dbias_sum_kernel(const __grid_constant__ BucketMap m,
                                                             const float* __restrict__ part, int64_t pairs, int nkt,
                                                             int hkv, int group, double* __restrict__ sums,
                                                             unsigned* __restrict__ ticket, int buckets,
                                                             __nv_bfloat16* __restrict__ dtable) {
  __shared__ bool last;
  __shared__ double by_interval[kMaxIntervals], shares[kThreads];
  const int h = blockIdx.x, hq = hkv * group;
  const int kvh = h / group, g = h - kvh * group;
  const int ni = m.intervals;
  const int64_t width = static_cast<int64_t>(group) * ni;
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
  const int64_t j0 = pairs * blockIdx.y / gridDim.y, j1 = pairs * (blockIdx.y + 1) / gridDim.y;
  double acc = 0.0;
  if (mine) {
    for (int64_t j = j0; j < j1; ++j) {
      const int64_t b = j / nkt;
      const float* p = part + ((b * hkv + kvh) * nkt + (j - b * nkt)) * kBwdComputeWarps * width + g * ni + ivl;
      float s = 0.f;
#pragma unroll 4
      for (int w = lot; w < kBwdComputeWarps; w += lots) s += __ldg(p + w * width);
      acc += static_cast<double>(s);
    }
  }
  add_shares(acc);
  if (threadIdx.x < ni) sums[(static_cast<int64_t>(blockIdx.y) * hq + h) * ni + threadIdx.x] = by_interval[threadIdx.x];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(ticket + h, 1u) == gridDim.y - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  acc = 0.0;
  if (mine) {
#pragma unroll 4
    for (unsigned sp = lot; sp < gridDim.y; sp += lots) acc += __ldcg(sums + (static_cast<int64_t>(sp) * hq + h) * ni + ivl);
  }
  add_shares(acc);
  for (int t = threadIdx.x; t < buckets; t += kThreads) {
    double s = 0.0;
    for (int i = 0; i < ni; ++i)
      if (m.bucket[i] == t) s += by_interval[i];
    dtable[static_cast<int64_t>(t) * hq + h] = __float2bfloat16_rn(static_cast<float>(s));
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
  size_t lut, interval, piece, tile, zero, part, ticket, sums, total;
  size_t zero_bytes;  // from `zero` on: the forward's max |V|; the backward's parts and tickets
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
    w.zero = fwd_ws_layout(d).amax;
    w.zero_bytes = 16;
  } else {
    const size_t width = static_cast<size_t>(d.hq / d.hkv) * (b.num_bounds + 1);
    w.zero = w.part = at;
    at += up256(static_cast<size_t>(bwd_blocks(d)) * kBwdComputeWarps * width * 4);
    w.ticket = at;
    at += up256(static_cast<size_t>(d.hq) * 4);
    w.zero_bytes = at - w.zero;
    w.sums = at;
    at += up256(static_cast<size_t>(kSumSplits) * d.hkv * width * 8);
  }
  w.total = at;
  return w;
}

// v: the forward's V, or null.
int expand(const loong_attn_desc& d, const loong_rel_bias& b, const BucketMap& m, const BiasWs& w, void* ws,
           const void* v, BiasView* view, cudaStream_t stream) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  view->lut = reinterpret_cast<float*>(base + w.lut);
  view->interval = base + w.interval;
  view->piece = reinterpret_cast<int*>(base + w.piece);
  view->tile = reinterpret_cast<int*>(base + w.tile);
  view->len = w.len;
  view->off = w.off;
  view->intervals = m.intervals;
  const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / std::sqrt(static_cast<float>(d.head_dim));
  const int64_t nb = (w.len + kThreads - 1) / kThreads;
  // short sequences spread the heads over blocks as well
  const unsigned ny = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(d.hq, 608 / nb)));
  const int64_t v_vecs = d.batch * d.seqlen * d.hkv * d.head_dim / 8;
  view->v_ready = v && v_vecs <= kBlockV;
  const FwdWsLayout L = fwd_ws_layout(d);
  expand_kernel<<<dim3(static_cast<unsigned>(nb + view->v_ready), ny), kThreads, 0, stream>>>(
      m, static_cast<const __nv_bfloat16*>(b.table), d.hq, 1.0f / scale, *view,
      reinterpret_cast<uint4*>(base + w.zero), view->v_ready ? 0 : static_cast<int64_t>(w.zero_bytes / 16),
      static_cast<const uint4*>(v), reinterpret_cast<uint4*>(base + L.v16), reinterpret_cast<unsigned*>(base + L.amax),
      view->v_ready ? static_cast<int>(v_vecs) : 0);
  return check_launch();
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
  BiasView view;
  if ((st = expand(*d, *bias, bucket_map(*bias), w, ws, v, &view, stream)) != LOONG_OK) return st;
  return run_attn_fwd(*d, q, k, v, o, lse, o_res, ws, stream, &view);  // max |V| is cleared or formed
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
  float* part = reinterpret_cast<float*>(base + w.part);
  double* sums = reinterpret_cast<double*>(base + w.sums);
  const BucketMap m = bucket_map(*bias);
  BiasView view;
  if ((st = expand(*d, *bias, m, w, ws, nullptr, &view, stream)) != LOONG_OK) return st;
  if ((st = run_attn_bwd(*d, q, k, v, o, o_res, lse, dout, dq, dk, dv, ws, stream, &view, part)) != LOONG_OK) return st;
  const int group = d->hq / d->hkv;
  const RingGeom g = ring_geom(*d);
  const int nkt = g.nblocks * g.ntile;
  const int64_t pairs = d->batch * nkt;
  // about 1,200 blocks, a pair each at least
  const int splits = static_cast<int>(std::min({int64_t{kSumSplits}, pairs, std::max<int64_t>(1, 1216 / d->hq)}));
  dbias_sum_kernel<<<dim3(static_cast<unsigned>(d->hq), static_cast<unsigned>(splits)), kThreads, 0, stream>>>(
      m, part, pairs, nkt, d->hkv, group, sums, reinterpret_cast<unsigned*>(base + w.ticket),
      bias->num_buckets, static_cast<__nv_bfloat16*>(dtable));
  return check_launch();
}

}  // extern "C"
