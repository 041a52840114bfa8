// qk_norm_rope.cu -- the step between a layer's fused Q/K/V projection and its
// attention: RMS norm of every query and key head, rotation of the head's first
// rot_dim elements by the token's position, and the layout the ring kernels
// read (natural or rank-major), in one pass; and the gradient of all of it.
//
//   forward   n = x r (w + w_offset), r = rsqrt(mean(x^2) + eps)
//             (a, b) -> (a c - b s, b c + a s) for every pair of the rotated
//             part, c + i s = rot_scale exp(i pos inv_freq)
//   backward  g = the inverse rotation of dy (with rot_scale once more),
//             dw = sum g x r, h = g (w + w_offset),
//             dx = r (h - x r mean(h x r))
//
// Bound by memory: forward reads and writes every element once, backward reads
// x and dy and writes dx.  A warp owns one token at a time (or, when tokens are
// few, some of a token's heads): its lanes form the token's angles once, D / 8
// lanes hold one head (8 elements each, one 16-byte vector), so a warp
// instruction moves 512 consecutive bytes of a token.  Every lane copies its
// own vectors into shared memory asynchronously, several batches of heads (and
// the next token's) ahead of their use, and reads back only what it copied
// itself, so the warps need no barrier.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "fastdiv.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "turns.h"

namespace loong {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxFreqs = 64;        // rot_dim / 2 at head_dim 128
constexpr int kBwdMaxBlocks = 1216;  // rows of the weight gradient's partial sums

// One of Q, K, V: its side at the projection (token-strided) and at the
// attention (contiguous, natural or rank-major).
struct HeadTensor {
  const __nv_bfloat16* x;    // projection side, input (forward and backward)
  const __nv_bfloat16* dy;   // attention side, input (backward)
  __nv_bfloat16* out;        // forward: attention side; backward: projection side
  const float* w;            // [D] or null (ones)
  int64_t x_stride;          // elements per token of x
  int64_t dx_stride;         // backward: elements per token of out
  int64_t x_elems, dx_elems;  // checked build: elements from the first token's to the last one's end
  int64_t plane;             // attention side, elements of one (ring rank, head rank) plane
  int heads, hpr;            // heads, heads per head rank (heads when natural)
  int slots;                 // ceil(heads / heads per warp)
};

struct QkArgs {
  HeadTensor t[3];
  int tokens, S;           // batch * S and S
  int P, cp, zigzag, blk;  // natural: P = cp = 1, blk = S
  FastDiv by_S, by_blk;
  int64_t s_rank;
  const int64_t* positions;  // [B, S] or null
  int64_t pos_begin;
  float eps, w_offset, rot_scale;
  int rot_dim;
  int parts;             // warps that share one token's heads
  float* dw_part;        // backward: [blocks][2][D]
  int64_t out_elems[3];  // checked build: elements of the attention side
  unsigned* err;
  // inv_freq / (2 pi) modulo 1 in 64-bit fixed point (turns.h): pos * freq modulo
  // 2^64 is the angle in turns for any 64-bit position, with the table's own
  // error times pos.
  uint64_t freq[kMaxFreqs];
};

template <int D>
struct Lane {
  static constexpr int LPH = D / 8;     // lanes per head
  static constexpr int HPW = 32 / LPH;  // heads per warp instruction
  int sub, li;                          // head within the warp, lane within the head
  __device__ Lane() : sub((threadIdx.x & 31) / LPH), li((threadIdx.x & 31) % LPH) {}
};

// 8 bf16 as four pairs of fp32, for the paired fp32 instructions.
struct Vec8 {
  float2 v[4];
};

__device__ __forceinline__ Vec8 unpack8(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  Vec8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return f;
}

__device__ __forceinline__ uint4 pack8(const Vec8& f) {
  return make_uint4(pack_bf16(f.v[0].x, f.v[0].y), pack_bf16(f.v[1].x, f.v[1].y), pack_bf16(f.v[2].x, f.v[2].y),
                    pack_bf16(f.v[3].x, f.v[3].y));
}

__device__ __forceinline__ float2 dup(float x) { return make_float2(x, x); }

__device__ __forceinline__ Vec8 mul(const Vec8& a, const Vec8& b) {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], b.v[i]);
  return r;
}

__device__ __forceinline__ Vec8 mul(const Vec8& a, float b) {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], dup(b));
  return r;
}

// a b + c
__device__ __forceinline__ Vec8 fma8(const Vec8& a, const Vec8& b, const Vec8& c) {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
  return r;
}

__device__ __forceinline__ Vec8 fma8(const Vec8& a, float b, const Vec8& c) {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], dup(b), c.v[i]);
  return r;
}

__device__ __forceinline__ float dot(const Vec8& a, const Vec8& b) {
  float2 s = __fmul2_rn(a.v[0], b.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = __ffma2_rn(a.v[i], b.v[i], s);
  return s.x + s.y;
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ uint4 shfl4(const uint4& v, int src) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src),
                    __shfl_sync(0xffffffffu, v.z, src), __shfl_sync(0xffffffffu, v.w, src));
}

// The other half of every pair: lane `partner`'s 8 elements (half-split pairs)
// or this lane's own with each pair swapped (interleaved pairs).
template <bool INTER>
__device__ __forceinline__ uint4 partners(const uint4& x, int partner) {
  if constexpr (INTER)
    return make_uint4(__byte_perm(x.x, 0, 0x1032), __byte_perm(x.y, 0, 0x1032), __byte_perm(x.z, 0, 0x1032),
                      __byte_perm(x.w, 0, 0x1032));
  else
    return shfl4(x, partner);
}

// The rotation of this lane's 8 elements at one token: out = own c + other s
// with `other` the other half of each element's pair and the sign of the sine
// folded into s; its transpose is own c - other s.  Half-split pairs
// (i, i + rot_dim / 2) have their other half in lane `partner`, interleaved
// ones (2i, 2i + 1) in this lane.  Past rot_dim c = 1, s = 0.
template <int D, bool INTER>
struct Rotation {
  Vec8 c, s;
  int partner;
  int at;          // first frequency of this lane's elements
  float sign;      // of the sine
  uint64_t f0, f1;  // frequencies lane and lane + 32

  __device__ __forceinline__ void init(const QkArgs& a, const Lane<D>& ln) {
    const int lane = threadIdx.x & 31;
    const int half = a.rot_dim / 2;
    f0 = lane < half ? a.freq[lane] : 0;
    f1 = D == 128 && lane + 32 < half ? a.freq[lane + 32] : 0;
    const int e = ln.li * 8;  // this lane's first element
    const bool hi = e >= half;
    partner = lane;
    at = -1;
    if (e < a.rot_dim) {
      if (!INTER) partner = hi ? lane - half / 8 : lane + half / 8;
      at = INTER ? e / 2 : hi ? e - half : e;
    }
    sign = hi ? 1.f : -1.f;
  }
  // Every lane calls: the warp forms each angle once, in its own `table` (cosines
  // of 64 frequencies, then sines).
  __device__ __forceinline__ void form(float* table, bool wide, int64_t pos, float rot_scale) {
    const int lane = threadIdx.x & 31;
    auto put = [&](int i, uint64_t f) {
      const uint64_t turns = static_cast<uint64_t>(pos) * f;
      // the top 32 bits as a signed fraction of a turn; 2^-31 gives half turns
      const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;
      float sv, cv;
      sincospif(x, &sv, &cv);
      table[i] = cv * rot_scale;
      table[64 + i] = sv * rot_scale;
    };
    __syncwarp();  // the previous token's table has been read
    put(lane, f0);
    if (D == 128 && wide) put(lane + 32, f1);  // uniform
    __syncwarp();
    if (at < 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c.v[j] = dup(1.f);
        s.v[j] = dup(0.f);
      }
    } else if constexpr (INTER) {
      const float4 cv = *reinterpret_cast<const float4*>(table + at);
      const float4 sv = *reinterpret_cast<const float4*>(table + 64 + at);
      c.v[0] = dup(cv.x);
      c.v[1] = dup(cv.y);
      c.v[2] = dup(cv.z);
      c.v[3] = dup(cv.w);
      s.v[0] = make_float2(-sv.x, sv.x);
      s.v[1] = make_float2(-sv.y, sv.y);
      s.v[2] = make_float2(-sv.z, sv.z);
      s.v[3] = make_float2(-sv.w, sv.w);
    } else {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float4 cv = *reinterpret_cast<const float4*>(table + at + 2 * j);
        const float4 sv = *reinterpret_cast<const float4*>(table + 64 + at + 2 * j);
        c.v[j] = make_float2(cv.x, cv.y);
        c.v[j + 1] = make_float2(cv.z, cv.w);
        s.v[j] = __fmul2_rn(make_float2(sv.x, sv.y), dup(sign));
        s.v[j + 1] = __fmul2_rn(make_float2(sv.z, sv.w), dup(sign));
      }
    }
  }
};

// Where a token's rows lie on the attention side: its row (b cp + c) P of
// planes, and its position within the ring rank.
struct TokenPlace {
  int64_t rank_row, u;
  int s;  // position in the sequence
  __device__ __forceinline__ void set(const QkArgs& a, int tok) {
    const int b = static_cast<int>(fdiv(tok, a.by_S));
    s = tok - b * a.S;
    const int k = static_cast<int>(fdiv(s, a.by_blk));
    const int off = s - k * a.blk;
    const bool second = a.zigzag && k >= a.cp;
    const int c = second ? 2 * a.cp - 1 - k : k;
    u = second ? a.blk + off : off;
    rank_row = static_cast<int64_t>(b * a.cp + c) * a.P;
  }
};

// This lane's vector on the attention side, walked head by head: `at` is its
// element offset for head h = p hpr + hr, moved on by whole slots (HPW heads),
// over a head rank's end into the next one's plane.
struct AttnCursor {
  int64_t at, jump;
  int hr, hpr;
  template <int D>
  __device__ __forceinline__ void set(const TokenPlace& tp, const HeadTensor& t, int h, int li) {
    hpr = t.hpr;
    hr = h;
    jump = t.plane - static_cast<int64_t>(hpr) * D;
    at = tp.rank_row * t.plane + (tp.u * hpr + h) * D + li * 8;
    wrap();
  }
  __device__ __forceinline__ void wrap() {
    while (hr >= hpr) {  // natural layout: past the last head only
      hr -= hpr;
      at += jump;
    }
  }
  template <int D>
  __device__ __forceinline__ void next() {
    at += Lane<D>::HPW * D;
    hr += Lane<D>::HPW;
    wrap();
  }
};

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// w + w_offset of 8 elements from e
__device__ __forceinline__ Vec8 load_w(const float* w, float w_offset, int e) {
  Vec8 f;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    if (!w) {
      f.v[i] = f.v[i + 1] = dup(1.f);
      continue;
    }
    const float4 v = __ldg(reinterpret_cast<const float4*>(w + e + 2 * i));
    f.v[i] = make_float2(v.x + w_offset, v.y + w_offset);
    f.v[i + 1] = make_float2(v.z + w_offset, v.w + w_offset);
  }
  return f;
}

// 16 bytes from global to shared memory, asynchronously; `live` false writes
// zeros and reads nothing, from an address that lies in the tensor all the same
// (its first head's; an address of Q's in its place took the 128K gradient from
// 680 to 709 us).
__device__ __forceinline__ void copy16(void* dst, const __nv_bfloat16* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's newest copy groups are under way.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Checked build: what a lane names in a projection, 8 elements from p, lies in it.
__device__ __forceinline__ bool in_projection(const HeadTensor& t, const __nv_bfloat16* p, unsigned* err) {
  return in_bounds(p >= t.x && p + 8 <= t.x + t.x_elems, err);
}

// A warp's items are tokens (or ranges of a token's slots: Q's, then K's, then
// V's; a slot is the heads of one warp instruction) it, it + nwarps, ..., each
// cut into batches of up to U slots of one tensor.  This walks them ahead of
// their use, to start their copies.
template <int D, int U>
struct BatchWalk {
  uint32_t it;
  int tok, lo, hi;  // the item
  int ti, first;    // the tensor, and the item's first slot of the next one
  int h, h1;        // this lane's head of the batch's first slot, and the tensor part's end
  bool new_item, new_tensor;
  __device__ __forceinline__ bool settle(const QkArgs& a, const Lane<D>& ln, uint32_t items, uint32_t nwarps) {
    new_item = false;
    new_tensor = true;
    int s0, s1;
    do {
      if (++ti == 3) {
        it += nwarps;
        if (it >= items) {
          h = h1 = 0;
          ti = 2;
          return false;
        }
        new_item = true;
        ti = first = 0;
        item_of(a, it, tok, lo, hi);
      }
      const int n = a.t[ti].slots;
      s0 = max(lo - first, 0);
      s1 = min(hi - first, n);
      first += n;
    } while (s0 >= s1);
    h = s0 * Lane<D>::HPW + ln.sub;
    h1 = min(s1 * Lane<D>::HPW, a.t[ti].heads);
    left = s1 - s0;
    return true;
  }
  int left;  // slots from the batch's first to the tensor part's end
  static __device__ __forceinline__ void item_of(const QkArgs& a, uint32_t it, int& tok, int& lo, int& hi) {
    const int slots = a.t[0].slots + a.t[1].slots + a.t[2].slots;
    if (a.parts == 1) {
      tok = static_cast<int>(it);
      lo = 0;
      hi = slots;
    } else {
      tok = static_cast<int>(it / a.parts);
      const int part = static_cast<int>(it - static_cast<uint32_t>(tok) * a.parts);
      lo = slots * part / a.parts;
      hi = slots * (part + 1) / a.parts;
    }
  }
};

// Slots per batch and batches per warp in shared memory: the loads of DEPTH - 1
// batches are in flight while one is used.  Measured at 32 + 8 heads of 128
// (ranks' layout), forward at 32K and backward at 128K tokens: forward 2 x 6
// 127 us (6.3 TB/s; a plain copy of the same bytes 121), 2 x 3 131, 3 x 4 132,
// 4 x 6 130, 4 x 4 141, 1 x 8 135, three blocks per SM spill; backward 2 x 3
// 678 us (6.7 TB/s), 2 x 2 727, 2 x 4 681, 1 x 6 700, 3 x 2 748.  Both store
// with the streaming hint: what a pass writes is larger than L2 long before
// time matters, and kept there it delays the loads (forward 141, backward 710 us
// without).
constexpr int kFwdBatch = 2, kFwdDepth = 6, kFwdBlocks = 2;
constexpr int kBwdBatch = 2, kBwdDepth = 3, kBwdBlocks = 2;
constexpr int kTableBytes = kWarps * 128 * 4;  // a warp's cosines and sines
constexpr int kFwdSmem = kTableBytes + kWarps * kFwdDepth * kFwdBatch * 512;
constexpr int kBwdSmem = kTableBytes + kWarps * kBwdDepth * kBwdBatch * 2 * 512;

template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, kFwdBlocks) qk_fwd_kernel(const __grid_constant__ QkArgs a) {
  using L = Lane<D>;
  constexpr int U = kFwdBatch, DEPTH = kFwdDepth, HPW = L::HPW;
  extern __shared__ uint4 smem[];
  const L ln;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* table = reinterpret_cast<float*>(smem) + warp * 128;
  // this lane's vectors, 32 apart
  uint4* ring = smem + kTableBytes / 16 + warp * (DEPTH * U * 32) + lane;
  const uint32_t items = static_cast<uint32_t>(a.tokens) * a.parts, nwarps = gridDim.x * kWarps;
  const bool wide = a.rot_dim > 64;

  BatchWalk<D, U> ahead;
  const __nv_bfloat16* src = nullptr;
  bool more = true;
  auto issue = [&](int stage) {
    if (more) {
      if (ahead.left <= 0) more = ahead.settle(a, ln, items, nwarps);
      if (more) {
        if (ahead.new_tensor) src = a.t[ahead.ti].x + ahead.tok * a.t[ahead.ti].x_stride + ln.li * 8;
        ahead.new_tensor = false;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const bool live = ahead.h < ahead.h1;
          const __nv_bfloat16* from = src + (live ? ahead.h * D : 0);
          if (in_projection(a.t[ahead.ti], from, a.err)) copy16(ring + (stage * U + k) * 32, from, live);
          ahead.h += HPW;
        }
        ahead.left -= U;
      }
    }
    copy_commit();
  };
  const uint32_t it0 = blockIdx.x * kWarps + warp;
  ahead.it = it0 - nwarps;
  ahead.ti = 2;
  ahead.left = 0;
#pragma unroll 1
  for (int i = 0; i < DEPTH - 1; ++i) issue(i);

  Rotation<D, INTER> rot;
  rot.init(a, ln);
  int stage = 0;
  for (uint32_t it = it0; it < items; it += nwarps) {
    int tok, lo, hi, first = 0;
    BatchWalk<D, U>::item_of(a, it, tok, lo, hi);
    TokenPlace tp;
    tp.set(a, tok);
    rot.form(table, wide, a.positions ? __ldg(a.positions + tok) : a.pos_begin + tp.s, a.rot_scale);
#pragma unroll 1
    for (int ti = 0; ti < 3; ++ti) {
      const HeadTensor& t = a.t[ti];
      const int s0 = max(lo - first, 0), s1 = min(hi - first, t.slots);
      first += t.slots;
      if (s0 >= s1) continue;
      // y = r (x (w c) + x_other (w_other s)): the weights go into this token's cosines and sines
      Vec8 wc = rot.c, ws = rot.s;
      if (NORM && ti < 2) {
        const Vec8 w = load_w(t.w, a.w_offset, ln.li * 8);
        wc = mul(w, wc);
        if constexpr (INTER) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ws.v[i] = __fmul2_rn(make_float2(w.v[i].y, w.v[i].x), ws.v[i]);
        } else {
          ws = mul(load_w(t.w, a.w_offset, (rot.partner % L::LPH) * 8), ws);
        }
      }
      int h = s0 * HPW + ln.sub;
      const int h1 = min(s1 * HPW, t.heads);
      AttnCursor out;
      out.set<D>(tp, t, h, ln.li);
      for (int sl = s0; sl < s1; sl += U) {
        issue(stage == 0 ? DEPTH - 1 : stage - 1);
        copy_wait<DEPTH - 1>();
        uint4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) x[k] = ring[(stage * U + k) * 32];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (sl + k >= s1) break;  // uniform
          uint4 y = x[k];
          if (ti < 2) {
            const Vec8 f = unpack8(x[k]);
            Vec8 g = unpack8(partners<INTER>(x[k], rot.partner));
            g = fma8(g, ws, mul(f, wc));
            if (NORM) g = mul(g, rsqrtf(head_sum<L::LPH>(dot(f, f)) * (1.f / D) + a.eps));
            y = pack8(g);
          }
          if (h < h1 && in_bounds(out.at >= 0 && out.at + 8 <= a.out_elems[ti], a.err))
            __stcs(reinterpret_cast<uint4*>(t.out + out.at), y);
          h += HPW;
          out.next<D>();
        }
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
      }
    }
  }
}

template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  using L = Lane<D>;
  constexpr int U = kBwdBatch, DEPTH = kBwdDepth, HPW = L::HPW;
  extern __shared__ uint4 smem[];
  const L ln;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* table = reinterpret_cast<float*>(smem) + warp * 128;
  // per stage: U vectors of dy, then U of x
  uint4* ring = smem + kTableBytes / 16 + warp * (DEPTH * U * 2 * 32) + lane;
  // The weight gradients of this warp: per lane, 8 elements of Q's and of K's,
  // summed in registers over one token's heads and then here over its tokens
  // (two short chains instead of one long one).
  __shared__ float4 dw_sh[NORM ? 2 : 1][NORM ? 2 : 1][NORM ? kThreads : 1];
  if (NORM)
    for (int i = 0; i < 4; ++i) dw_sh[i >> 1][i & 1][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  const uint32_t items = static_cast<uint32_t>(a.tokens) * a.parts, nwarps = gridDim.x * kWarps;
  const bool wide = a.rot_dim > 64;

  BatchWalk<D, U> ahead;
  TokenPlace ahead_tp;
  const __nv_bfloat16* src = nullptr;
  AttnCursor in;
  bool more = true;
  auto issue = [&](int stage) {
    if (more) {
      if (ahead.left <= 0) more = ahead.settle(a, ln, items, nwarps);
      if (more) {
        const HeadTensor& t = a.t[ahead.ti];
        if (ahead.new_item) ahead_tp.set(a, ahead.tok);
        if (ahead.new_tensor) {
          src = t.x + ahead.tok * t.x_stride + ln.li * 8;
          in.set<D>(ahead_tp, t, ahead.h, ln.li);
        }
        ahead.new_item = ahead.new_tensor = false;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const bool live = ahead.h < ahead.h1;
          const bool ok = live && in_bounds(in.at >= 0 && in.at + 8 <= a.out_elems[ahead.ti], a.err);
          copy16(ring + (stage * 2 * U + k) * 32, t.dy + (ok ? in.at : 0), ok);
          if (NORM && ahead.ti < 2) {
            const __nv_bfloat16* from = src + (live ? ahead.h * D : 0);
            if (in_projection(t, from, a.err)) copy16(ring + ((stage * 2 + 1) * U + k) * 32, from, live);
          }
          ahead.h += HPW;
          in.next<D>();
        }
        ahead.left -= U;
      }
    }
    copy_commit();
  };
  const uint32_t it0 = blockIdx.x * kWarps + warp;
  ahead.it = it0 - nwarps;
  ahead.ti = 2;
  ahead.left = 0;
#pragma unroll 1
  for (int i = 0; i < DEPTH - 1; ++i) issue(i);

  Rotation<D, INTER> rot;
  rot.init(a, ln);
  rot.sign = -rot.sign;  // the transpose
  int stage = 0;
  for (uint32_t it = it0; it < items; it += nwarps) {
    int tok, lo, hi, first = 0;
    BatchWalk<D, U>::item_of(a, it, tok, lo, hi);
    const int s = tok - static_cast<int>(fdiv(tok, a.by_S)) * a.S;
    rot.form(table, wide, a.positions ? __ldg(a.positions + tok) : a.pos_begin + s, a.rot_scale);
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) rot.s.v[i] = make_float2(-rot.s.v[i].x, -rot.s.v[i].y);
    }
#pragma unroll 1
    for (int ti = 0; ti < 3; ++ti) {
      const HeadTensor& t = a.t[ti];
      const int s0 = max(lo - first, 0), s1 = min(hi - first, t.slots);
      first += t.slots;
      if (s0 >= s1) continue;
      const bool normed = NORM && ti < 2;
      Vec8 w, dw{};
      if (normed) w = load_w(t.w, a.w_offset, ln.li * 8);
      int h = s0 * HPW + ln.sub;
      const int h1 = min(s1 * HPW, t.heads);
      __nv_bfloat16* dst = t.out + tok * t.dx_stride + h * D + ln.li * 8;
      for (int sl = s0; sl < s1; sl += U) {
        issue(stage == 0 ? DEPTH - 1 : stage - 1);
        copy_wait<DEPTH - 1>();
        uint4 dy[U], x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          dy[k] = ring[(stage * 2 * U + k) * 32];
          if (normed) x[k] = ring[((stage * 2 + 1) * U + k) * 32];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (sl + k >= s1) break;  // uniform
          uint4 y = dy[k];
          if (ti < 2) {
            Vec8 g = mul(unpack8(dy[k]), rot.c);
            g = fma8(unpack8(partners<INTER>(dy[k], rot.partner)), rot.s, g);
            if (NORM) {
              const Vec8 f = unpack8(x[k]);
              const Vec8 gx = mul(g, f);
              const float ss = head_sum<L::LPH>(dot(f, f)), gwx = head_sum<L::LPH>(dot(gx, w));
              const float r = rsqrtf(ss * (1.f / D) + a.eps);
              dw = fma8(gx, h < h1 ? r : 0.f, dw);  // past the last head x is 0 and, with eps 0, r infinite
              // dx = r (g w - x r mean(g w x r))
              g = mul(fma8(f, -r * (r * gwx * (1.f / D)), mul(g, w)), r);
            }
            y = pack8(g);
          }
          if (h < h1 && in_bounds(dst >= t.out && dst + 8 <= t.out + t.dx_elems, a.err))
            __stcs(reinterpret_cast<uint4*>(dst), y);
          h += HPW;
          dst += HPW * D;
        }
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
      }
      if (normed) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float4 v = dw_sh[ti][i][threadIdx.x];
          v.x += dw.v[2 * i].x;
          v.y += dw.v[2 * i].y;
          v.z += dw.v[2 * i + 1].x;
          v.w += dw.v[2 * i + 1].y;
          dw_sh[ti][i][threadIdx.x] = v;
        }
      }
    }
  }
  if (NORM && a.dw_part) {
    __syncthreads();
    // element e of a head lies in lanes li = e / 8 of every head slot of every warp
    for (int j = threadIdx.x; j < 2 * D; j += kThreads) {
      const int ti = j / D, e = j % D;
      float sum = 0.f;
      for (int th = e / 8; th < kThreads; th += L::LPH)
        sum += reinterpret_cast<const float*>(&dw_sh[ti][(e % 8) / 4][th])[e % 4];
      a.dw_part[static_cast<int64_t>(blockIdx.x) * 2 * D + j] = sum;
    }
  }
}

// dw[e] = sum over the blocks' partial sums, always in the same order: a block
// owns 32 elements, its warps every 32nd row each (one 128-byte line a row), in
// 64 bits.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) dw_sum_kernel(const float* __restrict__ part, int blocks, int d,
                                                             float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ double by_warp[kSumThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;  // of 2 d, a multiple of 32
  double s = 0.0;
#pragma unroll 8
  for (int b = warp; b < blocks; b += kSumThreads / 32) s += __ldg(part + static_cast<int64_t>(b) * 2 * d + j);
  by_warp[warp][lane] = s;
  __syncthreads();
  if (warp > 0) return;
  double t[4] = {};
#pragma unroll
  for (int w = 0; w < kSumThreads / 32; ++w) t[w & 3] += by_warp[w][lane];
  float* dst = j < d ? dwq : dwk;
  if (dst) dst[j < d ? j : j - d] = static_cast<float>((t[0] + t[1]) + (t[2] + t[3]));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_opts(const loong_attn_desc& d, const loong_qk_opts* o) {
  if (!o) return LOONG_ERR_INVALID_ARG;
  if (o->norm != 0 && o->norm != 1) return LOONG_ERR_INVALID_ARG;
  if (o->interleaved != 0 && o->interleaved != 1) return LOONG_ERR_INVALID_ARG;
  if (o->rot_dim < 0 || o->rot_dim > d.head_dim || o->rot_dim % 16) return LOONG_ERR_INVALID_ARG;
  if (o->norm && !(o->eps >= 0.f && std::isfinite(o->eps))) return LOONG_ERR_INVALID_ARG;
  if (!std::isfinite(o->w_offset) || !std::isfinite(o->rot_scale)) return LOONG_ERR_INVALID_ARG;
  if (o->rot_dim > 0) {
    if (o->inv_freq) {
      for (int i = 0; i < o->rot_dim / 2; ++i)
        if (!std::isfinite(o->inv_freq[i])) return LOONG_ERR_INVALID_ARG;
    } else if (!(o->rot_base >= DBL_MIN) || !std::isfinite(o->rot_base)) {
      return LOONG_ERR_INVALID_ARG;  // below DBL_MIN the last frequencies are infinite
    }
  }
  const int64_t stride[6] = {o->q_stride, o->k_stride, o->v_stride, o->dq_stride, o->dk_stride, o->dv_stride};
  for (int i = 0; i < 6; ++i) {
    const int64_t row = static_cast<int64_t>(i % 3 == 0 ? d.hq : d.hkv) * d.head_dim;
    if (stride[i] != 0 && (stride[i] < row || stride[i] % 8 || stride[i] > (int64_t{1} << 31)))
      return LOONG_ERR_INVALID_ARG;
  }
  return LOONG_OK;
}

void fill_args(QkArgs& a, const loong_attn_desc& d, const loong_qk_opts& o, const int64_t* positions, bool with_v) {
  const bool rm = d.layout == LOONG_LAYOUT_RANK_MAJOR;
  const RingGeom g = ring_geom(d);
  const int hpw = 32 / (d.head_dim / 8);
  a.tokens = static_cast<int>(d.batch * d.seqlen);
  a.S = static_cast<int>(d.seqlen);
  a.P = rm ? d.hp : 1;
  a.cp = rm ? d.cp : 1;
  a.zigzag = rm && g.zigzag;
  a.blk = rm ? g.blk : a.S;
  a.s_rank = d.seqlen / a.cp;
  a.by_S = make_fastdiv(static_cast<uint32_t>(a.S));
  a.by_blk = make_fastdiv(static_cast<uint32_t>(a.blk));
  a.positions = positions;
  a.pos_begin = o.pos_begin;
  a.eps = o.eps;
  a.w_offset = o.w_offset;
  a.rot_scale = o.rot_scale;
  a.rot_dim = o.rot_dim;
  const int64_t x_stride[3] = {o.q_stride, o.k_stride, o.v_stride};
  const int64_t dx_stride[3] = {o.dq_stride, o.dk_stride, o.dv_stride};
  const int heads[3] = {d.hq, d.hkv, d.hkv};
  for (int i = 0; i < 3; ++i) {
    HeadTensor& t = a.t[i];
    const int64_t row = static_cast<int64_t>(heads[i]) * d.head_dim;
    t.heads = heads[i];
    t.hpr = heads[i] / a.P;
    t.x_stride = x_stride[i] ? x_stride[i] : row;
    t.dx_stride = dx_stride[i] ? dx_stride[i] : row;
    t.x_elems = (a.tokens - int64_t{1}) * t.x_stride + row;
    t.dx_elems = (a.tokens - int64_t{1}) * t.dx_stride + row;
    t.plane = a.s_rank * t.hpr * d.head_dim;
    t.slots = i == 2 && !with_v ? 0 : (heads[i] + hpw - 1) / hpw;
    a.out_elems[i] = static_cast<int64_t>(a.tokens) * row;
  }
  for (int i = 0; i < o.rot_dim / 2; ++i)
    a.freq[i] = turn_fraction(o.inv_freq ? o.inv_freq[i] : std::pow(o.rot_base, -2.0 * i / o.rot_dim));
}

// Blocks of the launch, and in a.parts how many warps share a token: one when
// the tokens alone give every resident warp one, more (up to one per slot of
// heads) when they do not.  (Three items per warp instead of one: 3,003 tokens of
// 10 + 5 heads of 64 forward 15.5 us for 13.4, 512 of 32 + 8 of 128 14.5 for 11.4;
// every item forms its token's angles again.)
unsigned plan_grid(QkArgs& a, int blocks_per_sm, int max_blocks) {
  const int slots = a.t[0].slots + a.t[1].slots + a.t[2].slots;
  const int64_t cap = std::min<int64_t>(static_cast<int64_t>(num_sms()) * blocks_per_sm, max_blocks);
  const int64_t warps = cap * kWarps;
  a.parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(slots, warps / a.tokens)));
  const int64_t items = static_cast<int64_t>(a.tokens) * a.parts;
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(cap, (items + kWarps - 1) / kWarps)));
}

using QkKernel = void (*)(QkArgs);

int launch(QkKernel kern, int smem, unsigned grid, const QkArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e);
  kern<<<grid, kThreads, smem, s>>>(a);
  return check_launch();
}

template <int D>
QkKernel fwd_kernel(bool inter, bool norm) {
  if (inter) return norm ? qk_fwd_kernel<D, true, true> : qk_fwd_kernel<D, true, false>;
  return norm ? qk_fwd_kernel<D, false, true> : qk_fwd_kernel<D, false, false>;
}

template <int D>
QkKernel bwd_kernel(bool inter, bool norm) {
  if (inter) return norm ? qk_bwd_kernel<D, true, true> : qk_bwd_kernel<D, true, false>;
  return norm ? qk_bwd_kernel<D, false, true> : qk_bwd_kernel<D, false, false>;
}

}  // namespace

}  // namespace loong

using namespace loong;

extern "C" {

int loong_qk_norm_rope_fwd(const loong_attn_desc* d, const loong_qk_opts* opts, const void* q, const void* k,
                           const void* v, const float* wq, const float* wk, const int64_t* positions, void* q_out,
                           void* k_out, void* v_out, loong_stream_t stream_) {
  NvtxRange range("loong_qk_norm_rope_fwd");
  int st = loong_attn_check(d);
  if (st != LOONG_OK) return st;
  if ((st = check_opts(*d, opts)) != LOONG_OK) return st;
  if (!q || !k || !q_out || !k_out || !v != !v_out) return LOONG_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, wq, wk, q_out, k_out, v_out};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return LOONG_ERR_INVALID_ARG;
  if (!aligned(positions, 8)) return LOONG_ERR_INVALID_ARG;
  if ((st = device_ready()) != LOONG_OK) return st;
  for (const void* p : ptrs)
    if (p && !on_device(p)) return LOONG_ERR_INVALID_ARG;
  if (positions && !on_device(positions)) return LOONG_ERR_INVALID_ARG;
  QkArgs a{};
  fill_args(a, *d, *opts, positions, v != nullptr);
  if (!(a.err = device_error_word())) return LOONG_ERR_CUDA;
  const void* in[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  const float* w[3] = {wq, wk, nullptr};
  for (int i = 0; i < 3; ++i) {
    a.t[i].x = static_cast<const __nv_bfloat16*>(in[i]);
    a.t[i].out = static_cast<__nv_bfloat16*>(out[i]);
    a.t[i].w = w[i];
  }
  const unsigned grid = plan_grid(a, kFwdBlocks, 1 << 20);
  return launch(d->head_dim == 128 ? fwd_kernel<128>(opts->interleaved, opts->norm)
                                   : fwd_kernel<64>(opts->interleaved, opts->norm),
                kFwdSmem, grid, a, reinterpret_cast<cudaStream_t>(stream_));
}

size_t loong_qk_norm_rope_bwd_workspace_size(const loong_attn_desc* d, const loong_qk_opts* opts) {
  if (loong_attn_check(d) != LOONG_OK || check_opts(*d, opts) != LOONG_OK) return 0;
  return opts->norm ? static_cast<size_t>(kBwdMaxBlocks) * 2 * d->head_dim * 4 : 0;
}

int loong_qk_norm_rope_bwd(const loong_attn_desc* d, const loong_qk_opts* opts, const void* q, const void* k,
                           const float* wq, const float* wk, const int64_t* positions, const void* dq_out,
                           const void* dk_out, const void* dv_out, void* dq, void* dk, void* dv, float* dwq, float* dwk,
                           void* ws, size_t ws_bytes, loong_stream_t stream_) {
  NvtxRange range("loong_qk_norm_rope_bwd");
  int st = loong_attn_check(d);
  if (st != LOONG_OK) return st;
  if ((st = check_opts(*d, opts)) != LOONG_OK) return st;
  if (!dq_out || !dk_out || !dq || !dk || !dv_out != !dv) return LOONG_ERR_INVALID_ARG;
  if (opts->norm && (!q || !k)) return LOONG_ERR_INVALID_ARG;
  if (!opts->norm && (dwq || dwk)) return LOONG_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, wq, wk, dq_out, dk_out, dv_out, dq, dk, dv};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return LOONG_ERR_INVALID_ARG;
  if (!aligned(positions, 8) || !aligned(dwq, 4) || !aligned(dwk, 4)) return LOONG_ERR_INVALID_ARG;
  const bool want_dw = dwq || dwk;
  if (want_dw && (!ws || ws_bytes < loong_qk_norm_rope_bwd_workspace_size(d, opts) || !aligned(ws, 16)))
    return LOONG_ERR_WORKSPACE;
  if ((st = device_ready()) != LOONG_OK) return st;
  for (const void* p : ptrs)
    if (p && !on_device(p)) return LOONG_ERR_INVALID_ARG;
  const void* more[] = {positions, dwq, dwk, want_dw ? ws : nullptr};
  for (const void* p : more)
    if (p && !on_device(p)) return LOONG_ERR_INVALID_ARG;
  QkArgs a{};
  fill_args(a, *d, *opts, positions, dv != nullptr);
  if (!(a.err = device_error_word())) return LOONG_ERR_CUDA;
  const void* x[3] = {q, k, nullptr};
  const void* dy[3] = {dq_out, dk_out, dv_out};
  void* out[3] = {dq, dk, dv};
  const float* w[3] = {wq, wk, nullptr};
  for (int i = 0; i < 3; ++i) {
    a.t[i].x = static_cast<const __nv_bfloat16*>(x[i]);
    a.t[i].dy = static_cast<const __nv_bfloat16*>(dy[i]);
    a.t[i].out = static_cast<__nv_bfloat16*>(out[i]);
    a.t[i].w = w[i];
  }
  a.dw_part = want_dw ? static_cast<float*>(ws) : nullptr;
  const unsigned grid = plan_grid(a, kBwdBlocks, kBwdMaxBlocks);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  st = launch(d->head_dim == 128 ? bwd_kernel<128>(opts->interleaved, opts->norm)
                                 : bwd_kernel<64>(opts->interleaved, opts->norm),
              kBwdSmem, grid, a, s);
  if (st != LOONG_OK || !want_dw) return st;
  dw_sum_kernel<<<2 * d->head_dim / 32, kSumThreads, 0, s>>>(a.dw_part, static_cast<int>(grid), d->head_dim, dwq, dwk);
  return check_launch();
}

}  // extern "C"
