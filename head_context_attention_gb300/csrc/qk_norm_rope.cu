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
// instruction moves 512 consecutive bytes of a token, and kUnroll heads' loads
// are in flight per lane before the first is used.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

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
  int64_t plane;             // attention side, elements of one (ring rank, head rank) plane
  int heads, hpr;            // heads, heads per head rank (heads when natural)
  int slots;                 // ceil(heads / heads per warp)
};

struct QkArgs {
  HeadTensor t[3];
  int tokens, S;           // batch * S and S
  int P, cp, zigzag, blk;  // natural: P = cp = 1, blk = S
  int64_t s_rank;
  const int64_t* positions;  // [B, S] or null
  int64_t pos_begin;
  float eps, w_offset, rot_scale;
  int rot_dim;
  int parts;             // warps that share one token's heads
  float* dw_part;        // backward: [blocks][2][D]
  int64_t out_elems[3];  // checked build: elements of the attention side
  unsigned* err;
  // inv_freq / (2 pi) modulo 1 in 64-bit fixed point: pos * freq modulo 2^64 is
  // the angle in turns for any 64-bit position, with the table's own error
  // (2^-53 relative to inv_freq) times pos.
  uint64_t freq[kMaxFreqs];
};

template <int D>
struct Lane {
  static constexpr int LPH = D / 8;     // lanes per head
  static constexpr int HPW = 32 / LPH;  // heads per warp instruction
  int sub, li;                          // head within the warp, lane within the head
  __device__ Lane() : sub((threadIdx.x & 31) / LPH), li((threadIdx.x & 31) % LPH) {}
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
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

// The rotation of this lane's 8 elements at one token.  Half-split pairs
// (i, i + rot_dim / 2): out_i = own_i c_i + partner_i s_i, with the partner's 8
// elements in lane `partner` and the sign of the sine folded into s.
// Interleaved pairs (2i, 2i + 1) lie inside the lane: c, s of pair j in c[j], s[j].
// A lane past rot_dim has c = 1, s = 0.
template <int D, bool INTER>
struct Rotation {
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
  int partner;

  // Lane l holds frequencies l and l + 32 (f0, f1); every lane calls.
  __device__ __forceinline__ void form(const Lane<D>& ln, int rot_dim, uint64_t f0, uint64_t f1, int64_t pos,
                                       float rot_scale) {
    const int lane = threadIdx.x & 31;
    const int half = rot_dim / 2;
    float c0, s0, c1 = 1.f, s1 = 0.f;
    auto sincos_turns = [&](uint64_t f, float& cv, float& sv) {
      const uint64_t turns = static_cast<uint64_t>(pos) * f;
      // the top 32 bits as a signed fraction of a turn; 2^-31 gives half turns
      const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;
      sincospif(x, &sv, &cv);
      cv *= rot_scale;
      sv *= rot_scale;
    };
    sincos_turns(f0, c0, s0);
    if (half > 32) sincos_turns(f1, c1, s1);  // uniform
    const int e = ln.li * 8;                  // this lane's first element
    const bool rotated = e < rot_dim;
    partner = lane;
    if constexpr (INTER) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = e / 2 + j;
        const float ca = __shfl_sync(0xffffffffu, c0, i & 31), cb = __shfl_sync(0xffffffffu, c1, i & 31);
        const float sa = __shfl_sync(0xffffffffu, s0, i & 31), sb = __shfl_sync(0xffffffffu, s1, i & 31);
        c[j] = rotated ? (i < 32 ? ca : cb) : 1.f;
        s[j] = rotated ? (i < 32 ? sa : sb) : 0.f;
      }
    } else {
      const bool hi = e >= half;
      if (rotated) partner = hi ? lane - half / 8 : lane + half / 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = (hi ? e - half : e) + j;
        const float ca = __shfl_sync(0xffffffffu, c0, i & 31), cb = __shfl_sync(0xffffffffu, c1, i & 31);
        const float sa = __shfl_sync(0xffffffffu, s0, i & 31), sb = __shfl_sync(0xffffffffu, s1, i & 31);
        const float sj = i < 32 ? sa : sb;
        c[j] = rotated ? (i < 32 ? ca : cb) : 1.f;
        s[j] = rotated ? (hi ? sj : -sj) : 0.f;
      }
    }
  }
};

// Token of a warp's work item and where its rows lie on both sides.
struct TokenPlace {
  int tok;
  int64_t rank_row;  // (b cp + c) P
  int64_t u;         // position within the ring rank
  int64_t pos;
  __device__ __forceinline__ void set(const QkArgs& a, int tok_) {
    tok = tok_;
    const int b = tok / a.S;
    const int s = tok - b * a.S;
    const int k = s / a.blk;
    const int off = s - k * a.blk;
    int c = k;
    u = off;
    if (a.zigzag && k >= a.cp) {
      c = 2 * a.cp - 1 - k;
      u = a.blk + off;
    }
    rank_row = (static_cast<int64_t>(b) * a.cp + c) * a.P;
    pos = a.positions ? __ldg(a.positions + tok) : a.pos_begin + s;
  }
  // element offset of head h on the attention side
  template <int D>
  __device__ __forceinline__ int64_t attn(const QkArgs& a, const HeadTensor& t, int h) const {
    const int p = a.P == 1 ? 0 : h / t.hpr;
    return (rank_row + p) * t.plane + (u * t.hpr + (h - p * t.hpr)) * D;
  }
  template <int D>
  __device__ __forceinline__ int64_t proj(int64_t stride, int h) const {
    return tok * stride + static_cast<int64_t>(h) * D;
  }
};

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// w + w_offset of 8 elements from e
__device__ __forceinline__ void load_w(const float* w, float w_offset, int e, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(w + e + i));
    f[i] = v.x + w_offset;
    f[i + 1] = v.y + w_offset;
    f[i + 2] = v.z + w_offset;
    f[i + 3] = v.w + w_offset;
  }
}

constexpr int kUnroll = 4;

template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const __grid_constant__ QkArgs a) {
  using L = Lane<D>;
  const L ln;
  const int lane = threadIdx.x & 31;
  const int half = a.rot_dim / 2;
  const uint64_t f0 = lane < half ? a.freq[lane] : 0, f1 = lane + 32 < half ? a.freq[lane + 32] : 0;
  const int slots = a.t[0].slots + a.t[1].slots + a.t[2].slots;
  const int64_t items = static_cast<int64_t>(a.tokens) * a.parts;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += nwarps) {
    const int tok = static_cast<int>(it / a.parts);
    const int part = static_cast<int>(it - static_cast<int64_t>(tok) * a.parts);
    const int lo = static_cast<int>(static_cast<int64_t>(slots) * part / a.parts);
    const int hi = static_cast<int>(static_cast<int64_t>(slots) * (part + 1) / a.parts);
    TokenPlace tp;
    tp.set(a, tok);
    Rotation<D, INTER> rot;
    rot.form(ln, a.rot_dim, f0, f1, tp.pos, a.rot_scale);
    int first = 0;  // the tensor's first slot
#pragma unroll 1
    for (int ti = 0; ti < 3; ++ti) {
      const HeadTensor& t = a.t[ti];
      const int s0 = max(lo, first) - first, s1 = min(hi, first + t.slots) - first;
      first += t.slots;
      if (s0 >= s1) continue;
      float w[8], wp[8];
      if (NORM && ti < 2) {
        load_w(t.w, a.w_offset, ln.li * 8, w);
        if (!INTER) load_w(t.w, a.w_offset, (rot.partner % L::LPH) * 8, wp);
      }
      for (int sl = s0; sl < s1; sl += kUnroll) {
        uint4 x[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const int h = (sl + k) * L::HPW + ln.sub;
          x[k] = make_uint4(0, 0, 0, 0);
          if (sl + k < s1 && h < t.heads) x[k] = load16(t.x + tp.proj<D>(t.x_stride, h) + ln.li * 8);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          if (sl + k >= s1) break;  // uniform
          const int h = (sl + k) * L::HPW + ln.sub;
          uint4 y = x[k];
          if (ti < 2) {
            float f[8];
            unpack8(x[k], f);
            float r = 1.f;
            if (NORM) {
              float ss = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
              r = rsqrtf(head_sum<L::LPH>(ss) * (1.f / D) + a.eps);
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] *= r * w[i];
            }
            if constexpr (INTER) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float u = f[2 * j], v = f[2 * j + 1];
                f[2 * j] = u * rot.c[j] - v * rot.s[j];
                f[2 * j + 1] = v * rot.c[j] + u * rot.s[j];
              }
            } else {
              float g[8];
              unpack8(shfl4(x[k], rot.partner), g);  // the partner's raw elements: the head's r is shared
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float gp = NORM ? g[i] * (r * wp[i]) : g[i];
                f[i] = fmaf(f[i], rot.c[i], gp * rot.s[i]);
              }
            }
            y = pack8(f);
          }
          if (h < t.heads) {
            const int64_t o = tp.attn<D>(a, t, h) + ln.li * 8;
            if (in_bounds(o >= 0 && o + 8 <= a.out_elems[ti], a.err)) *reinterpret_cast<uint4*>(t.out + o) = y;
          }
        }
      }
    }
  }
}

constexpr int kBwdUnroll = 2;

template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  using L = Lane<D>;
  const L ln;
  // The weight gradients of this warp: per lane, 8 elements of Q's and of K's,
  // summed in registers over one token's heads and then here over its tokens
  // (two short chains instead of one long one).
  __shared__ float4 dw_sh[NORM ? 2 : 1][NORM ? 2 : 1][NORM ? kThreads : 1];
  if (NORM)
    for (int i = 0; i < 4; ++i) dw_sh[i >> 1][i & 1][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int lane = threadIdx.x & 31;
  const int half = a.rot_dim / 2;
  const uint64_t f0 = lane < half ? a.freq[lane] : 0, f1 = lane + 32 < half ? a.freq[lane + 32] : 0;
  const int slots = a.t[0].slots + a.t[1].slots + a.t[2].slots;
  const int64_t items = static_cast<int64_t>(a.tokens) * a.parts;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += nwarps) {
    const int tok = static_cast<int>(it / a.parts);
    const int part = static_cast<int>(it - static_cast<int64_t>(tok) * a.parts);
    const int lo = static_cast<int>(static_cast<int64_t>(slots) * part / a.parts);
    const int hi = static_cast<int>(static_cast<int64_t>(slots) * (part + 1) / a.parts);
    TokenPlace tp;
    tp.set(a, tok);
    Rotation<D, INTER> rot;
    rot.form(ln, a.rot_dim, f0, f1, tp.pos, a.rot_scale);
    int first = 0;
#pragma unroll 1
    for (int ti = 0; ti < 3; ++ti) {
      const HeadTensor& t = a.t[ti];
      const int s0 = max(lo, first) - first, s1 = min(hi, first + t.slots) - first;
      first += t.slots;
      if (s0 >= s1) continue;
      const bool normed = NORM && ti < 2;
      float w[8], dw[8] = {};
      if (normed) load_w(t.w, a.w_offset, ln.li * 8, w);
      for (int sl = s0; sl < s1; sl += kBwdUnroll) {
        uint4 x[kBwdUnroll], dy[kBwdUnroll];
#pragma unroll
        for (int k = 0; k < kBwdUnroll; ++k) {
          const int h = (sl + k) * L::HPW + ln.sub;
          x[k] = dy[k] = make_uint4(0, 0, 0, 0);
          if (sl + k < s1 && h < t.heads) {
            if (normed) x[k] = load16(t.x + tp.proj<D>(t.x_stride, h) + ln.li * 8);
            const int64_t o = tp.attn<D>(a, t, h) + ln.li * 8;
            if (in_bounds(o >= 0 && o + 8 <= a.out_elems[ti], a.err)) dy[k] = load16(t.dy + o);
          }
        }
#pragma unroll
        for (int k = 0; k < kBwdUnroll; ++k) {
          if (sl + k >= s1) break;  // uniform
          const int h = (sl + k) * L::HPW + ln.sub;
          uint4 y = dy[k];
          if (ti < 2) {
            float g[8];
            unpack8(dy[k], g);
            if constexpr (INTER) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float u = g[2 * j], v = g[2 * j + 1];
                g[2 * j] = u * rot.c[j] + v * rot.s[j];
                g[2 * j + 1] = v * rot.c[j] - u * rot.s[j];
              }
            } else {
              float p[8];
              unpack8(shfl4(dy[k], rot.partner), p);
#pragma unroll
              for (int i = 0; i < 8; ++i) g[i] = fmaf(g[i], rot.c[i], -p[i] * rot.s[i]);
            }
            if (NORM) {
              float f[8];
              unpack8(x[k], f);
              float ss = 0.f, dot = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                ss = fmaf(f[i], f[i], ss);
                dot = fmaf(g[i] * w[i], f[i], dot);
              }
              ss = head_sum<L::LPH>(ss);
              dot = head_sum<L::LPH>(dot);
              const float r = rsqrtf(ss * (1.f / D) + a.eps);
              const float m = dot * r * (1.f / D);  // mean(h x r)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float xr = f[i] * r;
                dw[i] = fmaf(g[i], xr, dw[i]);
                g[i] = r * fmaf(-xr, m, g[i] * w[i]);
              }
            }
            y = pack8(g);
          }
          if (h < t.heads) *reinterpret_cast<uint4*>(t.out + tp.proj<D>(t.dx_stride, h) + ln.li * 8) = y;
        }
      }
      if (normed) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float4 v = dw_sh[ti][i][threadIdx.x];
          v.x += dw[4 * i];
          v.y += dw[4 * i + 1];
          v.z += dw[4 * i + 2];
          v.w += dw[4 * i + 3];
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

// dw[e] = sum over the blocks' partial sums, always in the same order: one warp
// per element, in 64 bits.
__global__ void __launch_bounds__(kThreads) dw_sum_kernel(const float* __restrict__ part, int blocks, int d,
                                                          float* __restrict__ dwq, float* __restrict__ dwk) {
  const int j = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (j >= 2 * d) return;
  double s = 0.0;
  for (int b = threadIdx.x & 31; b < blocks; b += 32) s += part[static_cast<int64_t>(b) * 2 * d + j];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  float* dst = j < d ? dwq : dwk;
  if ((threadIdx.x & 31) == 0 && dst) dst[j < d ? j : j - d] = static_cast<float>(s);
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
    } else if (!(o->rot_base > 0.0) || !std::isfinite(o->rot_base)) {
      return LOONG_ERR_INVALID_ARG;
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

// inv_freq / (2 pi) modulo 1 as a 64-bit fraction.
uint64_t turn_fraction(double inv_freq) {
  double t = inv_freq / 6.283185307179586476925;
  t -= std::floor(t);
  if (t >= 1.0) t = 0.0;  // a tiny negative frequency rounds up to a whole turn
  const double hi = std::floor(t * 4294967296.0);
  const double lo = (t * 4294967296.0 - hi) * 4294967296.0;  // exact: powers of two
  return (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo);
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
    t.plane = a.s_rank * t.hpr * d.head_dim;
    t.slots = i == 2 && !with_v ? 0 : (heads[i] + hpw - 1) / hpw;
    a.out_elems[i] = static_cast<int64_t>(a.tokens) * row;
  }
  for (int i = 0; i < o.rot_dim / 2; ++i)
    a.freq[i] = turn_fraction(o.inv_freq ? o.inv_freq[i] : std::pow(o.rot_base, -2.0 * i / o.rot_dim));
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 152;
  return n;
}

// Blocks of the launch, and in a.parts how many warps share a token: one when
// the tokens alone give every resident warp one, more (up to one per slot of
// heads) when they do not.
unsigned plan_grid(QkArgs& a, int blocks_per_sm, int max_blocks) {
  const int slots = a.t[0].slots + a.t[1].slots + a.t[2].slots;
  const int64_t cap = std::min<int64_t>(static_cast<int64_t>(sm_count()) * blocks_per_sm, max_blocks);
  const int64_t warps = cap * kWarps;
  a.parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(slots, warps / a.tokens)));
  const int64_t items = static_cast<int64_t>(a.tokens) * a.parts;
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(cap, (items + kWarps - 1) / kWarps)));
}

template <int D>
void launch_fwd_kernel(const QkArgs& a, bool inter, bool norm, unsigned grid, cudaStream_t s) {
  if (inter)
    norm ? qk_fwd_kernel<D, true, true><<<grid, kThreads, 0, s>>>(a)
         : qk_fwd_kernel<D, true, false><<<grid, kThreads, 0, s>>>(a);
  else
    norm ? qk_fwd_kernel<D, false, true><<<grid, kThreads, 0, s>>>(a)
         : qk_fwd_kernel<D, false, false><<<grid, kThreads, 0, s>>>(a);
}

template <int D>
void launch_bwd_kernel(const QkArgs& a, bool inter, bool norm, unsigned grid, cudaStream_t s) {
  if (inter)
    norm ? qk_bwd_kernel<D, true, true><<<grid, kThreads, 0, s>>>(a)
         : qk_bwd_kernel<D, true, false><<<grid, kThreads, 0, s>>>(a);
  else
    norm ? qk_bwd_kernel<D, false, true><<<grid, kThreads, 0, s>>>(a)
         : qk_bwd_kernel<D, false, false><<<grid, kThreads, 0, s>>>(a);
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
  const unsigned grid = plan_grid(a, 6, 1 << 20);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  if (d->head_dim == 128)
    launch_fwd_kernel<128>(a, opts->interleaved, opts->norm, grid, s);
  else
    launch_fwd_kernel<64>(a, opts->interleaved, opts->norm, grid, s);
  return check_launch();
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
  const unsigned grid = plan_grid(a, 4, kBwdMaxBlocks);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  if (d->head_dim == 128)
    launch_bwd_kernel<128>(a, opts->interleaved, opts->norm, grid, s);
  else
    launch_bwd_kernel<64>(a, opts->interleaved, opts->norm, grid, s);
  if ((st = check_launch()) != LOONG_OK || !want_dw) return st;
  dw_sum_kernel<<<(2 * d->head_dim + kWarps - 1) / kWarps, kThreads, 0, s>>>(a.dw_part, static_cast<int>(grid),
                                                                             d->head_dim, dwq, dwk);
  return check_launch();
}

}  // extern "C"
