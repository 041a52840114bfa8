// mask_fwd.cu -- the masked (and capped) attention's forward in FUSED mode: every
// query sees a range of keys of its own (mask_attn.cu).
//
// The arithmetic, the score buffers and the softmax are attn_fwd.cu's: S = Q K^T, P =
// exp2(S scale log2e - m) as fp16, O += P V with V's fp16 copy, a row in every lane. What
// differs is the walk and who walks it.  Over documents a tile of queries meets few
// tiles of keys, and what a block needs to start and to end (descriptors, barriers, the
// first copies' latency, the last rows) would take as long as its tiles; so one block an
// SM stays and takes item after item (a query tile of two heads of a kv head, or two
// tiles of an odd group's last head, heavy tiles first) from a counter that the launch
// before cleared.  Its producer has the next item's first keys, and its queries once the
// last Q K^T of this one is done, on their way while the softmax warps still write this
// one's rows.  32 + 8 heads of 128, a block an item and here: 32K tokens in documents of
// about 4K 1.34 and 1.18 ms, of about 256 490 and 422 us, 16K in one with a cap 2.41 and
// 2.24 ms, and where one round of blocks does it nothing.  Items go by their place first,
// all kv heads of all sequences at one, so that the light ones come last; a kv head after
// the other took 1.25 ms, prefixes of 2 x 4K with 16 heads 275 us for 228.
// What bounds an item is the softmax's exponentials (1.70 PFLOP/s at 32K in one piece, as
// without a mask) and, short, its ends: first scores and last rows, some 4 us that nothing
// else of the SM's covers.
// SLOTS = 1: one head's tile an item, where even those do not fill the SMs.
//
// An item walks the key tiles between the first and the last key that any of its rows
// sees (RangeWalk; the launch before summed the ranges up).  A softmax warp some of
// whose rows do not see a whole tile masks it by four words of bits a row.  Scores of
// masked keys are replaced, so what the keys hold does not matter; V, whose rows a
// product adds up with P = 0, is 0 in its copy where it is not finite, and where there
// was such a value (v_amax[1]) the scores of its key become NaN for the rows that see it.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fwd_jobs.h"
#include "internal.h"
#include "ptx.cuh"
#include "softcap.cuh"
#include "v16.cuh"

namespace loong {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kPBias = 7.0f;             // P = exp2(x + 7): attn_fwd.cu
constexpr float kSumBound = 32768.0f;      // 2^(bias + threshold)

template <int D, int SLOTS>
struct MaskFwdCfg {
  static constexpr int NS = D == 128 ? 2 : 4;  // K and V stages
  static constexpr int ATOMS = D / 64;
  static constexpr int ATOM_BYTES = kTile * 128;
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int NSB = fwd_score_buffers(D, SLOTS);
  static constexpr int SEGS = 4;  // items whose description is kept
  static constexpr int NBARS = 2 * SEGS + 1 + 4 * NS + 3 + 3 + 2 + 1 + 1;
  static constexpr int SMEM_BYTES = (2 + 2 * NS) * TILE_BYTES + NBARS * 8 + 1024;
  // a third whole warpgroup (two of its warps idle), whose registers go to the softmax warps
  static constexpr int THREADS = 384, SPLIT_REGS = 168, SOFTMAX_REGS = 216, OTHER_REGS = 72;
  static_assert(256 * SOFTMAX_REGS + 128 * OTHER_REGS <= THREADS * SPLIT_REGS, "register split");
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t S_COL(int buf) { return static_cast<uint32_t>(buf) * 128u; }
  __host__ __device__ static constexpr uint32_t O_COL(int h) { return NSB * 128u + static_cast<uint32_t>(h) * D; }
  static_assert(NSB * 128 + SLOTS * D <= 512 && NSB <= 2 * SLOTS, "tensor memory; see fwd_jobs.h");
};

struct MaskFwdArgs {
  int batch, S, hq, hkv, G, items;
  RingGeom ring;
  Layout lay;
  float scale_log2;
  __nv_bfloat16* o;
  __nv_bfloat16* o_res;  // or null
  float* lse;
  const unsigned* v_amax;
  MaskView mask;
  unsigned* err;
};

// A query tile of two heads, two tiles of one head, or (SLOTS = 1) one of one.
struct Item {
  int b, kvh, bq;
  int q0, q1;        // the slots' first tokens
  int head0, head1;
  int dup;           // slot 1 repeats slot 0
  int kmin, kmax;    // keys that some row sees
  int tiles;         // key tiles; -1: no further item
};

template <int D, int SLOTS, bool CAP>
__global__ void __launch_bounds__(MaskFwdCfg<D, SLOTS>::THREADS, 1)
    mask_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ MaskFwdArgs a) {
  using C = MaskFwdCfg<D, SLOTS>;
  constexpr int NSB = C::NSB, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ Item items[C::SEGS];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * C::TILE_BYTES;
  uint8_t* sV = sK + NS * C::TILE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NS * C::TILE_BYTES);
  uint64_t* item_full = bars;                    // SEGS: an item's description and Q (producer -> all)
  uint64_t* item_empty = item_full + C::SEGS;    // SEGS: the description has been read (all -> producer)
  uint64_t* q_empty = item_empty + C::SEGS;      // an item's Q K^T done (MMA -> producer)
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + NS;
  uint64_t* v_full = k_empty + NS;
  uint64_t* v_empty = v_full + NS;
  uint64_t* s_full = v_empty + NS;  // NSB
  uint64_t* p_full = s_full + 3;    // NSB
  uint64_t* pv_done = p_full + 3;   // SLOTS
  uint64_t* o_full = pv_done + 2;   // an item's O (MMA -> softmax)
  uint64_t* drain = o_full + 1;
  volatile int* abort_flag = &abort_sh;
  const RingGeom& g = a.ring;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SEGS; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], 4 * SLOTS + 1);
    }
    mbar_init(q_empty, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < NSB; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
    }
    for (int h = 0; h < SLOTS; ++h) mbar_init(&pv_done[h], 1);
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base_sh;
  previous_launch_wait();
  if (warp >= 8) regs_dec<C::OTHER_REGS>();
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err));
  };

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    const uint32_t leader = lane == 0;
    auto decode = [&](int idx) {
      Item x;
      // the kv heads of all sequences at one place, then the place before it
      const int heads = a.batch * a.hkv;
      x.kvh = idx % heads % a.hkv;
      x.b = idx % heads / a.hkv;
      int i = idx / heads, pair;
      bool tile_pair = false;
      if constexpr (SLOTS == 1) {
        pair = i % a.G;  // the head
        i /= a.G;
      } else {  // first the pairs of tiles of an odd group's last head, then the pairs of heads
        const int npt = (a.G & 1) ? g.nblocks * ((g.ntile + 1) / 2) : 0, npairs = a.G / 2;
        tile_pair = i < npt;
        if (!tile_pair) i -= npt;
        pair = tile_pair ? 0 : i % npairs;
        if (!tile_pair) i /= npairs;
      }
      const int r = i;
      const int per_block = tile_pair ? (g.ntile + 1) / 2 : g.ntile;
      x.bq = g.nblocks - 1 - r / per_block;
      const int from_last = r % per_block;
      const int qi0 = tile_pair ? 2 * (per_block - 1 - from_last) : g.ntile - 1 - from_last;
      const int qi1 = tile_pair ? min(qi0 + 1, g.ntile - 1) : qi0;
      x.head0 = x.kvh * a.G + (tile_pair ? a.G - 1 : SLOTS * pair);
      x.head1 = SLOTS == 1 || tile_pair ? x.head0 : x.head0 + 1;
      x.dup = tile_pair && qi1 == qi0;
      x.q0 = x.bq * g.blk + qi0 * kTile;
      x.q1 = x.bq * g.blk + qi1 * kTile;
      const int4* t = a.mask.tiles + (static_cast<int64_t>(x.b) * g.nblocks + x.bq) * g.ntile;
      const int4 t0 = t[qi0], t1 = t[qi1];
      x.kmin = min(t0.x, t1.x);
      x.kmax = max(t0.y, t1.y);
      return x;
    };
    int it = 0, seg = 0;
    bool ok = true;
    // what every item begins with: its place among the descriptions, Q's buffer
    auto place = [&]() {
      return (seg < C::SEGS || warp_wait(&item_empty[seg % C::SEGS], (seg / C::SEGS - 1) & 1)) &&
             (seg == 0 || warp_wait(q_empty, (seg - 1) & 1));
    };
    for (int idx = blockIdx.x; idx < a.items && ok;) {
      int next = 0;
      if (leader) next = static_cast<int>(gridDim.x) + atomicAdd(a.mask.counter, 1);  // there by the item's end
      Item x = decode(idx);
      RangeWalk walk;
      walk.init(g, 0, 0, g.cp, x.kmin, x.kmax);
      x.tiles = walk.total();
      uint64_t* full = &item_full[seg % C::SEGS];
      bool begun = false;
      if (x.tiles == 0) {  // no row sees a key: the softmax warps write that
        ok = begun = place();
        if (ok) {
          if (leader) items[seg % C::SEGS] = x;
          mbar_arrive_p(leader, full);
        }
      }
      for (int j = 0; j < x.tiles; ++j, ++it) {
        const int s = it % NS;
        int kvc;
        const int64_t row64 = a.lay.view_row(x.b, walk.k0(), x.kvh, a.hkv, kvc);
        in_bounds(row64 >= 0 && row64 < a.lay.view_rows(a.batch) && kvc >= 0 && kvc < a.lay.view_heads(a.hkv), a.err);
        const int row = static_cast<int>(row64);
        walk.advance();
        if (it >= NS && !warp_wait(&k_empty[s], (it / NS - 1) & 1)) {
          ok = false;
          break;
        }
        mbar_expect_tx_p(leader, &k_full[s], C::TILE_BYTES);
        for (int at = 0; at < C::ATOMS; ++at)
          tma_load_3d_p(leader, sK + s * C::TILE_BYTES + at * C::ATOM_BYTES, &tmK, &k_full[s], at * 64, kvc, row);
        if (j == 0 && (begun = place())) {
          if (leader) items[seg % C::SEGS] = x;
          mbar_expect_tx_p(leader, full, SLOTS * C::TILE_BYTES);
          for (int h = 0; h < SLOTS; ++h) {
            int hc;
            const int64_t qr = a.lay.view_row(x.b, h ? x.q1 : x.q0, h ? x.head1 : x.head0, a.hq, hc);
            // checked build: the tile starts inside the tensor (TMA fills rows past its end with zeros)
            in_bounds(qr >= 0 && qr < a.lay.view_rows(a.batch) && hc >= 0 && hc < a.lay.view_heads(a.hq), a.err);
            for (int at = 0; at < C::ATOMS; ++at)
              tma_load_3d_p(leader, sQ + h * C::TILE_BYTES + at * C::ATOM_BYTES, &tmQ, full, at * 64, hc,
                            static_cast<int>(qr));
          }
        }
        if (!begun || (it >= NS && !warp_wait(&v_empty[s], (it / NS - 1) & 1))) {
          mbar_drain(&k_full[s], (it / NS) & 1, a.err);
          ok = false;
          break;
        }
        mbar_expect_tx_p(leader, &v_full[s], C::TILE_BYTES);
        for (int at = 0; at < C::ATOMS; ++at)
          tma_load_3d_p(leader, sV + s * C::TILE_BYTES + at * C::ATOM_BYTES, &tmV, &v_full[s], at * 64, kvc, row);
      }
      if (begun) ++seg;
      idx = __shfl_sync(0xffffffffu, next, 0);
    }
    if (ok && place()) {
      if (leader) items[seg % C::SEGS].tiles = -1;
      mbar_arrive_p(leader, &item_full[seg % C::SEGS]);
    }
    // every copy lands before the block ends
    for (int s = 0; s < NS; ++s) {
      const int cnt = it > s ? (it - 1 - s) / NS + 1 : 0;
      if (cnt) {
        mbar_drain(&k_full[s], (cnt - 1) & 1, a.err);
        mbar_drain(&v_full[s], (cnt - 1) & 1, a.err);
      }
    }
    if (seg > 0) mbar_drain(&item_full[(seg - 1) % C::SEGS], ((seg - 1) / C::SEGS) & 1, a.err);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_qk = idesc_bf16(128, 128, false, false);
    constexpr uint32_t id_pv = idesc_f16(128, D, false, true);  // P and V in fp16
    const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sK), v_addr = smem_u32(sV);
    unsigned it = 0;  // tiles of the items before
    int buf = 0;      // the next job's score buffer, its phase
    uint32_t par = 0;
    bool ok = true;
    for (unsigned seg = 0; ok; ++seg) {
      if (!warp_wait(&item_full[seg % C::SEGS], (seg / C::SEGS) & 1)) break;
      tc_fence_after();
      const int n = items[seg % C::SEGS].tiles;
      __syncwarp();
      mbar_arrive_p(lane == 0, &item_empty[seg % C::SEGS]);
      if (n < 0) break;
      if (n == 0) {
        mma_commit_w(q_empty);
        continue;
      }
      // Q K^T of the item's job i into buffer sb
      auto issue_qk = [&](int i, int sb) {
        const int h = i % SLOTS;
        const unsigned jt = it + i / SLOTS, st = jt % NS;
        if (h == 0) {
          if (!warp_wait(&k_full[st], (jt / NS) & 1)) return false;
          tc_fence_after();
        }
        const uint64_t qa = sdesc_sw128(q_addr + h * C::TILE_BYTES, 16, 1024);
        const uint64_t kb = sdesc_sw128(k_addr + st * C::TILE_BYTES, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32) >> 4;
          mma_ss_w(tbase + C::S_COL(sb), qa + off, kb + off, id_qk, kk > 0);
        }
        mma_commit_w(&s_full[sb]);
        if (h == SLOTS - 1) mma_commit_w(&k_empty[st]);
        if (i == SLOTS * n - 1) mma_commit_w(q_empty);
        return true;
      };
      for (int i = 0, sb = buf; i < NSB && i < SLOTS * n && ok; ++i) {
        ok = issue_qk(i, sb);
        if (++sb == NSB) sb = 0;
      }
      for (int j = 0; j < n && ok; ++j) {
        const unsigned st = (it + j) % NS;
        if (!(ok = warp_wait(&v_full[st], ((it + j) / NS) & 1))) break;
#pragma unroll
        for (int h = 0; h < SLOTS; ++h) {
          const int i = SLOTS * j + h;
          const int sb = NSB == SLOTS ? h : buf;
          if (!(ok = warp_wait(&p_full[sb], par))) break;
          tc_fence_after();
          const uint64_t vb = sdesc_sw128(v_addr + st * C::TILE_BYTES, C::ATOM_BYTES, 1024);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts_w(tbase + C::O_COL(h), tbase + C::S_COL(sb) + kk * 8, vb + (kk * 2048 >> 4), id_pv,
                     j > 0 || kk > 0);
          mma_commit_w(&pv_done[h]);
          if (h == SLOTS - 1) mma_commit_w(&v_empty[st]);
          if (i + NSB < SLOTS * n && !(ok = issue_qk(i + NSB, sb))) break;  // the buffer that P left
          if (NSB == SLOTS ? h == SLOTS - 1 : ++buf == NSB) {
            buf = 0;
            par ^= 1;
          }
        }
      }
      if (ok) mma_commit_w(o_full);
      it += n;
    }
    mma_commit_w(drain);
    mbar_drain(drain, 0, a.err);
  } else if (warp < 4 * SLOTS) {
    regs_inc<C::SOFTMAX_REGS>();
    // ------------------------------------------------------------ softmax
    const int h = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tO = tbase + t_lane + C::O_COL(h);
    const float sl2 = a.scale_log2;
    const bool v_bad = a.v_amax[1] != 0;
    int buf = h;  // this slot's next score buffer, its phase
    uint32_t par = 0, out = 0, pv = 0;
    bool ok = true;
    for (unsigned seg = 0; ok; ++seg) {
      if (!warp_wait(&item_full[seg % C::SEGS], (seg / C::SEGS) & 1)) break;
      const Item x = items[seg % C::SEGS];
      __syncwarp();
      mbar_arrive_p(lane == 0, &item_empty[seg % C::SEGS]);
      const int n = x.tiles;
      if (n < 0) break;
      const int tok = (h ? x.q1 : x.q0) + row, head = h ? x.head1 : x.head0;
      const bool stored = tok < (x.bq + 1) * g.blk;  // rows past the block see all, they are not stored
      const int64_t qv = stored ? a.lay.vec(x.b, tok, head, a.hq) : 0;  // this row's d-vector in Q / O
      const int64_t lse_i = (static_cast<int64_t>(x.b) * a.hq + head) * a.S + tok;
      // checked build: the row's O and LSE entries lie inside their tensors
      const bool valid = stored && !(h == 1 && x.dup) &&
                         in_bounds(qv >= 0 && qv < static_cast<int64_t>(a.batch) * a.S * a.hq && lse_i >= 0 &&
                                       lse_i < static_cast<int64_t>(a.batch) * a.hq * a.S,
                                   a.err);
      __nv_bfloat16* orow = a.o + qv * D;
      __nv_bfloat16* rrow = a.o_res ? a.o_res + qv * D : nullptr;
      if (n == 0) {
        if (valid) {
          for (int i = 0; i < D / 8; ++i) {
            reinterpret_cast<uint4*>(orow)[i] = make_uint4(0, 0, 0, 0);
            if (rrow) reinterpret_cast<uint4*>(rrow)[i] = make_uint4(0, 0, 0, 0);
          }
          a.lse[lse_i] = -INFINITY;
        }
        continue;
      }
      int2 see = stored ? mask_range(a.mask, x.b, tok, a.S, g.causal) : make_int2(0, 0);
      // a row that sees nothing (padding) goes along as if it saw all, so that its warp does not
      // mask for its sake, and its result is dropped: 2 x 1990 tokens less some padding, every key,
      // 6 + 3 heads of 64, 48.4 -> 30.7 us, with a cap 78 -> 53 (documents without: 1 % slower)
      constexpr int kAll = 0x7fffffff;
      if (see.x >= see.y) see = make_int2(0, kAll);
      RangeWalk walk;
      walk.init(g, 0, 0, g.cp, x.kmin, x.kmax);
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < n; ++j, walk.advance()) {
        const uint32_t tS = tbase + t_lane + C::S_COL(buf);
        if (!(ok = warp_wait(&s_full[buf], par))) break;
        tc_fence_after();
        uint32_t sr[4][32];
        const int k0 = walk.k0(), klen = walk.klen();
        // the columns that this row sees, and whether the warp's rows see all
        const int see_lo = see.x - k0, see_hi = min(see.y - k0, klen);
        const bool masked = __any_sync(0xffffffffu, see_lo > 0 || see_hi < kTile);
        auto seen = [&](int c) { return low_bits(see_hi - c) & ~low_bits(see_lo - c); };
        // the tile's scores, masked columns at -inf, NaN where the key's V is not finite
        auto load_s = [&]() {
#pragma unroll
          for (int cb = 0; cb < 4; ++cb) tmem_ld32(tS + cb * 32, sr[cb]);
          tmem_wait_ld();
          if (v_bad) {
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
              bool bad = false;  // of the lane's key
              const int key = cb * 32 + lane;
              if (key < klen) {
                const uint4* vv = reinterpret_cast<const uint4*>(a.mask.v + a.lay.vec(x.b, k0 + key, x.kvh, a.hkv) * D);
                unsigned m = 0;
                for (int i = 0; i < D / 8; ++i) v16_finite(__ldg(vv + i), m);
                bad = m != 0;
              }
              const unsigned keys = __ballot_sync(0xffffffffu, bad);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (keys >> i & 1) sr[cb][i] = 0x7fffffffu;
            }
          }
          if (masked) {
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
              const uint32_t bits = seen(cb * 32);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(bits >> i & 1)) sr[cb][i] = __float_as_uint(-INFINITY);
            }
          }
        };
        if constexpr (CAP) cap_tile<32>(tS, a.mask.cap, see.y != kAll, masked, seen);
        load_s();
        // P = exp2(s*scale*log2e - ref + bias) for the whole tile; returns this row's sum of
        // P (l carries the factor 2^bias as well)
        uint32_t pk[2][32];
        auto form_p = [&](float ref) {
          const float2 sl2v = make_float2(sl2, sl2), nref = make_float2(kPBias - ref, kPBias - ref);
          float2 lsum = make_float2(0.f, 0.f);
#pragma unroll
          for (int cb = 0; cb < 4; ++cb)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[cb][i]), __uint_as_float(sr[cb][i + 1])),
                                          sl2v, nref);
              const float p0 = fast_exp2(y.x), p1 = fast_exp2(y.y);
              lsum = __fadd2_rn(lsum, make_float2(p0, p1));
              pk[cb >> 1][(cb & 1) * 16 + (i >> 1)] = pack_f16(p0, p1);
            }
          return lsum.x + lsum.y;
        };
        // against the running maximum; where a row's sum reaches the bound (or on NaN), and
        // at first, with the tile's own (attn_fwd.cu)
        bool full = j == 0, over = false;
        if (!full) {
          const float ts = form_p(m_run);
          over = !(ts < kSumBound);
          full = __any_sync(0xffffffffu, over);
          if (!full) l_run += ts;
        }
        if (full) {
          if (j > 0) load_s();  // P of this tile is not stored yet: the scores are still in place
          float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
          for (int cb = 0; cb < 4; ++cb)
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              mx0 = fmax3(mx0, __uint_as_float(sr[cb][i]), __uint_as_float(sr[cb][i + 1]));
              mx1 = fmax3(mx1, __uint_as_float(sr[cb][i + 2]), __uint_as_float(sr[cb][i + 3]));
            }
          const float m_new = fmaxf(m_run, fmaxf(mx0, mx1) * sl2);
          const bool rescale = j > 0 && m_new > m_run + (over ? 0.f : kRescaleThreshold);
          if (j == 0) m_run = m_new;
          if (__any_sync(0xffffffffu, rescale)) {
            // O_h holds the tile before's P V: with as many buffers as slots these scores
            // prove it, else its completion is waited for (fwd_jobs.h)
            if (NSB > SLOTS && !(ok = warp_wait(&pv_done[h], (pv + j - 1) & 1))) break;
            tc_fence_after();
            const float f = rescale ? fast_exp2(m_run - m_new) : 1.f;
            l_run *= f;
#pragma unroll 1
            for (int cb = 0; cb < D / 32; ++cb) {
              uint32_t o32[32];
              tmem_ld32(tO + cb * 32, o32);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o32[i] = __float_as_uint(__uint_as_float(o32[i]) * f);
              tmem_st32(tO + cb * 32, o32);
            }
            if (rescale) m_run = m_new;
          }
          l_run += form_p(m_run == -INFINITY ? 0.f : m_run);
        }
        tmem_st32(tS, pk[0]);
        tmem_st32(tS + 32, pk[1]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_p(lane == 0, &p_full[buf]);
        if (NSB > SLOTS) buf += SLOTS;  // else it stays
        if (NSB == SLOTS || buf >= NSB) {
          if (NSB > SLOTS) buf -= NSB;
          par ^= 1;
        }
      }
      pv += n;
      if (!ok || !(ok = warp_wait(o_full, out++ & 1))) break;
      tc_fence_after();
      // ---------------------------------------------------------- the item's rows
      // l_run and O carry 2^kPBias; O also carries V's 2^-e.  A row without keys has l_run
      // = 0, and one that met a NaN keeps it (in its LSE for the gradient as well)
      const bool any = see.y != kAll && l_run != 0.f;
      const float inv = any ? __int_as_float((127 + v16_shift(*a.v_amax)) << 23) / l_run : 0.f;
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t ov[32];
        tmem_ld32(tO + cb * 32, ov);
        tmem_wait_ld();
        if (valid) {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(ov[e]) * inv;
          if (!any) {  // whatever its Q held
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0.f;
          }
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = pack_bf16(y[v4 * 8 + 2 * u], y[v4 * 8 + 2 * u + 1]);
            reinterpret_cast<uint4*>(orow + cb * 32)[v4] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (rrow) {  // y - bf16(y) is exact in fp32; rounded once more it carries the next 8 bits of O
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
              uint32_t w[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float a0 = y[v4 * 8 + 2 * u], a1 = y[v4 * 8 + 2 * u + 1];
                w[u] = pack_bf16(a0 - __bfloat162float(__float2bfloat16_rn(a0)),
                                 a1 - __bfloat162float(__float2bfloat16_rn(a1)));
              }
              reinterpret_cast<uint4*>(rrow + cb * 32)[v4] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      if (valid) a.lse[lse_i] = any ? (m_run + log2f(l_run) - kPBias) * kLn2 : -INFINITY;
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

template <int D, int SLOTS, bool CAP>
int launch_t(const loong_attn_desc& d, const void* q, const void* k, void* o, float* lse, const FwdScratch& sc,
             const MaskView& mask, cudaStream_t stream) {
  using C = MaskFwdCfg<D, SLOTS>;
  MaskFwdArgs a;
  a.lay = layout_of(d);
  const int64_t rows = a.lay.view_rows(d.batch);
  CUtensorMap mq, mk, mv;
  int st;
  // V is read as its fp16 copy (the map moves 2-byte elements either way)
  if ((st = make_head_tile_map(&mq, q, rows, a.lay.view_heads(d.hq), D)) != LOONG_OK ||
      (st = make_head_tile_map(&mk, k, rows, a.lay.view_heads(d.hkv), D)) != LOONG_OK ||
      (st = make_head_tile_map(&mv, sc.v16, rows, a.lay.view_heads(d.hkv), D)) != LOONG_OK)
    return st;
  a.batch = static_cast<int>(d.batch);
  a.S = static_cast<int>(d.seqlen);
  a.hq = d.hq;
  a.hkv = d.hkv;
  a.G = d.hq / d.hkv;
  a.ring = ring_geom(d);
  const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / std::sqrt(static_cast<float>(D));
  a.scale_log2 = scale * kLog2e;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.o_res = static_cast<__nv_bfloat16*>(sc.o_res);
  a.lse = lse;
  a.v_amax = sc.v_amax;
  a.mask = mask;
  if (!(a.err = device_error_word())) return LOONG_ERR_CUDA;
  const int64_t nt = a.ring.ntile, blocks = a.ring.nblocks;
  const int64_t per_kvh =
      SLOTS == 1 ? blocks * nt * a.G : blocks * (nt * (a.G / 2) + (a.G & 1) * ((nt + 1) / 2));
  const int64_t items = d.batch * d.hkv * per_kvh;
  const int sms = num_sms();
  if (items <= 0 || items > 0x7fffffff - 2 * sms) return LOONG_ERR_INVALID_ARG;
  a.items = static_cast<int>(items);
  constexpr auto kern = mask_fwd_kernel<D, SLOTS, CAP>;
  if ((st = kernel_ready<kern>(C::SMEM_BYTES, C::SPLIT_REGS)) != LOONG_OK) return st;
  record_start(stream);
  st = launch_dependent(kern, dim3(static_cast<unsigned>(std::min<int64_t>(items, sms))), C::THREADS, C::SMEM_BYTES,
                        stream, mq, mk, mv, a);
  record_stop(stream);
  return st;
}

}  // namespace

int launch_mask_fwd(const loong_attn_desc& d, const void* q, const void* k, void* o, float* lse, const FwdScratch& sc,
                    const MaskView& mask, cudaStream_t stream) {
  const RingGeom g = ring_geom(d);
  // One slot where single tiles find an SM each (fwd_jobs.h), and up to two tiles an SM where
  // they are uneven, the light ones filling up: causal rows of 2K and 4K tokens without ranges,
  // two slots and one, 192 tiles of 64 with a cap 47.5 and 36.4 us, 288 48.7 and 48.0, of 128 57.3
  // and 50.0, 256 of 32 tiles a row without one 63 and 52.  Ranges may make every tile short, and the ends of
  // twice the items weigh more (documents of about 128, 192 tiles, 21.5 and 23.5 us).
  const int rounds = !mask.range && d.causal ? 2 : 1;
  const bool one = fwd_one_slot(d.batch * d.hq * g.nblocks * g.ntile, rounds * num_sms());
  auto launch = [&](auto dim, auto slots) {
    constexpr int D = decltype(dim)::value, SLOTS = decltype(slots)::value;
    return mask.cap.inv > 0.f ? launch_t<D, SLOTS, true>(d, q, k, o, lse, sc, mask, stream)
                              : launch_t<D, SLOTS, false>(d, q, k, o, lse, sc, mask, stream);
  };
  using std::integral_constant;
  if (d.head_dim == 128)
    return one ? launch(integral_constant<int, 128>{}, integral_constant<int, 1>{})
               : launch(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  return one ? launch(integral_constant<int, 64>{}, integral_constant<int, 1>{})
             : launch(integral_constant<int, 64>{}, integral_constant<int, 2>{});
}

}  // namespace loong
