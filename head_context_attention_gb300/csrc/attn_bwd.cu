// attn_bwd.cu -- backward ring-step attention on tcgen05 tensor cores.
//
// The gradient of softmax attention, causal or not (plain chain rule; the pages
// give no backward).  One CTA owns one 128-key tile of one kv head and walks every
// (query tile, query head of the group) that attends to it, in the order the
// key/value chunk travels around the ring: step t visits ring rank
// dst(j, t), the rank that holds source j's K/V at step t.  Per iteration:
//   S^T  = K Q^T                 (keys on TMEM lanes, queries on columns)
//   dP^T = V dO^T
//   P^T  = exp2(S^T*scale*log2e - LSE*log2e),  dS^T = P^T * (dP^T - D)
//   dV  += P^T dO                (P^T from tensor memory)
//   dK  += dS^T Q                (dS^T from shared memory, K-major)
//   dQ   = dS K  -> staged in shared memory, added into the fp32 dQ
//                   accumulator by TMA bulk tensor reductions
// dK and dV stay in tensor memory and are folded into fp32 accumulators every
// kFlush iterations; the last partial is added and written as bf16 (FUSED) or
// left in the accumulators (STEPWISE, one launch per step; a step maps ranks to
// sources one to one, so no two CTAs share a tile).  The compute warps form P^T
// as soon as S^T is ready, while dP^T is still on the tensor cores, and drain
// dQ while dK is computed.  Tensors are addressed through a Layout (natural or
// rank-major, ring.cuh); in STEPWISE_COPY modes the K/V tile is read from the
// plane of the rank that holds it at the launch's step (exchange.h), while dK
// and dV go to the owner's rows.
//
// Warp roles: compute warps form four groups of four warps that each cover all
// 128 TMEM lanes (608 threads with the three below); group g
// handles query columns [GW g, GW (g+1)) of S^T/dP^T and head-dim columns
// [GD g, GD (g+1)) of dQ, and folds a share of dV (first half of the groups)
// or dK (second half).  After them, one warp issues TMA loads, one allocates
// TMEM and issues the MMAs, one issues the dQ bulk reductions (so no compute
// warp waits on their completion).
// Tensor memory (512 columns): R0 [0,128) S^T, then P^T as bf16 pairs, each
// group packing its GW queries into the first GW/2 columns of its own GW (the
// groups share lanes, so none may write where another still reads);
// R1 [128,256) dP^T then dQ; dV and dK after that (D columns each).
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "exchange.h"
#include "internal.h"
#include "ptx.cuh"
#include "softcap.cuh"
#include "v16.cuh"

namespace loong {

namespace {

template <int D>
struct BwdCfg {
  static constexpr int NS = D == 64 ? 3 : 2;      // Q / dO pipeline stages (d = 64: 3 measured fastest)
  static constexpr int ATOMS = D / 64;
  static constexpr int ATOM_BYTES = kTile * 128;  // 16 KB
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int DS_BYTES = kTile * kTile * 2;  // dS^T tile, bf16 [keys][queries]
  static constexpr int NBARS = 1 + 4 * NS + 13;
  static constexpr int STAT_BYTES = 2 * kTile * 4;  // LSE*log2e and D of one query tile
  // Tiles first (1024-byte aligned, checked at run time), then the row
  // statistics stages, the barriers, the TMEM base address and the abort
  // flag, then per stage an iteration descriptor and the bias's pieces (with a
  // mask: what a block and its iterations share).
  static constexpr int SMEM_BYTES =
      (2 + 2 * NS) * TILE_BYTES + DS_BYTES + NS * STAT_BYTES + NBARS * 8 + 16 + NS * 144;
  // Compute groups of four warps, each covering all 128 TMEM lanes: group g
  // owns query columns [GW g, GW (g+1)) of S^T / dP^T and head-dim columns
  // [GD g, GD (g+1)) of dQ.  Four groups (four compute warps per scheduler)
  // overlap the compute warps' chain of TMEM loads, exponentials and stores
  // better than two (measured faster at d = 64 and d = 128).
#ifndef LOONG_BWD_GROUPS
#define LOONG_BWD_GROUPS 4
#endif
  static constexpr int GROUPS = LOONG_BWD_GROUPS;
  static constexpr int GW = kTile / GROUPS;  // query columns per group
  static constexpr int GCH = GW / 32;        // 32-column chunks per group
  static constexpr int GD = D / GROUPS;      // dQ head-dim columns per group
  static constexpr int ACC_COLS = 2 * D / GROUPS;  // dV / dK columns each group folds
  static constexpr int CW = 4 * GROUPS;      // compute warps; then producer, MMA, reducer
  static_assert(CW == kBwdComputeWarps, "rows of the bias gradient's parts");
  static constexpr int THREADS = 32 * (CW + 3);
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t R0 = 0, R1 = 128, RV = 256, RK = 256 + D;
  // dQ leaves through TMA bulk reductions of 32-float x 128-row boxes; the
  // boxes are staged in the Q / dO stage of the iteration they belong to.
  static constexpr int DQ_BOXES = D / 32;
  static constexpr int BOX_BYTES = kTile * 128;
  static constexpr int BOXES_PER_STAGE = TILE_BYTES / BOX_BYTES;
  // The groups whose dQ columns land in the dO half of the stage stage them at
  // once (dV(i), the last reader of that half, retired before dQ(i) exists)
  // and the reducer adds that half first; the Q half waits for dK(i).
  // Measured faster at both head dimensions with four compute groups.
  static constexpr bool EARLY_O = true;
  // groups whose dQ columns lie in the Q half of the stage (the rest: the dO half)
  static constexpr int QHALF_GROUPS = BOXES_PER_STAGE * 32 / GD;
  // the iteration descriptors (int4) after the barriers and two words
  static_assert(((2 + 2 * NS) * TILE_BYTES + DS_BYTES + NS * STAT_BYTES + NBARS * 8 + 16) % 16 == 0,
                "descriptor alignment");
};

// dK and dV build up in tensor memory; every kFlush iterations they are added
// into fp32 accumulators in global memory and the tensor-memory sums restart,
// which bounds the length of each tensor-core accumulation chain.
constexpr int kFlush = 512;

struct BwdArgs {
  int batch, S, hq, hkv, G;
  RingGeom ring;
  Layout lay;  // where Q, K, V, dO, dQ (and its accumulator), dK, dV keep (token, head)
  int kv_held;  // K, V are receive buffers (one step per launch): read the holder rank's plane
  int t_begin, t_end;
  float scale, scale_log2;
  // Row statistics, [B*Hq][stat_len] each, block b's rows at b*blk_pad:
  const float* lse2;   // LSE * log2(e); with a bias or a mask its negative
  const float* dstat;  // D = rowsum(dO * O); with a mask its negative
  int blk_pad, stat_len;
  float* dq_acc;      // fp32, the layout of Q
  __nv_bfloat16* dk;  // FUSED outputs
  __nv_bfloat16* dv;
  // fp32 accumulators, the layout of K, zeroed by the launcher; FUSED with a mask: not, the
  // first flush writes them (and where a group's heads are split the last one, the blocks' parts)
  float* dk_acc;
  float* dv_acc;
  BiasView bias;      // BIAS: the bias by distance
  float* dbias_part;  // BIAS: [blocks][compute warps][G][intervals], zeroed
  unsigned* err;
  MaskView mask;      // MASK: the keys that a query sees, the cap
};

constexpr float kLog2e = 1.4426950408889634f;

// BIAS: the scores carry the bias of their distance and the kernel sums dS by
// interval of distances, the gradient of the bias, both per piece of 32 keys by
// 32 queries, a compute warp's share of a tile (see attn_fwd.cu).  A piece
// inside one interval adds its constant to the exponent's offset and its dS sum
// to one number: the warp sums it by shuffles and lane g keeps the running
// sum of the group's head g, written out when the interval changes.  In a piece
// that one boundary crosses, a score and its dS go to one of two constants and
// sums by the column at which its row passes the boundary.  With more
// boundaries, dS is summed along the diagonals and the diagonals' sums are added
// up by interval.  Every warp adds to numbers of its own, so the sums do not depend on
// the order in which blocks run.  The sums fit between dS and the wait for dQ; what
// they cost is instructions: 32 + 8 heads of 128, 16K tokens, 64 buckets up to 8192
// 5.2-5.3 ms (without a bias 4.8; tensor cores 47 %), 2K ragged tokens of 64 111-113 us (96).
struct BwdPiece {
  float lo, hi;  // the bias of the first and the last place
  int code;      // PieceCode; entry 7: the head in its group
  int place;     // entry 7: the place of distance q0 - k0
};

// MASK: every query sees a range of keys, scores may be capped (attn_fwd.cu).  A
// block counts, all threads together, the query tiles some row of which sees one of
// its keys, by the launch before's sums over their rows; the producer then looks 32
// of them up at a time.  In a tile not all of whose rows see all keys, a warp
// turns the ranges of its 32 queries, one in each lane, into bits for its 32 keys and
// transposes the 32 x 32 bits by five exchanges, so that each lane has a word for
// its key's row.  With a cap, dS takes the factor 1 - tanh^2, which P is multiplied
// with once it has been stored for dV, so no further registers are held.
// A product adds masked rows up with a factor 0, so what they hold has to be finite:
// rows of K that are not are cleared in shared memory by the compute warps, rows of Q
// and dO by the producer, in the tiles that the launch before marked.  Instead the
// row's own P is NaN, for those that see it.
// Where key tiles do not fill the SMs, the query heads of a group go to several blocks.
// 32 + 8 heads of 128: 16K tokens in one piece 4.98 ms (K2's rate), capped 5.5; 64K in
// documents of about 8K 14.7 ms.
enum BwdVariant { kBwdPlain, kBwdBias, kBwdMask, kBwdCap };

// The query tiles, in natural order, that see a block's keys [k0, k1), a word of 32
// at a time, and the heads of the group for each.
struct RangeQWalk {
  const int4* tiles;
  const RingGeom* g;
  int k0, k1, last, G, rank;  // rank: the ring rank whose tiles count, -1: all
  int base, hk;
  unsigned live, part;  // of tiles base ..: seen, and not by all rows whole
  int x;                // the tile

  __device__ static bool sees(int4 r, int k0, int k1) { return r.x < k1 && r.y > k0 && r.x < r.y; }
  __device__ void fetch(int lane) {
    const int i = base + lane;
    bool l = false, p = false;
    if (i <= last) {
      const int4 r = tiles[i];
      l = sees(r, k0, k1) && (rank < 0 || block_owner(*g, i / g->ntile) == rank);
      p = !(r.z <= k0 && r.w >= k1) || k1 - k0 < kTile;
    }
    live = __ballot_sync(0xffffffffu, l);
    part = __ballot_sync(0xffffffffu, p);
  }
  // There is a further tile (the caller counts).
  __device__ void settle(int lane) {
    while (live == 0 && base <= last) {
      base += 32;
      fetch(lane);
    }
    x = base + __ffs(live) - 1;
    hk = 0;
  }
  __device__ void advance(int lane) {
    if (++hk < G) return;
    live &= live - 1;
    settle(lane);
  }
  __device__ bool partial() const { return part >> (x - base) & 1; }
};

template <int D, bool STEP, int VARIANT>
__global__ void __launch_bounds__(BwdCfg<D>::THREADS, 1)
    ring_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                    const __grid_constant__ CUtensorMap tmDQ, const BwdArgs a) {
  using C = BwdCfg<D>;
  constexpr bool BIAS = VARIANT == kBwdBias, CAP = VARIANT == kBwdCap, MASK = VARIANT == kBwdMask || CAP;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // uniform over the CTA; the swizzled tiles need it
    if (threadIdx.x == 0) atomicOr(a.err, kErrSmemAlign);
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::TILE_BYTES;
  uint8_t* sQ = sV + C::TILE_BYTES;              // NS stages
  uint8_t* sdO = sQ + C::NS * C::TILE_BYTES;     // NS stages
  uint8_t* sdS = sdO + C::NS * C::TILE_BYTES;    // [2 query atoms][128 keys][128 B]
  float* sStat = reinterpret_cast<float*>(sdS + C::DS_BYTES);  // NS x [LSE2[128], D[128]]
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sStat) + C::NS * C::STAT_BYTES);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;
  uint64_t* q_empty = q_full + C::NS;
  uint64_t* s_full = q_empty + C::NS;   // S^T(i) in R0          (MMA -> warps)
  uint64_t* dp_full = s_full + 1;       // dP^T(i) in R1         (MMA -> warps)
  uint64_t* p_full = dp_full + 1;       // P^T(i) in R0          (warps -> MMA)
  uint64_t* ds_full = p_full + 1;       // dS^T(i) in smem       (warps -> MMA)
  uint64_t* dq_full = ds_full + 1;      // dQ(i) in R1           (MMA -> warps)
  uint64_t* dq_empty = dq_full + 1;     // R1 drained            (warps -> MMA)
  uint64_t* dk_done = dq_empty + 1;     // dK(i) done: Q/dO stage free for staging
  uint64_t* acc_full = dk_done + 1;     // dK/dV ready to flush  (MMA -> warps)
  uint64_t* acc_empty = acc_full + 1;   // dK/dV flushed         (warps -> MMA)
  uint64_t* done_bar = acc_empty + 1;
  uint64_t* drain = done_bar + 1;
  // per stage, so that neither runs a phase ahead of the reducer: a stage is
  // staged into again only after the reducer has read it and it was reloaded
  uint64_t* staged_q = drain + 1;       // NS: dQ(i) columns staged in the Q half (warps -> reducer)
  uint64_t* staged_o = staged_q + C::NS;  // NS: dQ(i) columns staged in the dO half (warps -> reducer)
  // MASK
  uint64_t* k_ready = staged_o + C::NS;  // K's rows are finite (compute warps -> MMA)
  uint64_t* patch = k_ready + 1;         // a stage whose rows the producer looks at first
  uint32_t& tmem_base_sh = *reinterpret_cast<uint32_t*>(bars + C::NBARS);
  int& abort_sh = *(reinterpret_cast<int*>(bars + C::NBARS) + 1);
  volatile int* abort_flag = &abort_sh;
  // Per stage, the iteration the producer loaded into it: view row of the
  // query tile, its view head, its length, and flags (1: the causal diagonal
  // tile, 2: a dQ reduction may start there).  Written before the stage's
  // q_full arrival, so everyone who waited for the stage's data sees it; the
  // compute and reducer warps then need no walk of their own.
  int4* sInfo = reinterpret_cast<int4*>(bars + C::NBARS + 2);
  // BIAS, per stage: piece diagonal i < 7 (queries 32 (i - 3) ahead of the keys);
  // entry 7: the tile's place and head.
  BwdPiece* sBias = reinterpret_cast<BwdPiece*>(sInfo + C::NS);
  static_assert(VARIANT == kBwdPlain || (C::GW == 32 && C::GCH == 1), "a compute warp covers one 32 x 32 piece");
  // MASK: the first query of every stage's tile (NS words), then the block's count of
  // tiles, the first and the last of them, then a byte per row of K that is not finite
  int* sQ0 = reinterpret_cast<int*>(sBias);
  int* sWalk = sQ0 + 4;
  uint8_t* sBadK = reinterpret_cast<uint8_t*>(sQ0 + 8);
  static_assert(C::NS <= 4 && 32 + kTile <= C::NS * 128, "fits the bias's place");

  // ---- work item: (batch, kv head, key tile); early (heavy) key tiles first
  const RingGeom& g = a.ring;
  int idx = blockIdx.x;
  int split = 0;
  if constexpr (MASK) {
    split = idx % a.mask.splits;
    idx /= a.mask.splits;
  }
  const int nkt = g.nblocks * g.ntile;
  // MASK: all kv heads of all sequences at one key tile, so that the light ones come last (a training
  // pass of 16K tokens of 32 + 8 heads of 128 with a cap 8.26 -> 7.84 ms, prefixes of 2 x 4K 790 -> 720 us)
  const int heads = MASK ? a.batch * a.hkv : nkt;
  const int r = MASK ? idx / heads : idx % nkt;
  idx = MASK ? idx % heads : idx / nkt;
  const int kvh = idx % a.hkv;
  const int b = idx / a.hkv;
  const int bk = r / g.ntile;
  const int kt = r % g.ntile;
  const int k0 = bk * g.blk + kt * kTile;
  const int klen = min(kTile, (bk + 1) * g.blk - k0);

  std::conditional_t<MASK, RangeQWalk, QWalk> walk;
  int n;
  if constexpr (MASK) {
    previous_launch_wait();
    const int nq = g.nblocks * g.ntile;
    walk.tiles = a.mask.tiles + static_cast<int64_t>(b) * nq;
    walk.g = &g;
    walk.k0 = k0;
    walk.k1 = k0 + klen;
    walk.G = min(a.mask.per_split, a.G - split * a.mask.per_split);
    walk.rank = STEP ? ring_dst(block_owner(g, bk), a.t_begin, g.inner, g.outer) : -1;
    if (threadIdx.x == 0) {
      sWalk[0] = 0;
      sWalk[1] = nq;
      sWalk[2] = -1;
    }
    __syncthreads();
    int count = 0, first = nq, last = -1;
    for (int i = threadIdx.x; i < nq; i += C::THREADS) {
      if (RangeQWalk::sees(walk.tiles[i], k0, k0 + klen) &&
          (!STEP || block_owner(g, i / g.ntile) == walk.rank)) {
        ++count;
        first = min(first, i);
        last = i;
      }
    }
    count = __reduce_add_sync(0xffffffffu, count);
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if ((threadIdx.x & 31) == 0 && count) {
      atomicAdd(sWalk, count);
      atomicMin(sWalk + 1, first);
      atomicMax(sWalk + 2, last);
    }
    __syncthreads();
    n = sWalk[0] * walk.G;
    walk.base = sWalk[1];
    walk.last = sWalk[2];
    if (n == 0) {
      if constexpr (!STEP) {  // no query sees the keys
        for (int i = threadIdx.x; i < klen * (D / 8); i += C::THREADS) {
          const int64_t kv = a.lay.vec(b, k0 + i / (D / 8), kvh, a.hkv);
          if (!in_bounds(kv >= 0 && kv < static_cast<int64_t>(a.batch) * a.S * a.hkv, a.err)) continue;
          if (a.mask.splits > 1) {
            const int64_t at = (static_cast<int64_t>(a.batch) * a.S * a.hkv * split + kv) * D;
            for (int u = 0; u < 2; ++u) {
              reinterpret_cast<float4*>(a.dk_acc + at)[2 * (i % (D / 8)) + u] = make_float4(0.f, 0.f, 0.f, 0.f);
              reinterpret_cast<float4*>(a.dv_acc + at)[2 * (i % (D / 8)) + u] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
          } else {
            reinterpret_cast<uint4*>(a.dk + kv * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(a.dv + kv * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
          }
        }
      }
      return;
    }
  } else {
    walk.init(g, a.G, bk, kt, a.t_begin, a.t_end);
    n = walk.total();
    if (n == 0) return;
  }
  const int nflush = (n - 1) / kFlush;  // flushes before the final write

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);  // the reducer, once the stage's dQ boxes are read
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_full, C::CW);
    mbar_init(ds_full, C::CW);
    mbar_init(dq_full, 1);
    mbar_init(dq_empty, C::CW);
    mbar_init(dk_done, 1);
    for (int st = 0; st < C::NS; ++st) {
      mbar_init(&staged_q[st], C::EARLY_O ? 4 * C::QHALF_GROUPS : C::CW);
      mbar_init(&staged_o[st], 4 * (C::GROUPS - C::QHALF_GROUPS));
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, C::CW);
    mbar_init(done_bar, 1);
    mbar_init(drain, 1);
    if constexpr (MASK) {
      mbar_init(k_ready, C::CW);
      mbar_init(patch, 1);
    }
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == C::CW + 1) {
    tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == C::CW && lane == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    tma_prefetch_map(&tmO);
    tma_prefetch_map(&tmDQ);
  }
  if constexpr (MASK) {
    if (threadIdx.x < kTile) sBadK[threadIdx.x] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base_sh;

  if (warp == C::CW) {
    // ------------------------------------------------------------ TMA producer
    {  // the whole warp runs the loop; lane 0 issues
      const uint32_t leader = lane == 0;
      auto warp_wait = [&](uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
      };

      mbar_expect_tx_p(leader, kv_full, 2 * C::TILE_BYTES);
      int kvc;
      // the rank that holds this key tile's chunk at the launch's (single) step
      const int holder = ring_dst(block_owner(g, bk), a.t_begin, g.inner, g.outer);
      const int64_t kr64 = a.kv_held ? a.lay.view_row_held(b, k0, kvh, a.hkv, holder, kvc)
                                     : a.lay.view_row(b, k0, kvh, a.hkv, kvc);
      // checked build: tiles start inside their tensors (TMA fills rows past the end with zeros)
      in_bounds(kr64 >= 0 && kr64 < a.lay.view_rows(a.batch) && kvc >= 0 && kvc < a.lay.view_heads(a.hkv), a.err);
      const int kr = static_cast<int>(kr64);
      for (int at = 0; at < C::ATOMS; ++at) {
        tma_load_3d_p(leader, sK + at * C::ATOM_BYTES, &tmK, kv_full, at * 64, kvc, kr);
        tma_load_3d_p(leader, sV + at * C::ATOM_BYTES, &tmV, kv_full, at * 64, kvc, kr);
      }
      int issued = 0;
      // lanes 0-6: a piece diagonal of the tile the walk stands at, lane 7: its place
      BwdPiece piece;
      auto look_up = [&]() {
        if constexpr (BIAS) {
          const int i0 = a.bias.off + walk.q0() - k0;
          if (lane < 7) {
            const int at = i0 + 32 * (lane - 3);
            // independent loads, waited for in the next trip
            piece.code = a.bias.piece[at];
            const float* l = a.bias.lut + (kvh * a.G + walk.head) * a.bias.len + at;
            piece.lo = l[-31];
            piece.hi = l[31];
          } else {
            piece.code = walk.head;
            piece.place = i0;
          }
        }
      };
      look_up();
      // MASK: whether the tile the walk stands at has rows to clear (for the next trip)
      unsigned marked = 0, patches = 0;
      const int head0 = kvh * a.G + (MASK ? split * a.mask.per_split : 0);
      auto look_up_mark = [&]() {
        if constexpr (MASK)
          marked = a.mask.bad[(static_cast<int64_t>(b) * a.hq + head0 + walk.hk) * g.nblocks * g.ntile + walk.x];
      };
      if constexpr (MASK) {
        walk.fetch(lane);
        walk.settle(lane);
      }
      look_up_mark();
      for (int i = 0; i < n; ++i) {
        const int s = i % C::NS;
        const int u = i / C::NS;
        // coordinates first, off the wait's critical path
        int head, q0, qlen, bq, qi, flags;
        if constexpr (MASK) {
          head = head0 + walk.hk;
          bq = walk.x / g.ntile;
          qi = walk.x - bq * g.ntile;
          q0 = bq * g.blk + qi * kTile;
          qlen = min(kTile, (bq + 1) * g.blk - q0);
          flags = walk.partial() || qlen < kTile ? 4 : 0;
        } else {
          head = kvh * a.G + walk.head;
          bq = walk.bq;
          qi = walk.qi;
          q0 = walk.q0();
          qlen = walk.qlen();
          flags = walk.diag() ? 1 : 0;
        }
        int hc;
        const int64_t qrow64 = a.lay.view_row(b, q0, head, a.hq, hc);
        in_bounds(qrow64 >= 0 && qrow64 < a.lay.view_rows(a.batch) && hc >= 0 && hc < a.lay.view_heads(a.hq), a.err);
        const int qrow = static_cast<int>(qrow64);
        // checked build: a reduction never starts outside the accumulator (skipped if it would)
        const bool red_ok =
            in_bounds(qrow64 >= 0 && qrow64 < a.lay.view_rows(a.batch) && hc >= 0 && hc < a.lay.view_heads(a.hq), a.err);
        if (i >= C::NS && !warp_wait(&q_empty[s], (u - 1) & 1, abort_flag, a.err)) break;
        if (leader) sInfo[s] = make_int4(qrow, hc, qlen, flags | (red_ok ? 2 : 0));
        if (MASK && leader) sQ0[s] = q0;
        // a stage with rows to clear arrives on `patch` first
        uint64_t* full = MASK && marked ? patch : &q_full[s];
        if constexpr (BIAS) {
          if (lane < 8) sBias[s * 8 + lane] = piece;
          __syncwarp();
        }
        mbar_expect_tx_p(leader, full, 2 * C::TILE_BYTES + C::STAT_BYTES);
        for (int at = 0; at < C::ATOMS; ++at) {
          tma_load_3d_p(leader, sQ + s * C::TILE_BYTES + at * C::ATOM_BYTES, &tmQ, full, at * 64, hc, qrow);
          tma_load_3d_p(leader, sdO + s * C::TILE_BYTES + at * C::ATOM_BYTES, &tmO, full, at * 64, hc, qrow);
        }
        // this tile's row statistics: 16-byte aligned and in bounds by construction
        int64_t srow = (static_cast<int64_t>(b) * a.hq + head) * a.stat_len + bq * a.blk_pad + qi * kTile;
        // checked build: a plain bulk copy must stay inside the statistics rows
        // (else it reads row 0 instead, keeping the barrier's byte count)
        if (!in_bounds(srow >= 0 && srow % 4 == 0 &&
                           srow + kTile <= (static_cast<int64_t>(b) * a.hq + head + 1) * a.stat_len,
                       a.err))
          srow = 0;
        bulk_load_p(leader, sStat + s * (2 * kTile), a.lse2 + srow, kTile * 4, full);
        bulk_load_p(leader, sStat + s * (2 * kTile) + kTile, a.dstat + srow, kTile * 4, full);
        if constexpr (MASK) {
          if (marked) {  // uniform over the warp
            if (!warp_wait(patch, patches++ & 1, abort_flag, a.err)) {
              mbar_drain(patch, (patches - 1) & 1, a.err);
              break;
            }
            const float* lse_row = sStat + s * (2 * kTile);
            const int line = lane & (D / 8 - 1);  // 16 bytes of a row of Q; D = 128: the upper lanes' of dO
#pragma unroll 1
            for (int r0 = 0; r0 < kTile; r0 += 32) {
              unsigned m = __ballot_sync(0xffffffffu, !(fabsf(lse_row[r0 + lane]) < INFINITY) || r0 + lane >= qlen);
              for (; m; m &= m - 1) {
                const int at =
                    s * C::TILE_BYTES + (line >> 3) * C::ATOM_BYTES + (r0 + __ffs(m) - 1) * 128 + (line & 7) * 16;
                if (D == 64 || lane < 16) *reinterpret_cast<uint4*>(sQ + at) = make_uint4(0, 0, 0, 0);
                if (D == 64 || lane >= 16) *reinterpret_cast<uint4*>(sdO + at) = make_uint4(0, 0, 0, 0);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_p(leader, &q_full[s]);
          }
        }
        ++issued;
        if constexpr (MASK)
          walk.advance(lane);
        else
          walk.advance();
        if (i + 1 < n) {  // used in the next trip
          look_up();
          look_up_mark();
        }
      }
      mbar_drain(kv_full, 0, a.err);
      for (int s = 0; s < C::NS; ++s) {
        const int cnt = issued > s ? (issued - 1 - s) / C::NS + 1 : 0;
        if (cnt) mbar_drain(&q_full[s], (cnt - 1) & 1, a.err);
      }
    }
  } else if (warp == C::CW + 1) {
    // ------------------------------------------------------------ MMA issuer
    {  // the whole warp runs the loop; one elected lane issues
      auto warp_wait = [&](uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
      };
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);  // S^T, dP^T: both K-major
      constexpr uint32_t id_dkv = idesc_bf16(128, D, false, true);   // dV, dK: B MN-major
      constexpr uint32_t id_dq = idesc_bf16(128, D, true, true);     // dQ: A and B MN-major
      const uint32_t k_addr = smem_u32(sK), v_addr = smem_u32(sV), q_addr = smem_u32(sQ),
                     o_addr = smem_u32(sdO), ds_addr = smem_u32(sdS);
      // Descriptors built once: an operand's descriptor at byte offset `off`
      // is its base descriptor plus off / 16 (the 14-bit address field cannot
      // carry: every shared-memory address is below 256 KB).
      auto d16 = [](uint32_t a) { return sdesc_sw128(a, 16, 1024); };           // K-major operands
      auto dmn = [](uint32_t a) { return sdesc_sw128(a, C::ATOM_BYTES, 1024); };  // MN-major operands
      const uint64_t k16 = d16(k_addr), kmn = dmn(k_addr), v16 = d16(v_addr), ds16 = d16(ds_addr),
                     dsmn = dmn(ds_addr);
      // X^T[keys x queries] = A[keys x d] * B[queries x d]^T, both K-major
      auto mm_s = [&](uint32_t dst, uint64_t a_desc, uint64_t b_desc) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32) >> 4;
          mma_ss_w(tbase + dst, a_desc + off, b_desc + off, id_s, kk > 0);
        }
      };
      bool ok = warp_wait(kv_full, 0, abort_flag, a.err) && (!MASK || warp_wait(k_ready, 0, abort_flag, a.err)) &&
                warp_wait(&q_full[0], 0, abort_flag, a.err);
      if (ok) {
        tc_fence_after();
        mm_s(C::R0, k16, d16(q_addr));
        mma_commit_w(s_full);
        mm_s(C::R1, v16, d16(o_addr));
        mma_commit_w(dp_full);
        bool fresh = true;  // next dV / dK start a new tensor-memory sum
        for (int i = 0; i < n; ++i) {
          const int s = i % C::NS;
          const uint64_t qmn = dmn(q_addr + s * C::TILE_BYTES), omn = dmn(o_addr + s * C::TILE_BYTES);
          if (!warp_wait(p_full, i & 1, abort_flag, a.err)) break;
          tc_fence_after();
          // dV += P^T dO: A = P^T (TMEM: each group's bf16 pairs in the first
          // columns of its own GW, 8 columns per 16 queries), B = dO MN-major
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts_w(tbase + C::RV,
                   tbase + C::R0 + (kk * 16 / C::GW) * C::GW + ((kk * 16 % C::GW) / 32) * 16 + (kk & 1) * 8,
                   omn + (kk * 2048 >> 4), id_dkv, !fresh || kk > 0);
          if (!warp_wait(ds_full, i & 1, abort_flag, a.err)) break;
          tc_fence_after();
          // dQ = dS K: A = dS (dS^T read MN-major), B = K MN-major; first, so
          // the drain of dQ overlaps the dK product
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ss_w(tbase + C::R1, dsmn + (kk * 2048 >> 4), kmn + (kk * 2048 >> 4), id_dq, kk > 0);
          mma_commit_w(dq_full);
          // dK += dS^T Q: A = dS^T K-major (queries contiguous), B = Q MN-major
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32) >> 4;
            mma_ss_w(tbase + C::RK, ds16 + off, qmn + (kk * 2048 >> 4), id_dkv, !fresh || kk > 0);
          }
          mma_commit_w(dk_done);
          fresh = false;
          const bool flush = i + 1 < n && (i + 1) % kFlush == 0;
          if (flush) {
            mma_commit_w(acc_full);
            fresh = true;
          }
          if (i + 1 < n) {
            const int s1 = (i + 1) % C::NS;
            if (!warp_wait(&q_full[s1], ((i + 1) / C::NS) & 1, abort_flag, a.err)) break;
            tc_fence_after();
            mm_s(C::R0, k16, d16(q_addr + s1 * C::TILE_BYTES));  // R0's P^T was read by dV(i), issued earlier
            mma_commit_w(s_full);
            if (!warp_wait(dq_empty, i & 1, abort_flag, a.err)) break;
            tc_fence_after();
            mm_s(C::R1, v16, d16(o_addr + s1 * C::TILE_BYTES));
            mma_commit_w(dp_full);
            if (flush) {
              if (!warp_wait(acc_empty, ((i + 1) / kFlush - 1) & 1, abort_flag, a.err)) break;
              tc_fence_after();
            }
          }
        }
        mma_commit_w(done_bar);
      }
      mma_commit_w(drain);
      mbar_drain(drain, 0, a.err);
    }
  } else if (warp == C::CW + 2) {
    // ------------------------------------------------------------ dQ reducer
    // Adds each staged dQ tile into the fp32 accumulator with TMA bulk tensor
    // reductions and hands the stage back to the producer once it is read.
    {  // the whole warp runs the loop; lane 0 issues
      const uint32_t leader = lane == 0;
      auto warp_wait = [&](uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
      };

      for (int i = 0; i < n; ++i) {
        const int s = i % C::NS;
        if constexpr (C::EARLY_O) {
          // the dO half first: it is staged without waiting for dK(i)
          if (!warp_wait(&staged_o[s], (i / C::NS) & 1, abort_flag, a.err)) break;
          const int4 info = sInfo[s];  // the producer wrote it before the stage's data
          const int qrow = info.x, hc = info.y;
          const bool red_ok = info.w & 2;
#pragma unroll
          for (int box = C::BOXES_PER_STAGE; box < C::DQ_BOXES; ++box)
            if (red_ok)
              tma_reduce_add_3d_p(leader, &tmDQ, sdO + s * C::TILE_BYTES + (box - C::BOXES_PER_STAGE) * C::BOX_BYTES,
                                box * 32, hc, qrow);
        }
        if (!warp_wait(&staged_q[s], (i / C::NS) & 1, abort_flag, a.err)) break;
        const int4 info = sInfo[s];
        const int qrow = info.x, hc = info.y;
        const bool red_ok = info.w & 2;
#pragma unroll
        for (int box = 0; box < (C::EARLY_O ? C::BOXES_PER_STAGE : C::DQ_BOXES); ++box) {
          const uint8_t* base = box < C::BOXES_PER_STAGE
                                    ? sQ + s * C::TILE_BYTES + box * C::BOX_BYTES
                                    : sdO + s * C::TILE_BYTES + (box - C::BOXES_PER_STAGE) * C::BOX_BYTES;
          if (red_ok) tma_reduce_add_3d_p(leader, &tmDQ, base, box * 32, hc, qrow);
        }
        bulk_commit_group_p(leader);
        bulk_wait_read_all_p(leader);
        mbar_arrive_p(leader, &q_empty[s]);
      }
      // the reductions must land before the kernel ends
      bulk_wait_all_p(leader);
    }
  } else {
    // ------------------------------------------------------------ compute warps
    const int grp = warp >> 2;  // query columns [GW grp, GW grp + GW)
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // key row in the pass, query row in the dQ drain
    const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
    // checked build: this key row's dK / dV / accumulator rows lie inside their tensors
    const bool key_ok = row < klen && in_bounds(a.lay.vec(b, k0 + row, kvh, a.hkv) >= 0 &&
                                                    a.lay.vec(b, k0 + row, kvh, a.hkv) <
                                                        static_cast<int64_t>(a.batch) * a.S * a.hkv,
                                                a.err);
    const int64_t krow = a.lay.vec(b, k0 + row, kvh, a.hkv);  // this key row's d-vector in K / dK / dV
    // the first half of the groups own dV, the second dK (keys on lanes), ACC_COLS columns each
    const bool owns_dv = grp < C::GROUPS / 2;
    const int acc_part = C::GROUPS == 2 ? 0 : (owns_dv ? grp : grp - C::GROUPS / 2) * C::ACC_COLS;
    const uint32_t acc_col = (owns_dv ? C::RV : C::RK) + acc_part;
    const int64_t slice = MASK ? static_cast<int64_t>(a.batch) * a.S * a.hkv * split : 0;
    float* acc_glob = (owns_dv ? a.dv_acc : a.dk_acc) + (slice + krow) * D + acc_part;
    const float acc_mul = owns_dv ? 1.f : a.scale;
    bool ok = true;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err));
    };
    // BIAS: this warp's sums of dS, [G][intervals]; lane g keeps the running sum
    // of head 32 sum_block + g in interval sum_ivl
    float* part = BIAS ? a.dbias_part + (static_cast<int64_t>(blockIdx.x) * C::CW + warp) * a.G * a.bias.intervals
                       : nullptr;
    float run_sum = 0.f;
    int sum_ivl = -1, sum_block = 0;
    auto flush_sum = [&]() {
      if (sum_ivl >= 0 && sum_block * 32 + lane < a.G)
        atomicAdd(part + (sum_block * 32 + lane) * a.bias.intervals + sum_ivl, run_sum);
      run_sum = 0.f;
    };
    // MASK: clear the rows of K that are not finite; four threads look at a row
    bool key_bad = false;
    if constexpr (MASK) {
      ok = warp_wait(kv_full, 0);
      constexpr int V = D / 8 / C::GROUPS;  // 16-byte parts of a thread
      uint8_t* line = sK + (grp * V / 8) * C::ATOM_BYTES + row * 128 + (grp * V % 8) * 16;
      unsigned m = 0;
      if (ok) {
#pragma unroll
        for (int u = 0; u < V; ++u) v16_finite(*reinterpret_cast<const uint4*>(line + u * 16), m);
      }
      if (m) sBadK[row] = 1;
      asm volatile("bar.sync 1, %0;" ::"n"(C::CW * 32) : "memory");
      key_bad = sBadK[row];
      if (key_bad) {
#pragma unroll
        for (int u = 0; u < V; ++u) *reinterpret_cast<uint4*>(line + u * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      mbar_arrive_p(lane == 0, k_ready);
    }
    for (int i = 0; i < n && ok; ++i) {
      // row statistics of this tile, staged by the producer with Q and dO
      const float* lse_row = sStat + (i % C::NS) * (2 * kTile);
      const float* d_row = lse_row + kTile;
      // BIAS: this warp's piece
      float tile_b = 0.f;
      int kind = kPieceConst;
      const BwdPiece* piece = nullptr;
      // ---- P^T = exp2(S^T * scale * log2e - LSE * log2e), two 32-query chunks
      if (!warp_wait(s_full, i & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // S^T(i) read Q(i): the stage's descriptor is in place
      const int4 info = sInfo[i % C::NS];
      const int qlen = info.z;
      if constexpr (BIAS) {
        piece = sBias + (i % C::NS) * 8 + grp - quarter + 3;
        kind = PieceCode::kind(piece->code);
        if (kind == kPieceConst) tile_b = piece->lo * a.scale_log2;
      }
      const bool dg = info.w & 1;
      float pv[C::GCH][32];
      {
        uint32_t sv[C::GCH][32];
#pragma unroll
        for (int ch = 0; ch < C::GCH; ++ch) tmem_ld32(tbase + t_lane + C::R0 + grp * C::GW + ch * 32, sv[ch]);
        tmem_wait_ld();
#pragma unroll
        for (int ch = 0; ch < C::GCH; ++ch)
#pragma unroll
          for (int e = 0; e < 32; ++e) pv[ch][e] = __uint_as_float(sv[ch][e]);
      }
      // kPieceStep: the columns (queries) past the boundary for this row
      auto past_step = [&]() {
        const int t = lane - PieceCode::step(piece->code);
        return t > 31 ? 0u : 0xffffffffu << max(t, 0);
      };
      if constexpr (BIAS) {
        if (kind == kPieceStep) {
          const float lo = piece->lo, hi = piece->hi;
          const uint32_t past = past_step();
#pragma unroll
          for (int e = 0; e < 32; ++e) pv[0][e] += past >> e & 1 ? hi : lo;
        } else if (kind == kPieceMixed) {
          const BwdPiece& place = sBias[(i % C::NS) * 8 + 7];
          const float* lp = a.bias.lut + static_cast<int64_t>(kvh * a.G + place.code) * a.bias.len + place.place +
                            32 * (grp - quarter) - lane;
#pragma unroll
          for (int e = 0; e < 32; ++e) pv[0][e] += __ldg(lp + e);
        }
      }
      // P^T before masking: with a bias in pairs, the statistics hold -LSE
      auto form_p = [&](float s0, float s1, float l0, float l1, float& p0, float& p1) {
        if constexpr (BIAS) {
          const float2 x = __ffma2_rn(make_float2(s0, s1), make_float2(a.scale_log2, a.scale_log2),
                                      __fadd2_rn(make_float2(l0, l1), make_float2(tile_b, tile_b)));
          p0 = fast_exp2(x.x);
          p1 = fast_exp2(x.y);
        } else {
          p0 = fast_exp2(fmaf(s0, a.scale_log2, -l0));
          p1 = fast_exp2(fmaf(s1, a.scale_log2, -l1));
        }
      };
      // Query columns c with lo <= c < hi are live for this key row (causal
      // diagonal, ragged query tile, key row past the block).  Interior tiles
      // have every column live and skip the per-element mask.
      const int lo = dg ? row : 0;
      const int hi = key_ok ? qlen : 0;
      const bool unmasked = MASK ? !(info.w & 4) : __all_sync(0xffffffffu, lo == 0 && hi == kTile);
      // MASK: the queries of the warp's columns that see this lane's key
      unsigned seen = 0xffffffffu;
      if constexpr (MASK) {
        if (!unmasked) {
          const int c = grp * 32 + lane, t = sQ0[i % C::NS] + c;
          const int2 r = c < qlen ? mask_range(a.mask, b, t, a.S, g.causal) : make_int2(0, 0);
          const int kq = k0 + quarter * 32;
          seen = transpose_bits(low_bits(min(r.y - kq, klen - quarter * 32)) & ~low_bits(r.x - kq), lane);
        }
        if constexpr (CAP) {
          uint32_t sv[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[e] = __float_as_uint(pv[0][e]);
          if (!unmasked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen >> e & 1)) sv[e] = 0;
          }
          cap_scores(sv, a.mask.cap);
#pragma unroll
          for (int e = 0; e < 32; ++e) pv[0][e] = __uint_as_float(sv[e]);
        }
        if (key_bad) {
#pragma unroll
          for (int e = 0; e < 32; ++e) pv[0][e] = __int_as_float(0x7fffffff);
        }
      }
#pragma unroll
      for (int ch = 0; ch < C::GCH; ++ch) {
        const int cbase = grp * C::GW + ch * 32;  // first query column of the chunk
        uint32_t pk[16];
        if constexpr (MASK) {
          // in pairs; the statistics hold -LSE and -D.  After P has been packed for dV it
          // takes the cap's derivative, 1 - (inv s)^2 of the capped score s, for dS.
          const float inv2 = -a.mask.cap.inv * a.mask.cap.inv;
          const float2 sl2 = make_float2(a.scale_log2, a.scale_log2), i2 = make_float2(inv2, inv2),
                       one = make_float2(1.f, 1.f);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(lse_row + cbase + e);
            const float2 lv[2] = {make_float2(l4.x, l4.y), make_float2(l4.z, l4.w)};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int c = e + 2 * u;
              const float2 s = make_float2(pv[0][c], pv[0][c + 1]);
              const float2 x = __ffma2_rn(s, sl2, lv[u]);
              float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              if (!unmasked) {
                p.x = seen >> c & 1 ? p.x : 0.f;
                p.y = seen >> (c + 1) & 1 ? p.y : 0.f;
              }
              pk[c / 2] = pack_bf16(p.x, p.y);
              if constexpr (CAP) {
                const float2 q = __fmul2_rn(p, __ffma2_rn(__fmul2_rn(s, i2), s, one));
                // a masked score may be NaN
                p = unmasked ? q : make_float2(p.x != 0.f ? q.x : 0.f, p.y != 0.f ? q.y : 0.f);
              }
              pv[0][c] = p.x;
              pv[0][c + 1] = p.y;
            }
          }
        } else if (unmasked) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            // the same query indices in every lane: broadcast shared-memory reads
            const float4 l4 = *reinterpret_cast<const float4*>(lse_row + cbase + e);
            form_p(pv[ch][e], pv[ch][e + 1], l4.x, l4.y, pv[ch][e], pv[ch][e + 1]);
            form_p(pv[ch][e + 2], pv[ch][e + 3], l4.z, l4.w, pv[ch][e + 2], pv[ch][e + 3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(lse_row + cbase + e);
            const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
              const int c = cbase + e + u;
              // masked columns may hold statistics of other rows or padding: select
              float x, y;
              form_p(pv[ch][e + u], pv[ch][e + u + 1], lv[u], lv[u + 1], x, y);
              pv[ch][e + u] = (c >= lo && c < hi) ? x : 0.f;
              pv[ch][e + u + 1] = (c + 1 >= lo && c + 1 < hi) ? y : 0.f;
            }
          }
        }
        if constexpr (!MASK) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) pk[e / 2] = pack_bf16(pv[ch][e], pv[ch][e + 1]);
        }
        // P^T (bf16 pairs) into this group's own columns of R0,
        // [GW grp + 16 ch, +16): already read by this group, never read by another.
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
            "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(tbase + t_lane + C::R0 + grp * C::GW + ch * 16),
            "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]),
            "r"(pk[8]), "r"(pk[9]), "r"(pk[10]), "r"(pk[11]), "r"(pk[12]), "r"(pk[13]), "r"(pk[14]), "r"(pk[15])
            : "memory");
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      mbar_arrive_p(lane == 0, p_full);

      // ---- dS^T = P^T * (dP^T - D) into shared memory
      if (!warp_wait(dp_full, i & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float2 ds_sum[2] = {};  // BIAS: this row's sum of dS
      uint32_t dpv2[C::GCH][32];
#pragma unroll
      for (int ch = 0; ch < C::GCH; ++ch) tmem_ld32(tbase + t_lane + C::R1 + grp * C::GW + ch * 32, dpv2[ch]);
      tmem_wait_ld();
#pragma unroll
      for (int ch = 0; ch < C::GCH; ++ch) {
        const int cbase = grp * C::GW + ch * 32;
        const uint32_t(&dpv)[32] = dpv2[ch];
        uint32_t dsk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d4 = *reinterpret_cast<const float4*>(d_row + cbase + e);
          const float dv4[4] = {d4.x, d4.y, d4.z, d4.w};
          float ds[4];
          if constexpr (MASK) {
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
              const float2 p = make_float2(pv[0][e + u], pv[0][e + u + 1]);
              const float2 x = __fmul2_rn(
                  p, __fadd2_rn(make_float2(__uint_as_float(dpv[e + u]), __uint_as_float(dpv[e + u + 1])),
                                make_float2(dv4[u], dv4[u + 1])));
              ds[u] = unmasked || p.x != 0.f ? x.x : 0.f;
              ds[u + 1] = unmasked || p.y != 0.f ? x.y : 0.f;
            }
          }
#pragma unroll
          for (int u = 0; u < (MASK ? 0 : 4); ++u) {
            const float p = pv[ch][e + u];
            const float x = p * (__uint_as_float(dpv[e + u]) - dv4[u]);
            // masked columns: p is 0 and D may be another row's or padding
            ds[u] = unmasked ? x : (p != 0.f ? x : 0.f);
            if constexpr (BIAS) pv[ch][e + u] = ds[u];  // kept for the bias gradient
          }
          if constexpr (BIAS) {
            ds_sum[0] = __fadd2_rn(ds_sum[0], make_float2(ds[0], ds[1]));
            ds_sum[1] = __fadd2_rn(ds_sum[1], make_float2(ds[2], ds[3]));
          }
          dsk[e / 2] = pack_bf16(ds[0], ds[1]);
          dsk[e / 2 + 1] = pack_bf16(ds[2], ds[3]);
        }
        // dS^T row `row`, queries [cbase, cbase+32): 4 of the 8 16-byte units of
        // the row's 128-byte line in query atom cbase / 64, 128-byte swizzled
        // (written so that GW = 64 folds to constants).
        uint8_t* line = sdS + (grp * C::GW / 64) * C::ATOM_BYTES + row * 128;
#pragma unroll
        for (int uu = 0; uu < 4; ++uu) {
          const int unit = (grp * C::GW % 64) / 8 + ch * 4 + uu;
          uint4 w;
          w.x = dsk[uu * 4 + 0];
          w.y = dsk[uu * 4 + 1];
          w.z = dsk[uu * 4 + 2];
          w.w = dsk[uu * 4 + 3];
          *reinterpret_cast<uint4*>(line + ((unit ^ (row & 7)) << 4)) = w;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      mbar_arrive_p(lane == 0, ds_full);

      // ---- the bias gradient's sums of dS, while dQ is computed
      if constexpr (BIAS) {
        const BwdPiece& place = sBias[(i % C::NS) * 8 + 7];
        const int head = place.code, ivl = PieceCode::interval(piece->code);
        auto warp_sum = [](float x) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          return x;
        };
        if (kind == kPieceConst) {
          if (ivl != sum_ivl || (head >> 5) != sum_block) {
            flush_sum();
            sum_ivl = ivl;
            sum_block = head >> 5;
          }
          const float s = warp_sum((ds_sum[0].x + ds_sum[0].y) + (ds_sum[1].x + ds_sum[1].y));
          if (lane == (head & 31)) run_sum += s;
        } else if (kind == kPieceStep) {
          const uint32_t past = past_step();
          float s2[2] = {}, p2[2] = {};
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (past >> e & 1)
              p2[e & 1] += pv[0][e];
            else
              s2[e & 1] += pv[0][e];
          }
          const float before = warp_sum(s2[0] + s2[1]), after = warp_sum(p2[0] + p2[1]);
          if (lane < 2) atomicAdd(part + head * a.bias.intervals + ivl + lane, lane ? after : before);
        } else {
          float* ph = part + head * a.bias.intervals;
          // lane l, column c: distance at place base + c - l
          const uint8_t* at = a.bias.interval + place.place + 32 * (grp - quarter);
          // The diagonals' sums, one column after the other: a distance's sum moves one
          // lane up with every column, a chain of shuffles that fits the wait for dQ.
          // (Columns joined pairwise in five levels of independent shuffles: twice the
          // code and no faster, 2K ragged tokens of 64 112.4 us for 110.9, 16K of 128
          // 5.15 ms for 5.16.)
          int ln = lane;
          asm volatile("" : "+r"(ln));  // keeps the lanes' tests from being formed, and held, outside the loop
          float acc = 0.f, fin = 0.f;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            acc += pv[0][c];
            const float done = __shfl_sync(0xffffffffu, acc, 31);  // complete: distance base + c - 31
            if (ln == c) fin = done;
            acc = __shfl_up_sync(0xffffffffu, acc, 1);
            if (ln == 0) acc = 0.f;
          }
          // every interval is a run of lanes
          auto add_runs = [&](float v, int id) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const float v2 = __shfl_down_sync(0xffffffffu, v, o);
              const int id2 = __shfl_down_sync(0xffffffffu, id, o);
              if (ln + o < 32 && id2 == id) v += v2;
            }
            const int before = __shfl_up_sync(0xffffffffu, id, 1);
            if (ln == 0 || before != id) atomicAdd(ph + id, v);
          };
          add_runs(acc, at[32 - max(ln, 1)]);  // nothing in lane 0
          add_runs(fin, at[ln - 31]);
        }
      }

      // ---- drain dQ (queries on lanes): TMEM -> registers, R1 released, then
      // staged (fp32, 128-byte swizzled boxes of 32 columns) into this
      // iteration's Q / dO stage once dK(i) no longer reads it, and added into
      // the fp32 accumulator by TMA bulk reductions.
      if (!warp_wait(dq_full, i & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      {
        const bool q_ok = row < qlen;
        // this group's GD columns of dQ in runs of RUN (one TMEM load each)
        constexpr int RUN = C::GD >= 32 ? 32 : 16;
        constexpr int NR = C::GD / RUN;
        uint32_t qv[NR][RUN];
#pragma unroll
        for (int cb = 0; cb < NR; ++cb) {
          if constexpr (RUN == 32)
            tmem_ld32(tbase + t_lane + C::R1 + grp * C::GD + cb * RUN, qv[cb]);
          else
            tmem_ld16(tbase + t_lane + C::R1 + grp * C::GD + cb * RUN, qv[cb]);
        }
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_p(lane == 0, dq_empty);
        // groups staging into the Q half wait for dK(i), which may still read
        // it; the others write the dO half, whose last reader dV(i) retired
        // before dQ(i)
        const bool q_half = grp < C::QHALF_GROUPS || !C::EARLY_O;
        if (q_half && !warp_wait(dk_done, i & 1)) {
          ok = false;
          break;
        }
        const int s = i % C::NS;
#pragma unroll
        for (int cb = 0; cb < NR; ++cb) {
          const int col = grp * C::GD + cb * RUN;  // first dQ column of the run
          const int box = col / 32;
          uint8_t* base = box < C::BOXES_PER_STAGE ? sQ + s * C::TILE_BYTES + box * C::BOX_BYTES
                                                   : sdO + s * C::TILE_BYTES + (box - C::BOXES_PER_STAGE) * C::BOX_BYTES;
          uint8_t* line = base + row * 128;
#pragma unroll
          for (int c = 0; c < RUN / 4; ++c) {
            const int unit = (col % 32) / 4 + c;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q_ok)
              x = make_float4(__uint_as_float(qv[cb][c * 4]) * a.scale, __uint_as_float(qv[cb][c * 4 + 1]) * a.scale,
                              __uint_as_float(qv[cb][c * 4 + 2]) * a.scale,
                              __uint_as_float(qv[cb][c * 4 + 3]) * a.scale);
            *reinterpret_cast<float4*>(line + ((unit ^ (row & 7)) << 4)) = x;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_p(lane == 0, q_half ? &staged_q[s] : &staged_o[s]);
      }

      // ---- every kFlush iterations: fold dV / dK into the fp32 accumulators
      if (i + 1 < n && (i + 1) % kFlush == 0) {
        if (!warp_wait(acc_full, ((i + 1) / kFlush - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int cb = 0; cb < C::ACC_COLS / 32; ++cb) {
          uint32_t v[32];
          tmem_ld32(tbase + t_lane + acc_col + cb * 32, v);
          tmem_wait_ld();
          if (key_ok) {
            float4* dst = reinterpret_cast<float4*>(acc_glob + cb * 32);
            // MASK, FUSED: the first flush finds an accumulator that was not cleared
            const bool fresh = MASK && !STEP && i + 1 == kFlush;
#pragma unroll
            for (int v4 = 0; v4 < 8; ++v4) {
              float4 x = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : dst[v4];
              x.x += __uint_as_float(v[v4 * 4 + 0]) * acc_mul;
              x.y += __uint_as_float(v[v4 * 4 + 1]) * acc_mul;
              x.z += __uint_as_float(v[v4 * 4 + 2]) * acc_mul;
              x.w += __uint_as_float(v[v4 * 4 + 3]) * acc_mul;
              dst[v4] = x;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_p(lane == 0, acc_empty);
      }
    }
    if constexpr (BIAS) flush_sum();
    // ---------------------------------------------------------- epilogue
    if (ok) ok = warp_wait(done_bar, 0);
    if (ok) {
      tc_fence_after();
      // the accumulator holds earlier flushes (FUSED) or earlier steps (STEPWISE)
      const bool add_glob = STEP || nflush > 0;
#pragma unroll 1
      for (int cb = 0; cb < C::ACC_COLS / 32; ++cb) {
        uint32_t v[32];
        tmem_ld32(tbase + t_lane + acc_col + cb * 32, v);
        tmem_wait_ld();
        if (key_ok) {
          float x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]) * acc_mul;
          if (add_glob) {
            const float4* src = reinterpret_cast<const float4*>(acc_glob + cb * 32);
#pragma unroll
            for (int v4 = 0; v4 < 8; ++v4) {
              const float4 y = src[v4];
              x[v4 * 4 + 0] += y.x;
              x[v4 * 4 + 1] += y.y;
              x[v4 * 4 + 2] += y.z;
              x[v4 * 4 + 3] += y.w;
            }
          }
          if (!STEP && !(MASK && a.mask.splits > 1)) {
            __nv_bfloat16* dst = (owns_dv ? a.dv : a.dk) + krow * D + acc_part + cb * 32;
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
              uint4 w;
              w.x = pack_bf16(x[v4 * 8 + 0], x[v4 * 8 + 1]);
              w.y = pack_bf16(x[v4 * 8 + 2], x[v4 * 8 + 3]);
              w.z = pack_bf16(x[v4 * 8 + 4], x[v4 * 8 + 5]);
              w.w = pack_bf16(x[v4 * 8 + 6], x[v4 * 8 + 7]);
              reinterpret_cast<uint4*>(dst)[v4] = w;
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(acc_glob + cb * 32);
#pragma unroll
            for (int v4 = 0; v4 < 8; ++v4)
              dst[v4] = make_float4(x[v4 * 4], x[v4 * 4 + 1], x[v4 * 4 + 2], x[v4 * 4 + 3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::CW + 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

template <int D, bool STEP, int VARIANT>
int launch_bwd_t(const loong_attn_desc& d, const void* q, const void* k, const void* v, const void* dout,
                 const float* stats, float* dq_acc, void* dk, void* dv, float* dk_acc,
                 float* dv_acc, cudaStream_t stream, void* kv_recv, const BiasView* bias, float* dbias_part,
                 const MaskView* mask) {
  using C = BwdCfg<D>;
  const Layout lay = layout_of(d);
  const int64_t rows = lay.view_rows(d.batch);
  const int vq = lay.view_heads(d.hq), vkv = lay.view_heads(d.hkv);
  CUtensorMap mq, mk, mv, mo;
  int st;
  if ((st = make_head_tile_map(&mq, q, rows, vq, D)) != LOONG_OK) return st;
  if ((st = make_head_tile_map(&mk, k, rows, vkv, D)) != LOONG_OK) return st;
  if ((st = make_head_tile_map(&mv, v, rows, vkv, D)) != LOONG_OK) return st;
  if ((st = make_head_tile_map(&mo, dout, rows, vq, D)) != LOONG_OK) return st;
  CUtensorMap mdq;
  if ((st = make_f32_tile_map(&mdq, dq_acc, rows, vq, D)) != LOONG_OK) return st;
  BwdArgs a;
  a.lay = lay;
  a.kv_held = 0;
  a.batch = static_cast<int>(d.batch);
  a.S = static_cast<int>(d.seqlen);
  a.hq = d.hq;
  a.hkv = d.hkv;
  a.G = d.hq / d.hkv;
  a.ring = ring_geom(d);
  a.scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / std::sqrt(static_cast<float>(D));
  a.mask = VARIANT == kBwdMask || VARIANT == kBwdCap ? *mask : MaskView{};
  a.scale_log2 = a.scale * kLog2e;
  a.lse2 = stats;
  a.blk_pad = stat_block_pad(a.ring.blk);
  a.stat_len = static_cast<int>(stat_row_len(a.ring));
  a.dstat = stats + d.batch * d.hq * static_cast<int64_t>(a.stat_len);
  a.dq_acc = dq_acc;
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.dk_acc = dk_acc;
  a.dv_acc = dv_acc;
  a.bias = VARIANT == kBwdBias ? *bias : BiasView{};
  a.dbias_part = dbias_part;
  a.err = device_error_word();
  if (!a.err) return LOONG_ERR_CUDA;
  constexpr auto kern = ring_bwd_kernel<D, STEP, VARIANT>;
  if ((st = kernel_ready<kern>(C::SMEM_BYTES, 0)) != LOONG_OK) return st;
  const int64_t grid = d.batch * d.hkv * static_cast<int64_t>(a.ring.nblocks) * a.ring.ntile * a.mask.splits;
  if (grid <= 0 || grid > 0x7fffffff) return LOONG_ERR_INVALID_ARG;
  const int t_first = 0, t_last = d.cp;
  if (!STEP) {
    a.t_begin = t_first;
    a.t_end = t_last;
    record_start(stream);
    if constexpr (VARIANT == kBwdMask || VARIANT == kBwdCap)
      st = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), C::THREADS, C::SMEM_BYTES, stream, mq, mk, mv, mo,
                            mdq, a);
    else
      kern<<<static_cast<unsigned>(grid), C::THREADS, C::SMEM_BYTES, stream>>>(mq, mk, mv, mo, mdq, a);
    record_stop(stream);
    return st == LOONG_OK ? check_launch() : st;
  }
  if (is_copy_mode(d)) {
    // receive buffers K0, K1, V0, V1, each the size of K (exchange.h); dK, dV
    // are accumulated at the owner's rows, so only K and V travel
    const size_t kv_bytes = static_cast<size_t>(rows) * vkv * D * 2;
    uint8_t* rb = static_cast<uint8_t*>(kv_recv);
    void* const rk[2] = {rb, rb + kv_bytes};
    void* const rv[2] = {rb + 2 * kv_bytes, rb + 3 * kv_bytes};
    CUtensorMap mkr[2], mvr[2];
    for (int i = 0; i < 2; ++i) {
      if ((st = make_head_tile_map(&mkr[i], rk[i], rows, vkv, D)) != LOONG_OK) return st;
      if ((st = make_head_tile_map(&mvr[i], rv[i], rows, vkv, D)) != LOONG_OK) return st;
    }
    record_start(stream);
    st = run_exchanged_steps(d, k, v, rk, rv, stream, [&](int t, int buf) {
      NvtxRange step("bwd ring step %d", t);
      a.t_begin = t;
      a.t_end = t + 1;
      a.kv_held = buf >= 0;
      kern<<<static_cast<unsigned>(grid), C::THREADS, C::SMEM_BYTES, stream>>>(
          mq, buf >= 0 ? mkr[buf] : mk, buf >= 0 ? mvr[buf] : mv, mo, mdq, a);
      return check_launch();
    });
    record_stop(stream);
    return st;
  }
  record_start(stream);
  for (int t = t_first; t < t_last; ++t) {
    NvtxRange step("bwd ring step %d", t);
    a.t_begin = t;
    a.t_end = t + 1;
    kern<<<static_cast<unsigned>(grid), C::THREADS, C::SMEM_BYTES, stream>>>(mq, mk, mv, mo, mdq, a);
    if ((st = check_launch()) != LOONG_OK) return st;
  }
  record_stop(stream);
  return LOONG_OK;
}

template <int VARIANT>
int launch_bwd_v(const loong_attn_desc& d, const void* q, const void* k, const void* v, const void* dout,
                 const float* stats, float* dq_acc, void* dk, void* dv, float* dk_acc, float* dv_acc,
                 cudaStream_t stream, void* kv_recv, const BiasView* bias, float* part, const MaskView* mask) {
  const bool step = d.mode != LOONG_MODE_FUSED;
  if (d.head_dim == 128)
    return step ? launch_bwd_t<128, true, VARIANT>(d, q, k, v, dout, stats, dq_acc, dk, dv, dk_acc, dv_acc, stream,
                                                   kv_recv, bias, part, mask)
                : launch_bwd_t<128, false, VARIANT>(d, q, k, v, dout, stats, dq_acc, dk, dv, dk_acc, dv_acc, stream,
                                                    kv_recv, bias, part, mask);
  if (d.head_dim == 64)
    return step ? launch_bwd_t<64, true, VARIANT>(d, q, k, v, dout, stats, dq_acc, dk, dv, dk_acc, dv_acc, stream,
                                                  kv_recv, bias, part, mask)
                : launch_bwd_t<64, false, VARIANT>(d, q, k, v, dout, stats, dq_acc, dk, dv, dk_acc, dv_acc, stream,
                                                   kv_recv, bias, part, mask);
  return LOONG_ERR_UNSUPPORTED;
}

}  // namespace

int launch_bwd(const loong_attn_desc& d, const void* q, const void* k, const void* v, const void* o,
               const void* o_res, const float* lse, const void* dout, void* dq, void* dk, void* dv, float* dq_acc,
               float* dvec, float* dk_acc, float* dv_acc, cudaStream_t stream, void* kv_recv, const BiasView* bias,
               float* dbias_part, const MaskView* mask) {
  const int64_t q_elems = d.batch * d.seqlen * d.hq * d.head_dim;
  const int64_t kv_elems = d.batch * d.seqlen * d.hkv * d.head_dim;
  const bool step = d.mode != LOONG_MODE_FUSED;
  if (mask && mask->splits > 1) {
    dk_acc = mask->dk_parts;
    dv_acc = mask->dv_parts;
  }
  int st;
  cudaError_t e = bias || mask ? cudaSuccess : cudaMemsetAsync(dq_acc, 0, static_cast<size_t>(q_elems) * 4, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  // FUSED walks of at most kFlush (tile, head) pairs never touch the dK, dV accumulators;
  // with a mask longer ones write them first
  const RingGeom g = ring_geom(d);
  const int64_t longest = static_cast<int64_t>(d.hq / d.hkv) * g.nblocks * g.ntile;
  if ((step || (longest > kFlush && !mask)) &&
      ((e = cudaMemsetAsync(dk_acc, 0, static_cast<size_t>(kv_elems) * 4, stream)) != cudaSuccess ||
       (e = cudaMemsetAsync(dv_acc, 0, static_cast<size_t>(kv_elems) * 4, stream)) != cudaSuccess))
    return cuda_fail(e);
  if (!bias && !mask && (st = launch_bwd_rowstats(d, o, o_res, dout, lse, dvec, stream)) != LOONG_OK) return st;
  st = bias   ? launch_bwd_v<kBwdBias>(d, q, k, v, dout, dvec, dq_acc, dk, dv, dk_acc, dv_acc, stream, kv_recv, bias,
                                       dbias_part, nullptr)
       : mask && mask->cap.inv > 0.f
           ? launch_bwd_v<kBwdCap>(d, q, k, v, dout, dvec, dq_acc, dk, dv, dk_acc, dv_acc, stream, kv_recv, nullptr,
                                   nullptr, mask)
       : mask ? launch_bwd_v<kBwdMask>(d, q, k, v, dout, dvec, dq_acc, dk, dv, dk_acc, dv_acc, stream, kv_recv,
                                       nullptr, nullptr, mask)
              : launch_bwd_v<kBwdPlain>(d, q, k, v, dout, dvec, dq_acc, dk, dv, dk_acc, dv_acc, stream, kv_recv,
                                        nullptr, nullptr, nullptr);
  if (st != LOONG_OK) return st;
  const bool parts = mask && mask->splits > 1;
  if (!bias && !parts && (st = launch_f32_to_bf16(dq_acc, dq, q_elems, stream)) != LOONG_OK) return st;
  if (step) {
    if ((st = launch_f32_to_bf16(dk_acc, dk, kv_elems, stream)) != LOONG_OK) return st;
    if ((st = launch_f32_to_bf16(dv_acc, dv, kv_elems, stream)) != LOONG_OK) return st;
  }
  return LOONG_OK;
}

}  // namespace loong
