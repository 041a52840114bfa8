// paged_attn.cu -- attention of new tokens over a cache of pages, which first takes
// their keys and values in: the next token of many sequences, a chunk of a long
// prompt, or a mixture.
//
//   z_ij = scale q_i.k_j, or cap tanh(scale q_i.k_j / cap)
//   O_i = sum_j softmax_j(z_ij) v_j over j <= i (and j > i - window), j a position of
//   i's sequence, its K and V at row j mod page of page table[sequence][j / page]
//
// Two launches, the second's blocks starting while the first runs.  paged_prep_kernel
// writes the new keys and values into their pages and lays the work out (block 0,
// paged_plan.h): a group is up to SLOTS * (128 / G) new tokens of a sequence, G query
// heads to a kv head; with a kv head it makes an item, whose rows (token by token, the kv
// head's G query heads each) fill SLOTS blocks of 128 rows of the matrix instructions,
// and its 128-key tiles are the units of work.
// paged_attn_kernel runs one block an SM; block c takes units [U c / blocks, U (c + 1) /
// blocks) of the whole list, whatever the sequences' lengths: the long axis is split
// where the rows are few, and every SM streams the same number of keys.  A block
// stores the items that it holds whole; of an item split between blocks each stores
// the rows' unnormalised output, maximum and sum, and the last warp to arrive (a
// ticket for every 32 rows, cleared by the first launch) joins them in the order of
// the keys, so the result does not depend on who is last.
//
// One kernel for both ends: with one new token the rows are few and memory is the
// bound (a 128 x 128 score tile takes the matrix instructions, most of whose rows are
// then empty, 0.45 of the time in which its 64 KB of K and V arrive: 0.67 and 1.48 us an
// SM at head dimension 128); with a chunk two blocks of rows share every K and V
// tile, and the matrix instructions and the softmax between them are the bound.
//
// Warps: 4 * SLOTS softmax warps (a row in every lane), a TMA warp, an MMA warp.  As
// in attn_fwd.cu, S = Q K^T goes to one of NSB score buffers in tensor memory, P
// overwrites it, O += P V; the softmax forms P against the running maximum and only
// looks for a tile's maximum when a row's sum passes 2^8 of it.  P and V are bf16,
// V being read where it lies; O is divided by the sum of the rounded P, so that a row
// that one key dominates has its V back to O's own rounding, and the LSE comes from
// the sum before rounding.
// What a masked place of a tile holds (rows of the page behind the sequence, keys
// that are yet to come) does not matter: its scores are replaced, and where a tile is
// not seen whole, rows of V that are not finite are cleared in shared memory first
// and the scores of their keys, for the rows that do see them, made NaN.
//
// Measured, both launches: the next token after 131,071 (32 + 8 heads of 128) 100 us, 5.3
// TB/s; of 61 sequences of 64 to 16,000 keys (64 + 8 heads) 135 us, 5.1 TB/s; 2,048 new
// tokens over 32K keys (32 + 8 heads) 0.79 ms, 1.35 PFLOP/s, with capped scores 1.22.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fwd_jobs.h"
#include "internal.h"
#include "paged_plan.h"
#include "ptx.cuh"
#include "softcap.cuh"
#include "v16.cuh"

namespace loong {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kSumBound = 256.0f;        // 2^threshold: the largest P let through without a new maximum
// What an item costs a block beside its tiles, in tiles: its first scores wait for Q and
// its rows for the last product.  Counted out of the division it left blocks that drew
// many short items behind: 61 sequences of 64 to 16,000 keys, 64 + 8 heads of 128, 226 us
// for 0, 167 for 2, 134 for 4; 13 sequences of up to 300 new tokens in a window 74, 46, 45.
constexpr int kItemUnits = 4;
constexpr int kMaxSequences = 4096;
constexpr int kPrepThreads = 1024;

template <int D, int SLOTS>
struct PagedCfg {
  static constexpr int ATOMS = D / 64;
  static constexpr int ATOM_BYTES = kTile * 128;
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int NSB = fwd_score_buffers(D, SLOTS);
  static constexpr int NS = D == 64 ? 6 : SLOTS == 1 ? 3 : 2;  // K and V stages: what shared memory holds
  // Segments whose description is kept.  The producer runs at most three ahead of the
  // softmax: Q of the next loads once this one's Q K^T are done, and NSB score buffers
  // let those of two segments of a tile each pass a softmax that has not begun them.
  static constexpr int SEGS = 4;
  static constexpr int SOFTMAX_WARPS = 4 * SLOTS;
  // two slots: as the ring forward, registers of a third warpgroup go to the softmax
  static constexpr bool SPLIT = SLOTS == 2;
  static constexpr int THREADS = SPLIT ? 384 : 192;
  static constexpr int SPLIT_REGS = 168, SOFTMAX_REGS = 216, OTHER_REGS = 72;
  static_assert(256 * SOFTMAX_REGS + 128 * OTHER_REGS <= 384 * SPLIT_REGS, "register split");
  static constexpr int NBARS = SEGS + 1 + 4 * NS + 3 + 3 + 2 + 1 + 1;
  static constexpr int SMEM_BYTES = (SLOTS + 2 * NS) * TILE_BYTES + NBARS * 8 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t S_COL(int buf) { return static_cast<uint32_t>(buf) * 128u; }
  __host__ __device__ static constexpr uint32_t O_COL(int h) { return NSB * 128u + static_cast<uint32_t>(h) * D; }
  static_assert(NSB * 128 + SLOTS * D <= 512 && SMEM_BYTES <= 232448, "tensor and shared memory");
};

struct PagedArgs {
  int batch, tokens, hq, hkv, G, per_slot;  // per_slot: tokens in 128 rows
  int page_log2, num_pages, max_pages;
  int window;  // 0 (none), or less than a row of the table holds
  int max_groups;
  float scale_log2;
  ScoreCap cap;
  const int* table;    // [batch][max_pages]
  const int* lens;     // [batch]
  const int* starts;   // [batch + 1]
  Group* groups;       // [max_groups]
  int* prefix;         // [max_groups + 1]: units before a group (of one kv head)
  int* count;          // groups
  unsigned* tickets;   // [max_groups * hkv * softmax warps]
  float* part_o;       // [blocks * 2][SLOTS * 128][D]
  float4* part_ml;     // [blocks * 2][SLOTS * 128]: maximum (log2 units), sum, sum of the rounded P, -
  __nv_bfloat16* o;    // [tokens][hq][D]
  float* lse;          // [hq][tokens]
  unsigned* err;
};

// ------------------------------------------------------------------ preparation
struct AppendArgs {
  const uint4 *k, *v;  // new tokens' rows, or null
  uint4 *k_pages, *v_pages;
  int64_t k_stride, v_stride;  // vectors of 8 from token to token
  int row_vecs;                // hkv * D / 8
  int tickets;
};

// Inclusive sum over the block's threads; *total their whole.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* total) {
  __shared__ T sums[kPrepThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  T s = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return warp ? x + before : x;
}

__device__ __forceinline__ SequenceCut sequence(const PagedArgs& a, int b) {
  const int64_t room = static_cast<int64_t>(a.max_pages) << a.page_log2;
  return cut_sequence(a.starts[b], a.starts[b + 1], a.lens[b], a.tokens, room);
}

// The groups and the units before each: an item's tiles, and kItemUnits.
__device__ __forceinline__ void plan(const PagedArgs& a, int per_group) {
  __shared__ int first[kMaxSequences];  // the sequences' first groups
  GroupSum sum = 0, part;
  bool fine = true;
  for (int b0 = 0; b0 < a.batch; b0 += kPrepThreads) {
    const int b = b0 + threadIdx.x;
    GroupSum n = 0;
    if (b < a.batch) {
      const SequenceCut c = sequence(a, b);
      fine &= c.fine;
      n = groups_of(c.count, per_group);
    }
    const GroupSum end = block_scan(n, &part);
    if (b < a.batch) first[b] = cut_groups(sum + end - n, a.max_groups);
    sum += part;
  }
  fine &= sum <= a.max_groups;  // else sequences share tokens: more work than there is room for
  const int base = cut_groups(sum, a.max_groups);
  if (!fine) atomicOr(a.err, kErrBounds);
  __syncthreads();
  int units_before = 0, total;
  for (int g0 = 0; g0 < base; g0 += kPrepThreads) {
    const int g = g0 + threadIdx.x;
    int n = 0;
    if (g < base) {
      const int b = sequence_of_group(first, a.batch, g);
      const Group r = make_group(sequence(a, b), b, (g - first[b]) * per_group, per_group, a.window);
      n = r.tiles + kItemUnits;
      a.groups[g] = r;
    }
    const int end = block_scan(n, &total);
    if (g < base) a.prefix[g] = units_before + end - n;
    units_before += total;
  }
  if (threadIdx.x == 0) {
    a.prefix[base] = units_before;
    *a.count = base;
  }
}

// The sequence that new token t belongs to (-1: none), by the whole warp: the last
// one that starts at or before it.
__device__ __forceinline__ int sequence_of(const PagedArgs& a, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.batch;
  while (n > 0) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && a.starts[i] <= t);
    if (m == 0) return -1;
    const int last = 31 - __clz(m);
    lo += last * step;
    n = min(step, n - last * step);
    if (step == 1) break;
  }
  return t < a.starts[lo + 1] ? lo : -1;
}

// Block 0 lays the work out, the others copy a new token's keys and values a warp.
__global__ void __launch_bounds__(kPrepThreads) paged_prep_kernel(const __grid_constant__ PagedArgs a,
                                                                  const __grid_constant__ AppendArgs n,
                                                                  int per_group) {
  next_launch_go();
  const int id = blockIdx.x * kPrepThreads + threadIdx.x, threads = gridDim.x * kPrepThreads;
  for (int i = id; i < n.tickets; i += threads) a.tickets[i] = 0;
  if (blockIdx.x == 0) {
    plan(a, per_group);
    return;
  }
  const int lane = threadIdx.x & 31, warps = (gridDim.x - 1) * (kPrepThreads / 32);
  const int page_rows = 1 << a.page_log2;
  for (int t = (blockIdx.x - 1) * (kPrepThreads / 32) + threadIdx.x / 32; t < a.tokens; t += warps) {
    const int b = sequence_of(a, t);
    if (b < 0) continue;
    const SequenceCut c = sequence(a, b);
    const int pos = c.len - c.count + t - c.tok;
    if (pos < 0) continue;  // reported by the plan
    const int page = a.table[static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_log2)];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(a.err, kErrBounds);
      continue;
    }
    const int64_t row = (static_cast<int64_t>(page) << a.page_log2) + (pos & (page_rows - 1));
    for (int i = lane; i < n.row_vecs; i += 32) {
      const uint4 kv = __ldg(n.k + t * n.k_stride + i), vv = __ldg(n.v + t * n.v_stride + i);
      n.k_pages[row * n.row_vecs + i] = kv;
      n.v_pages[row * n.row_vecs + i] = vv;
    }
  }
}

// ---------------------------------------------------------------------- attention
// A block's share of an item.
struct Segment {
  int tok, count, pos, kvh;
  int seq, tile, tiles;  // tiles of this share; 0: no further segment
  int part;              // where to store it, -1: the item is whole
  int parts, first_part, first_block, item;
};

template <int D, int SLOTS, bool CAP>
__global__ void __launch_bounds__(PagedCfg<D, SLOTS>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedArgs a) {
  using C = PagedCfg<D, SLOTS>;
  constexpr int NSB = C::NSB, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ Segment segs[C::SEGS];
  __shared__ unsigned bad_v[NS][4];  // a tile's keys whose V is not finite
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + SLOTS * C::TILE_BYTES;
  uint8_t* sV = sK + NS * C::TILE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NS * C::TILE_BYTES);
  uint64_t* seg_full = bars;                // SEGS: a segment's description and Q (producer -> all)
  uint64_t* q_empty = seg_full + C::SEGS;   // a segment's Q K^T done (MMA -> producer)
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + NS;
  uint64_t* v_full = k_empty + NS;
  uint64_t* v_empty = v_full + NS;
  uint64_t* s_full = v_empty + NS;  // NSB
  uint64_t* p_full = s_full + 3;    // NSB
  uint64_t* pv_done = p_full + 3;   // SLOTS
  uint64_t* o_full = pv_done + 2;   // a segment's O (MMA -> softmax)
  uint64_t* drain = o_full + 1;
  volatile int* abort_flag = &abort_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SEGS; ++s) mbar_init(&seg_full[s], 1);
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
  if (warp == C::SOFTMAX_WARPS + 1) {
    tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == C::SOFTMAX_WARPS && lane == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base_sh;
  previous_launch_wait();
  if constexpr (C::SPLIT) {
    if (warp >= C::SOFTMAX_WARPS) regs_dec<C::OTHER_REGS>();
  }
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err));
  };

  if (warp == C::SOFTMAX_WARPS) {
    // ------------------------------------------------------------ TMA producer
    const uint32_t leader = lane == 0;
    const int groups = *a.count;
    const int64_t U = static_cast<int64_t>(a.prefix[groups]) * a.hkv;
    const int64_t blocks = min(static_cast<int64_t>(gridDim.x), U);
    const int c = blockIdx.x;
    const int64_t u0 = c < blocks ? U * c / blocks : 0, u1 = c < blocks ? U * (c + 1) / blocks : 0;
    // the block that unit u belongs to: the last one whose units begin at or before it
    auto block_of = [&](int64_t u) { return static_cast<int>(((u + 1) * blocks - 1) / U); };
    int gi = 0;
    for (int n = groups; n > 1;) {  // the last group that begins at or before u0
      const int step = (n + 31) / 32, i = gi + lane * step;
      const bool before = lane * step < n && static_cast<int64_t>(a.prefix[i]) * a.hkv <= u0;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
      gi += last * step;
      n = min(step, n - last * step);
    }
    const int page_rows = 1 << a.page_log2;
    const int box = min(page_rows, kTile), boxes = kTile / box;
    int it = 0, seg = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const int group = gi;
      const Group g = a.groups[gi];
      const int64_t base = static_cast<int64_t>(a.prefix[gi]) * a.hkv;
      const int units = g.tiles + kItemUnits;
      const int kvh = static_cast<int>((u - base) / units), off = static_cast<int>((u - base) % units);
      const int64_t begin = u - off, end = begin + units;  // the item's units, kItemUnits and then its tiles
      const int skip = max(off - kItemUnits, 0);
      u = min(end, u1);
      const int n = max(static_cast<int>(u - begin) - kItemUnits, 0) - skip;
      if (u == end && kvh == a.hkv - 1) ++gi;
      if (n == 0) continue;
      Segment sg;
      sg.tok = g.tok;
      sg.count = g.count;
      sg.pos = g.pos;
      sg.kvh = kvh;
      sg.seq = g.seq;
      sg.tile = g.tile + skip;
      sg.tiles = n;
      sg.item = group * a.hkv + kvh;
      sg.part = -1;
      sg.parts = 1;
      sg.first_part = sg.first_block = 0;
      if (n < g.tiles) {
        sg.part = 2 * c + (seg == 0 ? 0 : 1);
        sg.first_block = block_of(begin + kItemUnits);
        sg.parts = block_of(end - 1) - sg.first_block + 1;
        sg.first_part = U * sg.first_block / blocks >= begin ? 0 : 1;  // a block's first share or its last
      }
      // keys [from, to) are seen by some row: only their boxes are loaded
      const int to = g.pos + g.count, from = a.window ? max(g.pos - a.window + 1, 0) : 0;
      const int* pages = a.table + static_cast<int64_t>(g.seq) * a.max_pages;
      int page = 0;
      auto look_up = [&](int tile) {  // a box in every lane
        const int key = tile * kTile + lane * box;
        page = lane < boxes && key < to && key + box > from ? __ldg(pages + (key >> a.page_log2)) : -1;
      };
      look_up(sg.tile);
      // Q, once the segment before has been multiplied with it: after the first tile of K
      auto load_q = [&]() {
        if (seg > 0 && !warp_wait(q_empty, (seg - 1) & 1)) return false;
        uint64_t* full = &seg_full[seg % C::SEGS];
        if (leader) segs[seg % C::SEGS] = sg;
        const int slots = SLOTS == 2 && g.count > a.per_slot ? 2 : 1;
        mbar_expect_tx_p(leader, full, slots * C::ATOMS * a.per_slot * a.G * 128);
        for (int h = 0; h < slots; ++h)
          for (int at = 0; at < C::ATOMS; ++at)
            tma_load_3d_p(leader, sQ + h * C::TILE_BYTES + at * C::ATOM_BYTES, &tmQ, full, at * 64, kvh * a.G,
                          g.tok + h * a.per_slot);
        return true;
      };
      bool q_loaded = false;
      for (int j = 0; j < n; ++j, ++it) {
        const int s = it % NS;
        const int key = (sg.tile + j) * kTile + lane * box;
        const bool live = lane < boxes && key < to && key + box > from;
        int row = a.num_pages << a.page_log2;  // a page that there is not reads as zeros
        if (live) {
          if (page >= 0 && page < a.num_pages)
            row = (page << a.page_log2) + (key & (page_rows - 1));
          else
            atomicOr(a.err, kErrBounds);
        }
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * box * 128 * C::ATOMS;
        if (j + 1 < n) look_up(sg.tile + j + 1);
        if (it >= NS && !warp_wait(&k_empty[s], (it / NS - 1) & 1)) {
          ok = false;
          break;
        }
        mbar_expect_tx_p(leader, &k_full[s], bytes);
        __syncwarp();
        if (live) {
          for (int at = 0; at < C::ATOMS; ++at)
            tma_load_3d(sK + s * C::TILE_BYTES + at * C::ATOM_BYTES + lane * box * 128, &tmK, &k_full[s], at * 64, kvh,
                        row);
        }
        if (j == 0) q_loaded = load_q();
        if (!q_loaded || (it >= NS && !warp_wait(&v_empty[s], (it / NS - 1) & 1))) {
          mbar_drain(&k_full[s], (it / NS) & 1, a.err);
          ok = false;
          break;
        }
        if (lane < 4) bad_v[s][lane] = 0;
        __syncwarp();
        mbar_expect_tx_p(leader, &v_full[s], bytes);
        __syncwarp();
        if (live) {
          for (int at = 0; at < C::ATOMS; ++at)
            tma_load_3d(sV + s * C::TILE_BYTES + at * C::ATOM_BYTES + lane * box * 128, &tmV, &v_full[s], at * 64, kvh,
                        row);
        }
      }
      if (q_loaded) ++seg;
    }
    if (ok) {  // the end (it needs no Q, but its place among the descriptions)
      if (seg == 0 || warp_wait(q_empty, (seg - 1) & 1)) {
        if (leader) segs[seg % C::SEGS].tiles = 0;
        mbar_arrive_p(leader, &seg_full[seg % C::SEGS]);
      }
    }
    // every copy lands before the block ends
    for (int s = 0; s < NS; ++s) {
      const int cnt = it > s ? (it - 1 - s) / NS + 1 : 0;
      if (cnt) {
        mbar_drain(&k_full[s], (cnt - 1) & 1, a.err);
        mbar_drain(&v_full[s], (cnt - 1) & 1, a.err);
      }
    }
    for (int s = max(0, seg - 1); s < seg; ++s) mbar_drain(&seg_full[s % C::SEGS], (s / C::SEGS) & 1, a.err);
  } else if (warp == C::SOFTMAX_WARPS + 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_qk = idesc_bf16(128, 128, false, false);
    constexpr uint32_t id_pv = idesc_bf16(128, D, false, true);
    const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sK), v_addr = smem_u32(sV);
    int it = 0, J = 0;  // tiles and jobs of the segments before
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      if (!warp_wait(&seg_full[seg % C::SEGS], (seg / C::SEGS) & 1)) break;
      tc_fence_after();
      const int n = segs[seg % C::SEGS].tiles;
      if (n == 0) break;
      // Q K^T of the segment's job i into buffer (J + i) mod NSB
      auto issue_qk = [&](int i) {
        const int jt = it + i / SLOTS, h = i % SLOTS, st = jt % NS;
        if (h == 0) {
          if (!warp_wait(&k_full[st], (jt / NS) & 1)) return false;
          tc_fence_after();
        }
        const uint64_t qa = sdesc_sw128(q_addr + h * C::TILE_BYTES, 16, 1024);
        const uint64_t kb = sdesc_sw128(k_addr + st * C::TILE_BYTES, 16, 1024);
        const int buf = (J + i) % NSB;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32) >> 4;
          mma_ss_w(tbase + C::S_COL(buf), qa + off, kb + off, id_qk, kk > 0);
        }
        mma_commit_w(&s_full[buf]);
        if (h == SLOTS - 1) mma_commit_w(&k_empty[st]);
        if (i == SLOTS * n - 1) mma_commit_w(q_empty);
        return true;
      };
      for (int i = 0; i < NSB && i < SLOTS * n && ok; ++i) ok = issue_qk(i);
      for (int j = 0; j < n && ok; ++j) {
        const int st = (it + j) % NS;
        if (!(ok = warp_wait(&v_full[st], ((it + j) / NS) & 1))) break;
#pragma unroll
        for (int h = 0; h < SLOTS; ++h) {
          const int i = SLOTS * j + h, buf = (J + i) % NSB;
          if (!(ok = warp_wait(&p_full[buf], ((J + i) / NSB) & 1))) break;
          tc_fence_after();
          const uint64_t vb = sdesc_sw128(v_addr + st * C::TILE_BYTES, C::ATOM_BYTES, 1024);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts_w(tbase + C::O_COL(h), tbase + C::S_COL(buf) + kk * 8, vb + (kk * 2048 >> 4), id_pv,
                     j > 0 || kk > 0);
          mma_commit_w(&pv_done[h]);
          if (h == SLOTS - 1) mma_commit_w(&v_empty[st]);
          if (i + NSB < SLOTS * n && !(ok = issue_qk(i + NSB))) break;
        }
      }
      if (ok) mma_commit_w(o_full);
      it += n;
      J += SLOTS * n;
    }
    mma_commit_w(drain);
    mbar_drain(drain, 0, a.err);
  } else if (warp < C::SOFTMAX_WARPS) {
    if constexpr (C::SPLIT) regs_inc<C::SOFTMAX_REGS>();
    // ------------------------------------------------------------ softmax
    const int h = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tO = tbase + t_lane + C::O_COL(h);
    const float sl2 = a.scale_log2;
    int it = 0, J = 0;
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      if (!warp_wait(&seg_full[seg % C::SEGS], (seg / C::SEGS) & 1)) break;
      const Segment sg = segs[seg % C::SEGS];
      const int n = sg.tiles;
      if (n == 0) break;
      // this row's token and head, and the keys that it sees (rows without a token: all)
      const int here = min(sg.count - h * a.per_slot, a.per_slot) * a.G;  // the slot's rows
      const int tl = row / a.G;
      const bool valid = row < here;
      int2 see = make_int2(0, 0x7fffffff);
      if (valid) {
        const int pos = sg.pos + h * a.per_slot + tl;
        see = make_int2(a.window ? max(pos - a.window + 1, 0) : 0, max(pos + 1, 0));
      }
      const bool some = quarter * 32 < here;  // the warp has rows
      float m_run = -INFINITY, l_run = 0.f, r_run = 0.f;  // r: the sum of the rounded P
      for (int j = 0; j < n; ++j) {
        const int i = J + SLOTS * j + h, buf = i % NSB;
        const uint32_t tS = tbase + t_lane + C::S_COL(buf);
        if (!(ok = warp_wait(&s_full[buf], (i / NSB) & 1))) break;
        tc_fence_after();
        if (some) {
          const int k0 = (sg.tile + j) * kTile;
          const int lo = see.x - k0, hi = see.y - k0;  // columns that the row sees
          // some row of the item does not see the whole tile (the same for every warp:
          // what one clears the others have to make NaN)
          const bool part = sg.pos + 1 < k0 + kTile || (a.window && sg.pos + sg.count - a.window > k0);
          unsigned bad[4] = {};  // keys whose V is not finite
          if (part) {
            const int st = (it + j) % NS;
            if (!(ok = warp_wait(&v_full[st], ((it + j) / NS) & 1))) break;
            uint8_t* tile = sV + st * C::TILE_BYTES;
            // a key in every lane; 16-byte parts in the order that has no bank conflicts
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
              const int key = cb * 32 + lane;
              // 0 times a value that is not finite is NaN, which the sum keeps
              __nv_bfloat162 nan = __float2bfloat162_rn(0.f);
              const __nv_bfloat162 zero = nan;
#pragma unroll 4
              for (int p = 0; p < D / 8; ++p) {
                const uint4 x = *reinterpret_cast<const uint4*>(tile + (p >> 3) * C::ATOM_BYTES + key * 128 +
                                                                (((p & 7) ^ (key & 7)) << 4));
                const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
                for (int e = 0; e < 4; ++e) nan = __hfma2(v[e], zero, nan);
              }
              bad[cb] = __ballot_sync(0xffffffffu, __hisnan(nan.x) || __hisnan(nan.y));
            }
            // noted before they are cleared: another warp that finds them cleared
            // finds them noted
            if (lane < 4)
              atomicOr(&bad_v[st][lane], lane == 0 ? bad[0] : lane == 1 ? bad[1] : lane == 2 ? bad[2] : bad[3]);
            __threadfence_block();
            __syncwarp();
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
              if (bad[cb] >> lane & 1) {
                for (int p = 0; p < D / 8; ++p)
                  *reinterpret_cast<uint4*>(tile + (p >> 3) * C::ATOM_BYTES + (cb * 32 + lane) * 128 + ((p & 7) << 4)) =
                      make_uint4(0, 0, 0, 0);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) bad[cb] |= *reinterpret_cast<volatile unsigned*>(&bad_v[st][cb]);
          }
          // of columns 32 cb .. of the tile: -inf for keys that are not seen, NaN for
          // those whose V holds values that are not finite
          auto seen = [&](int c) { return low_bits(hi - c) & ~low_bits(lo - c); };
          auto mask_columns = [&](uint32_t(&s)[32], int cb, uint32_t nan) {
            const uint32_t bits = seen(cb * 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (nan >> e & 1) s[e] = 0x7fffffffu;
              if (!(bits >> e & 1)) s[e] = __float_as_uint(-INFINITY);
            }
          };
          uint32_t sr[4][32], pk[2][32];
          // the scores, masked columns at -inf
          auto load_s = [&]() {
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) tmem_ld32(tS + cb * 32, sr[cb]);
            tmem_wait_ld();
            if (part) {
#pragma unroll
              for (int cb = 0; cb < 4; ++cb) mask_columns(sr[cb], cb, bad[cb]);
            }
          };
          // a pair of P rounded and packed, and added to the row's sums
          float2 sum = make_float2(0.f, 0.f), rsum = sum;
          auto pack = [&](float p0, float p1) {
            const uint32_t p = pack_bf16(p0, p1);
            sum = __fadd2_rn(sum, make_float2(p0, p1));
            rsum = __fadd2_rn(rsum, make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)));
            return p;
          };
          // P = exp2(s * scale * log2e - ref); the row's sums of it
          auto form_p = [&](float ref) {
            const float2 sl2v = make_float2(sl2, sl2), nref = make_float2(-ref, -ref);
            sum = rsum = make_float2(0.f, 0.f);
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 x = __ffma2_rn(
                    make_float2(__uint_as_float(sr[cb][e]), __uint_as_float(sr[cb][e + 1])), sl2v, nref);
                pk[cb >> 1][(cb & 1) * 16 + (e >> 1)] = pack(fast_exp2(x.x), fast_exp2(x.y));
              }
            }
            return make_float2(sum.x + sum.y, rsum.x + rsum.y);
          };
          auto tile_max = [&]() {  // log2 units
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int cb = 0; cb < 4; ++cb)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                mx0 = fmax3(mx0, __uint_as_float(sr[cb][e]), __uint_as_float(sr[cb][e + 1]));
                mx1 = fmax3(mx1, __uint_as_float(sr[cb][e + 2]), __uint_as_float(sr[cb][e + 3]));
              }
            return fmaxf(mx0, mx1) * sl2;
          };
          // the running maximum takes the tile's in; false: a wait gave up
          auto new_reference = [&](float m_tile, bool over) {
            const float m_new = fmaxf(m_run, m_tile);
            const bool rescale = j > 0 && m_new > m_run + (over ? 0.f : kRescaleThreshold);
            if (j == 0) m_run = m_new;
            if (__any_sync(0xffffffffu, rescale)) {
              // O_h holds the tile before's P V: with as many buffers as slots these scores
              // prove it, else its completion is waited for (fwd_jobs.h)
              if (NSB > SLOTS && !warp_wait(&pv_done[h], (it + j - 1) & 1)) return false;
              tc_fence_after();
              const float f = rescale ? fast_exp2(m_run - m_new) : 1.f;
              l_run *= f;
              r_run *= f;
#pragma unroll 1
              for (int cb = 0; cb < D / 32; ++cb) {
                uint32_t orow[32];
                tmem_ld32(tO + cb * 32, orow);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) orow[e] = __float_as_uint(__uint_as_float(orow[e]) * f);
                tmem_st32(tO + cb * 32, orow);
              }
              if (rescale) m_run = m_new;
            }
            return true;
          };
          if constexpr (CAP)  // 32 columns at a time: 2K new tokens over 32K keys 1.22 ms for 1.18
            cap_tile<64>(tS, a.cap, valid, part, seen);
          // against the running maximum, and where some row's sum reaches the bound (or j is
          // 0) with the tile's own: two turns of one loop, a copy of the code less
          bool over = false;
#pragma unroll 1
          for (int turn = j == 0 ? 1 : 0; turn < 2; ++turn) {
            load_s();
            if (turn == 1 && !(ok = new_reference(tile_max(), over))) break;
            // the first turn: against a row's -inf so far, NaN or more than the bound
            const float2 ts = form_p(turn == 1 && m_run == -INFINITY ? 0.f : m_run);
            over = !(ts.x < kSumBound);
            if (turn == 1 || !__any_sync(0xffffffffu, over)) {
              l_run += ts.x;
              r_run += ts.y;
              break;
            }
          }
          if (!ok) break;
          tmem_st32(tS, pk[0]);
          tmem_st32(tS + 32, pk[1]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_p(lane == 0, &p_full[buf]);
      }
      it += n;
      J += SLOTS * n;
      if (!ok || !(ok = warp_wait(o_full, seg & 1))) break;
      if (!some) continue;
      tc_fence_after();
      // ------------------------------------------------------- the item's rows
      const int tok = sg.tok + h * a.per_slot + tl, head = sg.kvh * a.G + row - tl * a.G;
      if (sg.part < 0) {
        const float inv = r_run != 0.f ? 1.f / r_run : 0.f;
        __nv_bfloat16* orow = a.o + (static_cast<int64_t>(tok) * a.hq + head) * D;
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t ov[32];
          tmem_ld32(tO + cb * 32, ov);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16(__uint_as_float(ov[v4 * 8 + 2 * e]) * inv,
                                 __uint_as_float(ov[v4 * 8 + 2 * e + 1]) * inv);
              reinterpret_cast<uint4*>(orow + cb * 32)[v4] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (valid)
          a.lse[static_cast<int64_t>(head) * a.tokens + tok] =
              l_run != 0.f ? (m_run + log2f(l_run)) * kLn2 : -INFINITY;
        tc_fence_before();
        continue;
      }
      const int64_t part_row = static_cast<int64_t>(sg.part) * (SLOTS * kTile) + h * kTile + row;
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t ov[32];
        tmem_ld32(tO + cb * 32, ov);
        tmem_wait_ld();
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o + part_row * D + cb * 32);
#pragma unroll
          for (int v4 = 0; v4 < 8; ++v4)
            __stcg(dst + v4, make_uint4(ov[v4 * 4], ov[v4 * 4 + 1], ov[v4 * 4 + 2], ov[v4 * 4 + 3]));
        }
      }
      if (valid) __stcg(a.part_ml + part_row, make_float4(m_run, l_run, r_run, 0.f));
      tc_fence_before();
      __threadfence();
      __syncwarp();
      unsigned before = 0;
      if (lane == 0) before = atomicAdd(a.tickets + static_cast<int64_t>(sg.item) * C::SOFTMAX_WARPS + warp, 1u);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before != static_cast<unsigned>(sg.parts) - 1) continue;
      __threadfence();
      // ---- the last of the item's parts: join them, D / 4 lanes a row
      constexpr int LANES = D / 4;
      const int sub = lane / LANES, part4 = lane % LANES;
      auto row_of = [&](int p, int r) {  // row r of the warp in part p of the item
        const int64_t at = 2 * (sg.first_block + p) + (p == 0 ? sg.first_part : 0);
        return at * (SLOTS * kTile) + h * kTile + quarter * 32 + r;
      };
      const int rows = min(32, here - quarter * 32);
      for (int r0 = 0; r0 < rows; r0 += 32 / LANES) {
        const int r = r0 + sub;
        const bool live = r < rows;
        float mx = -INFINITY;
        if (live)
          for (int p = part4; p < sg.parts; p += LANES) mx = fmaxf(mx, __ldcg(a.part_ml + row_of(p, r)).x);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (!live) continue;  // no lane exchanges anything from here on
        const float ref = mx == -INFINITY ? 0.f : mx;
        float l = 0.f, rl = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int p = 0; p < sg.parts; ++p) {
          const int64_t at = row_of(p, r);
          const float4 ml = __ldcg(a.part_ml + at);
          const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D) + part4);
          if (ml.y != 0.f) {  // a part without keys of the row adds nothing
            const float w = fast_exp2(ml.x - ref);
            l = fmaf(w, ml.y, l);
            rl = fmaf(w, ml.z, rl);
            acc.x = fmaf(w, x.x, acc.x);
            acc.y = fmaf(w, x.y, acc.y);
            acc.z = fmaf(w, x.z, acc.z);
            acc.w = fmaf(w, x.w, acc.w);
          }
        }
        const int rr = quarter * 32 + r, t2 = rr / a.G;
        const int64_t tok2 = sg.tok + h * a.per_slot + t2;
        const int head2 = sg.kvh * a.G + rr - t2 * a.G;
        const float inv = rl != 0.f ? 1.f / rl : 0.f;
        reinterpret_cast<uint2*>(a.o + (tok2 * a.hq + head2) * D)[part4] =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (part4 == 0)
          a.lse[static_cast<int64_t>(head2) * a.tokens + tok2] = l != 0.f ? (mx + log2f(l)) * kLn2 : -INFINITY;
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::SOFTMAX_WARPS + 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// bf16 rows [rows][heads][d], `stride` elements from row to row, as (d, heads, rows)
// with a box of (64, box_heads, box_rows), 128-byte swizzle.
int make_rows_map(CUtensorMap* map, const void* base, int64_t rows, int heads, int d, int64_t stride, int box_heads,
                  int box_rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return LOONG_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LOONG_OK : cuda_fail(cudaErrorInvalidValue);
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

int check_paged(const loong_paged_desc* d) {
  if (!d) return LOONG_ERR_INVALID_ARG;
  if (d->batch < 1 || d->tokens < 0 || d->hq < 1 || d->hkv < 1 || d->hq % d->hkv || d->num_pages < 1 ||
      d->max_pages < 1 || d->window < 0 || d->page_size < 1)
    return LOONG_ERR_INVALID_ARG;
  const int64_t strides[3] = {d->q_stride, d->k_stride, d->v_stride};
  for (int i = 0; i < 3; ++i) {
    const int64_t row = static_cast<int64_t>(i ? d->hkv : d->hq) * d->head_dim;
    if (strides[i] && (strides[i] < row || strides[i] % 8 || strides[i] > (int64_t{1} << 31)))
      return LOONG_ERR_INVALID_ARG;
  }
  if (!std::isfinite(d->softmax_scale) || !std::isfinite(d->score_cap) || d->score_cap < 0.f)
    return LOONG_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return LOONG_ERR_UNSUPPORTED;
  if (d->page_size < 8 || d->page_size > 1024 || (d->page_size & (d->page_size - 1))) return LOONG_ERR_UNSUPPORTED;
  if (d->hq / d->hkv > kTile || d->batch > kMaxSequences) return LOONG_ERR_UNSUPPORTED;
  // rows of the pool and positions of a sequence are 32-bit coordinates, a tile and more past the last one included
  if ((static_cast<int64_t>(d->num_pages) + 1) * d->page_size > (1 << 30) ||
      static_cast<int64_t>(d->max_pages) * d->page_size > (1 << 30) || d->tokens > (1 << 30))
    return LOONG_ERR_UNSUPPORTED;
  return score_cap_fits(d->softmax_scale, d->score_cap) ? LOONG_OK : LOONG_ERR_UNSUPPORTED;
}

// Two slots of 128 rows share a tile of keys where the new tokens of a sequence fill
// more than one on the average.
int paged_slots(const loong_paged_desc& d) {
  const int64_t rows = static_cast<int64_t>(d.tokens) * (d.hq / d.hkv);
  return rows > static_cast<int64_t>(d.batch) * kTile ? 2 : 1;
}

struct PagedWs {
  int slots, per_slot, max_groups, blocks, tickets;
  size_t groups, prefix, count, ticket, part_o, part_ml, total;
};
PagedWs paged_ws(const loong_paged_desc& d) {
  PagedWs w{};
  w.slots = paged_slots(d);
  w.per_slot = kTile / (d.hq / d.hkv);
  w.max_groups = d.tokens / (w.slots * w.per_slot) + d.batch;
  w.blocks = 152;
  w.tickets = w.max_groups * d.hkv * 4 * w.slots;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  w.groups = take(sizeof(Group) * w.max_groups);
  w.prefix = take(4 * (static_cast<size_t>(w.max_groups) + 1));
  w.count = take(4);
  w.ticket = take(4 * static_cast<size_t>(w.tickets));
  const size_t rows = static_cast<size_t>(w.blocks) * 2 * w.slots * kTile;
  w.part_ml = take(rows * sizeof(float4));
  w.part_o = take(rows * d.head_dim * 4);
  w.total = at;
  return w;
}

// Units of work fit 32 bits, tickets too.
bool paged_fits(const loong_paged_desc& d) {
  const int64_t per_group = static_cast<int64_t>(paged_slots(d)) * (kTile / (d.hq / d.hkv));
  const int64_t groups = d.tokens / per_group + d.batch;
  const int64_t tiles = (static_cast<int64_t>(d.max_pages) * d.page_size + kTile - 1) / kTile + 1 + kItemUnits;
  return groups * tiles < (int64_t{1} << 31) && groups * d.hkv * 8 < (int64_t{1} << 31);
}

template <int D, int SLOTS, bool CAP>
int launch_paged(const loong_paged_desc& d, const PagedArgs& a, const AppendArgs& n, const void* q, const void* k_pages,
                 const void* v_pages, cudaStream_t stream) {
  using C = PagedCfg<D, SLOTS>;
  CUtensorMap mq, mk, mv;
  int st;
  const int64_t q_stride = d.q_stride ? d.q_stride : static_cast<int64_t>(d.hq) * D;
  const int64_t rows = static_cast<int64_t>(d.num_pages) * d.page_size, kv_stride = static_cast<int64_t>(d.hkv) * D;
  const int box = std::min(d.page_size, kTile);
  if ((st = make_rows_map(&mq, q, d.tokens, d.hq, D, q_stride, a.G, a.per_slot)) != LOONG_OK ||
      (st = make_rows_map(&mk, k_pages, rows, d.hkv, D, kv_stride, 1, box)) != LOONG_OK ||
      (st = make_rows_map(&mv, v_pages, rows, d.hkv, D, kv_stride, 1, box)) != LOONG_OK)
    return st;
  const int sms = std::min(num_sms(), 152);
  const int copy_blocks = n.k ? std::min((d.tokens + kPrepThreads / 32 - 1) / (kPrepThreads / 32), 2 * sms) : 0;
  paged_prep_kernel<<<1 + copy_blocks, kPrepThreads, 0, stream>>>(a, n, SLOTS * a.per_slot);
  if ((st = check_launch()) != LOONG_OK) return st;
  constexpr auto kern = paged_attn_kernel<D, SLOTS, CAP>;
  if ((st = kernel_ready<kern>(C::SMEM_BYTES, C::SPLIT ? C::SPLIT_REGS : 0)) != LOONG_OK) return st;
  return launch_dependent(kern, dim3(sms), C::THREADS, C::SMEM_BYTES, stream, mq, mk, mv, a);
}

}  // namespace

}  // namespace loong

using namespace loong;

extern "C" {

int loong_paged_check(const loong_paged_desc* d) {
  const int st = check_paged(d);
  return st != LOONG_OK ? st : paged_fits(*d) ? LOONG_OK : LOONG_ERR_UNSUPPORTED;
}

size_t loong_paged_attn_workspace_size(const loong_paged_desc* d) {
  return loong_paged_check(d) == LOONG_OK ? paged_ws(*d).total : 0;
}

int loong_paged_attn(const loong_paged_desc* d, const void* q, const void* k, const void* v, void* k_pages,
                     void* v_pages, const int32_t* table, const int32_t* lens, const int32_t* starts, void* o,
                     float* lse, void* ws, size_t ws_bytes, loong_stream_t stream_) {
  NvtxRange range("loong_paged_attn");
  int st = loong_paged_check(d);
  if (st != LOONG_OK) return st;
  if ((k == nullptr) != (v == nullptr)) return LOONG_ERR_INVALID_ARG;
  if (d->tokens == 0) return LOONG_OK;
  const void* ptrs[] = {q, k_pages, v_pages, o};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 16)) return LOONG_ERR_INVALID_ARG;
  const void* words[] = {table, lens, starts, lse};
  for (const void* p : words)
    if (!p || !aligned(p, 4)) return LOONG_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return LOONG_ERR_INVALID_ARG;
  const PagedWs w = paged_ws(*d);
  if (!ws || ws_bytes < w.total || !aligned(ws, 16)) return LOONG_ERR_WORKSPACE;
  if ((st = device_ready()) != LOONG_OK) return st;
  for (const void* p : ptrs)
    if (!on_device(p)) return LOONG_ERR_INVALID_ARG;
  for (const void* p : words)
    if (!on_device(p)) return LOONG_ERR_INVALID_ARG;
  if (!on_device(ws) || (k && (!on_device(k) || !on_device(v)))) return LOONG_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  PagedArgs a;
  a.batch = d->batch;
  a.tokens = d->tokens;
  a.hq = d->hq;
  a.hkv = d->hkv;
  a.G = d->hq / d->hkv;
  a.per_slot = w.per_slot;
  a.page_log2 = log2_of(d->page_size);
  a.num_pages = d->num_pages;
  a.max_pages = d->max_pages;
  a.window = window_within(d->window, static_cast<int64_t>(d->max_pages) * d->page_size);
  a.max_groups = w.max_groups;
  const float scale =
      d->softmax_scale > 0.f ? d->softmax_scale : 1.0f / std::sqrt(static_cast<float>(d->head_dim));
  a.cap = make_score_cap(scale, d->score_cap);
  a.scale_log2 = scale * kLog2e;
  a.table = table;
  a.lens = lens;
  a.starts = starts;
  a.groups = reinterpret_cast<Group*>(base + w.groups);
  a.prefix = reinterpret_cast<int*>(base + w.prefix);
  a.count = reinterpret_cast<int*>(base + w.count);
  a.tickets = reinterpret_cast<unsigned*>(base + w.ticket);
  a.part_o = reinterpret_cast<float*>(base + w.part_o);
  a.part_ml = reinterpret_cast<float4*>(base + w.part_ml);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  if (!(a.err = device_error_word())) return LOONG_ERR_CUDA;
  AppendArgs n;
  n.k = static_cast<const uint4*>(k);
  n.v = static_cast<const uint4*>(v);
  n.k_pages = static_cast<uint4*>(k_pages);
  n.v_pages = static_cast<uint4*>(v_pages);
  n.row_vecs = d->hkv * d->head_dim / 8;
  n.k_stride = d->k_stride ? d->k_stride / 8 : n.row_vecs;
  n.v_stride = d->v_stride ? d->v_stride / 8 : n.row_vecs;
  n.tickets = w.tickets;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  auto launch = [&](auto dim, auto slots) {
    constexpr int D = decltype(dim)::value, SLOTS = decltype(slots)::value;
    return d->score_cap > 0.f ? launch_paged<D, SLOTS, true>(*d, a, n, q, k_pages, v_pages, stream)
                              : launch_paged<D, SLOTS, false>(*d, a, n, q, k_pages, v_pages, stream);
  };
  using std::integral_constant;
  if (d->head_dim == 128)
    return w.slots == 2 ? launch(integral_constant<int, 128>{}, integral_constant<int, 2>{})
                        : launch(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  return w.slots == 2 ? launch(integral_constant<int, 64>{}, integral_constant<int, 2>{})
                      : launch(integral_constant<int, 64>{}, integral_constant<int, 1>{});
}

}  // extern "C"
