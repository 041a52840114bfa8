// paged_plan.h -- how a batch's new tokens become groups (paged_attn.cu): the arithmetic
// of the plan, whose arrays are the caller's and may hold anything.
#pragma once

#include <stdint.h>

#include "ring.cuh"

namespace loong {

// New tokens [tok, tok + count) of sequence `seq`, the first at position pos; key
// tiles [tile, tile + tiles) hold what they see.
struct Group {
  int seq, tok, count, pos, tile, tiles, pad0, pad1;
};

// A sequence's new tokens and its length with them, in the arrays' bounds; not fine
// where they had to be cut.
struct SequenceCut {
  int tok, count, len;
  bool fine;
};
__host__ __device__ inline SequenceCut cut_sequence(int s0, int s1, int length, int tokens, int64_t room) {
  auto within = [](int64_t x, int64_t most) { return static_cast<int>(x < 0 ? 0 : x < most ? x : most); };
  SequenceCut c;
  c.tok = within(s0, tokens);
  const int end = within(s1, tokens);
  c.count = end > c.tok ? end - c.tok : 0;
  c.len = within(length, room);
  c.fine = c.tok == s0 && c.count == static_cast<int64_t>(s1) - s0 && c.len == length && c.count <= c.len;
  return c;
}

__host__ __device__ inline int groups_of(int count, int per_group) { return (count + per_group - 1) / per_group; }

// Starts that fall share tokens among sequences: 4096 of them with 2^30 tokens each
// pass 32 bits, so the groups are added up in 64 before they are cut to those that
// there is room for.
using GroupSum = int64_t;
__host__ __device__ inline int cut_groups(GroupSum groups, int max_groups) {
  return static_cast<int>(groups < max_groups ? groups : max_groups);
}

// The sequence of group g: the last one of `batch` whose first group is at or before it.
__host__ __device__ inline int sequence_of_group(const int* first, int batch, int g) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first[mid] <= g)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// A window as wide as a sequence may be leaves every key, like none (0), and positions less
// such a window stay within 32 bits.
__host__ __device__ inline int window_within(int window, int64_t room) { return window < room ? window : 0; }

// The group that begins `off` tokens into the sequence's new ones.
__host__ __device__ inline Group make_group(const SequenceCut& c, int seq, int off, int per_group, int window) {
  Group r;
  r.seq = seq;
  r.tok = c.tok + off;
  r.count = c.count - off < per_group ? c.count - off : per_group;
  r.pos = c.len - c.count + off;
  const int to = r.pos + r.count > 0 ? r.pos + r.count : 0;
  const int from = window && r.pos - window + 1 > 0 ? r.pos - window + 1 : 0;  // window: of window_within
  r.tile = from / kTile;
  const int tiles = (to + kTile - 1) / kTile - r.tile;
  r.tiles = tiles > 1 ? tiles : 1;  // where nothing is seen that has to be stored
  r.pad0 = r.pad1 = 0;
  return r;
}

}  // namespace loong
