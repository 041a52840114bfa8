// Host check of the paged attention's plan (paged_plan.h), the kernel's steps one after
// the other: every new token of a well-formed batch is in one group, whose tiles hold
// what its tokens see; and whatever starts and lengths hold, the groups stay within the
// workspace's and their tokens within the arrays.  Compiled by
// tests/test_mask_paged_corrections.py.
#include <cstdio>
#include <random>
#include <vector>

#define __host__
#define __device__
#include "paged_plan.h"

using namespace loong;

static long bad = 0, checked = 0;
static void hold(bool x) {
  ++checked;
  bad += !x;
}

// What block 0 of the first launch does; false where it reports.
static bool plan(const std::vector<int>& starts, const std::vector<int>& lens, int tokens, int64_t room, int per_group,
                 int max_groups, int window, std::vector<Group>& groups, size_t keep) {
  const int batch = static_cast<int>(lens.size());
  std::vector<int> first(batch);
  GroupSum sum = 0;
  bool fine = true;
  for (int b = 0; b < batch; ++b) {
    const SequenceCut c = cut_sequence(starts[b], starts[b + 1], lens[b], tokens, room);
    fine &= c.fine;
    hold(c.tok >= 0 && c.count >= 0 && c.tok + c.count <= tokens && c.len >= 0 && c.len <= room);
    first[b] = cut_groups(sum, max_groups);
    hold(first[b] >= 0 && (b == 0 || first[b] >= first[b - 1]));
    sum += groups_of(c.count, per_group);
  }
  fine &= sum <= max_groups;
  const int base = cut_groups(sum, max_groups);
  hold(base >= 0 && base <= max_groups);
  groups.clear();
  // all of them, or as many from either end
  for (int g = 0; g < base; ++g) {
    if (static_cast<size_t>(g) >= keep && static_cast<size_t>(base - g) > keep) continue;
    const int b = sequence_of_group(first.data(), batch, g);
    hold(b >= 0 && b < batch);
    const SequenceCut c = cut_sequence(starts[b], starts[b + 1], lens[b], tokens, room);
    const Group r = make_group(c, b, (g - first[b]) * per_group, per_group, window);
    hold(r.count >= 1 && r.count <= per_group && r.tok >= c.tok && r.tok + r.count <= c.tok + c.count);
    hold(r.pos + r.count <= c.len && r.tile >= 0 && r.tiles >= 1);
    hold(static_cast<int64_t>(r.tile + r.tiles - 1) * kTile < room + kTile);
    groups.push_back(r);
  }
  return fine;
}

int main() {
  std::mt19937_64 rng(1);
  auto below = [&](int64_t n) { return static_cast<int64_t>(rng() % static_cast<uint64_t>(n)); };
  std::vector<Group> groups;
  for (int round = 0; round < 2000; ++round) {  // well-formed batches
    const int batch = static_cast<int>(1 + below(9)), per_group = static_cast<int>(1 + below(256));
    const int64_t room = 8 + below(3000);
    const int window = below(2) ? static_cast<int>(1 + below(2 * room)) : 0;
    std::vector<int> starts(batch + 1), lens(batch);
    starts[0] = static_cast<int>(below(3));
    for (int b = 0; b < batch; ++b) {
      lens[b] = static_cast<int>(below(room + 1));
      starts[b + 1] = starts[b] + static_cast<int>(below(lens[b] + 1));
    }
    const int tokens = starts[batch] + static_cast<int>(below(3)), max_groups = tokens / per_group + batch;
    hold(plan(starts, lens, tokens, room, per_group, max_groups, window, groups, ~size_t{0}));
    std::vector<int> seen(tokens);
    for (const Group& r : groups)
      for (int i = 0; i < r.count; ++i) {
        ++seen[r.tok + i];
        const int pos = r.pos + i;
        hold(pos == lens[r.seq] - (starts[r.seq + 1] - starts[r.seq]) + r.tok + i - starts[r.seq]);
        const int64_t from = window && pos - window + 1 > 0 ? pos - window + 1 : 0;
        hold(int64_t{r.tile} * kTile <= from && pos < int64_t{r.tile + r.tiles} * kTile);
      }
    for (int t = 0; t < tokens; ++t) hold(seen[t] == (t >= starts[0] && t < starts[batch]));
  }
  for (int round = 0; round < 2000; ++round) {  // anything
    const int batch = static_cast<int>(1 + below(9)), per_group = static_cast<int>(1 + below(256));
    const int tokens = static_cast<int>(below(2000)), max_groups = tokens / per_group + batch;
    auto any = [&]() {
      const int64_t v[] = {below(2100), below(2100), -below(100), int64_t{1} << 31, -(int64_t{1} << 31), below(1ll << 32)};
      return static_cast<int>(v[below(6)]);
    };
    std::vector<int> starts(batch + 1), lens(batch);
    for (int& x : starts) x = any();
    for (int& x : lens) x = any();
    plan(starts, lens, tokens, 8 + below(3000), per_group, max_groups, below(2) ? static_cast<int>(1 + below(3000)) : 0,
         groups, ~size_t{0});
  }
  // starts that go up and down between 0 and many tokens: the sum passes 32 bits
  for (const int tokens : {1 << 21, (1 << 22) + 3, 1 << 30}) {
    std::vector<int> starts(4097), lens(4096);
    for (int b = 0; b < 4097; ++b) starts[b] = b & 1 ? tokens : 0;
    const int per_group = 2, max_groups = tokens / per_group + 4096;
    hold(!plan(starts, lens, tokens, 1 << 20, per_group, max_groups, 0, groups, 1000));
  }
  // a window of any size, up to the largest number, where tokens stand before position 0
  for (const int64_t wide : {int64_t{300}, int64_t{1} << 30, (int64_t{1} << 31) - 6, (int64_t{1} << 31) - 1})
    for (int len = 0; len < 300; len += 7) {
      const int64_t room = 4096;
      const std::vector<int> starts{0, 200}, lens{len};
      plan(starts, lens, 200, room, 32, 8, window_within(static_cast<int>(wide), room), groups, ~size_t{0});
      hold(groups.size() == 7);
      for (const Group& r : groups)
        for (int i = 0; i < r.count; ++i) {
          const int64_t pos = r.pos + i, from = pos - wide + 1 > 0 ? pos - wide + 1 : 0;
          hold(pos == len - 200 + r.tok + i);
          if (pos >= 0) hold(int64_t{r.tile} * kTile <= from && pos < int64_t{r.tile + r.tiles} * kTile);
        }
    }
  std::printf("%ld checks, %ld failed\n", checked, bad);
  return bad ? 1 : 0;
}
