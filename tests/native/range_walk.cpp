// Host check of the masked forward's walk (RangeWalk in ring.cuh): over the whole
// ring, and over all single ring steps together, it visits every key tile that holds a
// key of the range once and no other, and total() is the number it visits.  Compiled
// by tests/test_range_walk.py.
#include <cstdio>
#include <vector>

#define __host__
#define __device__
#include "ring.cuh"

using namespace loong;

int main() {
  // cp = inner * outer, zigzag, tokens per block
  const int geoms[][4] = {{1, 1, 1, 384}, {4, 2, 1, 200}, {6, 3, 0, 250}, {4, 4, 1, 300},
                          {8, 2, 0, 128}, {2, 1, 1, 16},  {1, 1, 0, 1},   {3, 3, 0, 129}};
  long bad = 0, checked = 0;
  for (const auto& q : geoms) {
    RingGeom g;
    g.cp = q[0];
    g.inner = q[1];
    g.outer = q[0] / q[1];
    g.zigzag = q[2];
    g.causal = 0;
    g.blk = q[3];
    g.nblocks = g.zigzag ? 2 * g.cp : g.cp;
    g.ntile = (g.blk + kTile - 1) / kTile;
    const int S = g.nblocks * g.blk;
    for (int lo = 0; lo <= S; lo += (lo % 3 ? 1 : 37))
      for (int hi = 0; hi <= S; hi += (hi % 5 ? 1 : 53)) {
        std::vector<int> want(g.nblocks * g.ntile, 0);
        for (int b = 0; b < g.nblocks; ++b)
          for (int t = 0; t < g.ntile; ++t) {
            const int k0 = b * g.blk + t * kTile;
            const int k1 = k0 + kTile < (b + 1) * g.blk ? k0 + kTile : (b + 1) * g.blk;
            want[b * g.ntile + t] = lo < hi && k0 < hi && k1 > lo;
          }
        for (int c = 0; c < g.cp; c += (g.cp > 1 ? g.cp - 1 : 1))
          for (int whole = 0; whole < 2; ++whole) {
            std::vector<int> seen(want.size(), 0);
            for (int t = 0; t < (whole ? 1 : g.cp); ++t) {
              RangeWalk w;
              w.init(g, c, whole ? 0 : t, whole ? g.cp : t + 1, lo, hi);
              const int n = w.total();
              for (int i = 0; i < n; ++i, w.advance()) {
                const int b = w.k0() / g.blk, kt = (w.k0() - b * g.blk) / kTile;
                ++seen[b * g.ntile + kt];
              }
              ++checked;
            }
            if (seen != want && bad++ < 5)
              std::printf("cp=%d blk=%d zz=%d [%d,%d) rank %d whole %d differs\n", g.cp, g.blk, g.zigzag, lo, hi, c, whole);
          }
      }
  }
  std::printf("%ld walks checked, %ld mismatches\n", checked, bad);
  return bad ? 1 : 0;
}
