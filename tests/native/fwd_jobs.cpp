// Host check of the forward's score buffers: the order in which its MMA warp
// issues Q K^T and P V is written out, and for every tile of every slot the
// P V products that its scores prove done (those issued before them) must
// include the one two tiles back, which the wait before a rescale builds on.
// Compiled by tests/test_fwd_jobs.py with the host compiler.
#include <cstdio>
#include <vector>

#include "fwd_jobs.h"

int main() {
  int bad = 0, checked = 0;
  for (int d : {64, 128})
    for (int slots : {1, 2}) {
      const int buffers = loong::fwd_score_buffers(d, slots);
      if (buffers < 2 || buffers * 128 + 2 * d > 512) {
        std::printf("d %d, %d slots: %d buffers\n", d, slots, buffers);
        ++bad;
      }
      for (int tiles = 1; tiles <= 12; ++tiles) {
        const int jobs = slots * tiles;
        std::vector<int> qk_at(jobs), pv_at(jobs);
        int at = 0;
        for (int J = 0; J < buffers && J < jobs; ++J) qk_at[J] = at++;
        for (int J = 0; J < jobs; ++J) {
          pv_at[J] = at++;
          if (J + buffers < jobs) qk_at[J + buffers] = at++;
        }
        for (int J = 2 * slots; J < jobs; ++J, ++checked)
          if (pv_at[J - 2 * slots] > qk_at[J] && bad++ < 10)
            std::printf("d %d, %d slots, %d tiles: scores of job %d do not wait for P V of job %d\n", d, slots, tiles, J,
                        J - 2 * slots);
      }
    }
  // one slot per block only where the device runs all blocks in one round
  for (int sms : {1, 76, 132, 148, 152, 160})
    if (!loong::fwd_one_slot(sms, sms) || loong::fwd_one_slot(sms + 1, sms)) {
      std::printf("%d SMs: the rule for one slot does not follow them\n", sms);
      ++bad;
    }
  std::printf("%d jobs checked, %d open\n", checked, bad);
  return bad ? 1 : 0;
}
