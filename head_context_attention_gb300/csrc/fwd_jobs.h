// fwd_jobs.h -- the forward kernel's query slots per block and score buffers.
//
// How many buffers, by what the order of its matrix instructions lets the softmax
// conclude.
//
// Job J = slots * j + h is key tile j of query slot h.  The MMA warp issues Q K^T
// of the first jobs, one per buffer, then P V of job J and Q K^T of job
// J + buffers in turn; they execute in that order.  Scores of job J therefore
// show that P V of jobs up to J - buffers is done, and no more.  A softmax that
// rescales O_h waits for P V of its previous tile, job J - slots, on a barrier
// with one phase per tile of the slot.  A wait tells a phase from the one before
// by one bit, so the phase before (job J - 2 slots) has to be known as done, or
// the wait passes while both are under way and O_h is read, scaled and stored
// under them: J - buffers >= J - 2 slots.  (One slot with three buffers and a wait
// on every tile instead: 4K tokens of 4 heads of 64 41.0 us for 38.9.)
#pragma once

namespace loong {

// What tensor memory has room for: two slots' O and this many buffers of 128
// columns in 512.
constexpr int fwd_max_score_buffers(int head_dim) { return head_dim == 64 ? 3 : 2; }

constexpr int fwd_score_buffers(int head_dim, int slots) {
  const int room = fwd_max_score_buffers(head_dim);
  return room < 2 * slots ? room : 2 * slots;
}

// With a bias or a mask, blocks of one slot where `tiles` query tiles of single heads find an
// SM each: a block takes two thirds of a two-slot block's time, so they pay in one
// round only.  One and two slots, 4K tokens of 4 heads of 128 (128 and 64 blocks)
// 43.0 and 65.5 us, of 64 38.9 and 49.0, 2K of 8 + 2 heads of 64 26.6 and 31.0, 512
// of 4 of 128 18.5 and 24.6; 16 heads twice 4K (1,024 and 512 blocks) would take
// seven rounds for four.
constexpr bool fwd_one_slot(long long tiles, int sms) { return tiles <= sms; }

}  // namespace loong
