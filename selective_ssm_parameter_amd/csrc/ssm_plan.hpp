// How the convolution (conv.hip) and one token of the selective scan (sscan.hip) divide
// their work among threads. Host code without HIP, so that a test can ask it which form
// a shape reaches.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace swimba {

constexpr int kStep = 8;     // rows in flight per thread of the convolution
constexpr int kStepBwd = 4;  // the same of the backward, of x and of dy

// Tokens per thread: long runs read few rows twice and leave few partial sums, as
// long as enough threads remain to fill the card, some 2^18 forward (8 x 2048 x
// 1536: 20 us; 2^17: 23, 2^19: 22) and, for the partial sums, 2^17 backward (36 us with
// their addition; 2^16: 43, 2^18: 34 but slower in float32, 2^19: 51).
constexpr int kFwdThreads = 18, kBwdThreads = 17;
inline int run_length(int64_t Bt, int64_t T, int64_t vecs, int threads) {
  const int64_t r = Bt * T * vecs >> threads;
  return (int)std::min<int64_t>(256, std::max<int64_t>(kStep, r / kStep * kStep));
}
// Channels per thread: v, where rows allow it.
inline int vec_of(int v, int C, int64_t ldx, int64_t lddx) {
  return C % v == 0 && ldx % v == 0 && lddx % v == 0 ? v : 1;
}
// 16 bytes of them forward; 8 in the backward, whose registers then leave room for
// three waves instead of one (padded 8 x 2048 x 1536: 78 -> 40 us when it was measured;
// 4 bytes: 54, now 32 against 31).
inline int vec_fwd(bool is_bf16) { return is_bf16 ? 8 : 4; }
inline int vec_bwd(bool is_bf16) { return is_bf16 ? 4 : 2; }

// Sequences per thread of one token of the scan: two where that leaves threads enough to
// fill the card (256 x 4096 x 16: 34 us; one: 39, four: 38, eight: 56).
inline int step_sequences(int64_t Bt, int64_t Ch) { return Bt * Ch >= int64_t(1) << 18 ? 2 : 1; }

}  // namespace swimba
