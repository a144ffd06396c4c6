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
// long as enough threads remain to fill the card, some 2^18 forward and, for the partial
// sums, 2^17 backward. With half as many threads, these and twice as many, bf16, us:
// forward 8 x 2048 x 1536 24.1, 20.1, 19.9, 4 x 8192 x 4096 104.5, 100.8, 101.2, 64 x 512 x
// 1024 23.9, 24.4, 26.3, 65536 x 2048 107, 105, 105; forward and backward 80.3, 68.1, 69.4
// (fp32 151, 116, 113), 266, 265, 279, 85.4, 80.9, 86.0 and 263, 263, 283.
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
// fill the card. With one and with two, 16 states, us: 32 and 64 x 4096 10.5 and 10.5 (the
// call's host time), 128 x 4096 16.0, 14.9, 256 x 4096 28.8, 25.1, 512 x 4096 73.8, 64.3. (Four
// and eight were slower than one.)
inline int step_sequences(int64_t Bt, int64_t Ch) { return Bt * Ch >= int64_t(1) << 18 ? 2 : 1; }

}  // namespace swimba
