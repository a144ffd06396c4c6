// Host-side launchers of the selective state space layer (conv.hip, sscan.hip).
// Each returns the hipError_t of its launches; arguments are validated by the
// API layer before any call.
#pragma once

#include "launch.hpp"

namespace swimba {

// ---- causal convolution
struct ConvArgs {
  const void* x;  // rows ldx apart
  int64_t ldx;
  const void *w, *bias;  // [C, W]; [C] or null
  const int32_t* lens;   // [Bt] or null
  const void* state_in;  // [Bt, W - 1, C] or null
  void *y, *state_out;   // state_out may be null
  // backward
  const void* dy;
  const float* dstate_out;
  void* dx;
  int64_t lddx;
  float *dw, *db, *dstate_in;
  float* part;  // [runs][W + 1][C]
  int Bt, T, C, W;
  int silu;
  int run;  // tokens per thread
};
size_t conv_bwd_ws_bytes(int Bt, int T, int C);  // for any width
hipError_t launch_conv(bool is_bf16, const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_backward(bool is_bf16, const ConvArgs& a, hipStream_t s);
// No tokens: to = from (or zeros), n elements.
hipError_t launch_conv_state(bool is_bf16, const void* from, void* to, size_t n, hipStream_t s);
hipError_t launch_conv_step(bool is_bf16, const ConvArgs& a, hipStream_t s);

// ---- selective scan
constexpr int kScanMaxN = 128;
struct SScanArgs {
  const void *x, *dt, *z;  // rows ldx, lddt, ldz apart; z may be null
  int64_t ldx, lddt, ldz;
  const void *B, *C;
  int64_t ldbc;
  const float *A, *D, *bias;  // D and bias may be null
  const int32_t* lens;
  const float* h_init;
  void* y;
  float* h_final;
  float* carry;
  // backward
  const float* carry_in;
  const void* dy;
  const float* dh_final;
  void *dx, *ddt, *dz;
  int64_t lddx, ldddt, lddz;
  void *dB, *dC;
  int64_t lddbc;
  float *dA, *dD, *dbias, *dh_init;
  // one token
  const float* h_prev;
  float* h;
  void* ws;
  int Bt, T, Ch, N, G;
  int segs;  // runs of blocks of tokens that a sequence is cut into
};
size_t sscan_carry_bytes(int Bt, int T, int Ch, int N);
size_t sscan_ws_bytes(int Bt, int T, int Ch, int N, int G);
size_t sscan_bwd_ws_bytes(int Bt, int T, int Ch, int N, int G);
int64_t sscan_threads(int64_t Bt, int64_t T, int64_t Ch, int64_t N, int64_t G);  // of the largest launch
hipError_t launch_sscan(bool is_bf16, const SScanArgs& a, hipStream_t s);
hipError_t launch_sscan_backward(bool is_bf16, const SScanArgs& a, hipStream_t s);
hipError_t launch_sscan_step(bool is_bf16, const SScanArgs& a, hipStream_t s);

}  // namespace swimba
