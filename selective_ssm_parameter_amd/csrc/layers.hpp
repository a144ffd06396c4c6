// Host-side launchers of the layer kernels (norm.hip, gscan.hip, dense.hip).
// Each returns the hipError_t of its launches; arguments are validated by the
// API layer before any call.
#pragma once

#include "launch.hpp"

namespace swimba {

// ---- layer norm
struct NormFwdArgs {
  const void *x, *residual, *weight, *bias;
  float eps;
  void *sum, *y;
  float *mean, *rstd;
  int M, D;
};
struct NormBwdArgs {
  const void *s, *weight;
  const float *mean, *rstd;
  const void* dy;
  const float* dres;
  float *dx, *dw, *db;
  float* part;  // [norm_bwd_parts(M, D)][2][D]
  int M, D;
};
constexpr int kNormMaxD = 32768;  // a row is held in the registers of 1024 threads
int norm_bwd_parts(int M, int D);
int64_t norm_fwd_threads(int64_t M, int D);  // of the forward's launch
hipError_t launch_norm_fwd(bool is_bf16, const NormFwdArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(bool is_bf16, bool dy_f32, const NormBwdArgs& a, hipStream_t s);

// ---- gated scan
struct GScanArgs {
  const void *x, *f, *o;  // rows ld elements apart; o may be null
  int64_t ld;
  const int32_t* lens;  // [Bt] or null
  const float* h_init;  // [Bt, C] or null
  void* y;              // [M, C]
  float* h_final;       // [Bt, C] or null
  float* carry;         // [Bt, chunks, C] or null: the state entering each chunk
  // backward
  const float* carry_in;
  const void* dy;
  const float* dh_final;
  void *dx, *df, *d_o;
  int64_t ldd;
  float* dh_init;
  void* ws;
  int Bt, T, C;
};
int gscan_chunks(int T);  // chunks of tokens per sequence
int64_t gscan_blocks(int64_t Bt, int64_t T, int64_t C);  // workgroups of a pass
size_t gscan_ws_bytes(int Bt, int T, int C);
hipError_t launch_gscan(bool is_bf16, const GScanArgs& a, hipStream_t s);
hipError_t launch_gscan_backward(bool is_bf16, const GScanArgs& a, hipStream_t s);
hipError_t launch_gscan_step(bool is_bf16, const void* x, const void* f, const void* o, int64_t ld,
                             const float* h_prev, float* h, void* y, int Bt, int C,
                             hipStream_t s);

// ---- dense products of the feed-forward and output projections
// h = act(g) u, [g | u] = x w_in^T; z may be null.
hipError_t launch_gated_project(bool is_bf16, int M, int D, int F, int act, const void* x,
                                const void* w_in, void* z, void* h, hipStream_t s);
// dz = [dh u act'(g) | dh act(g)] [M, 2F], g and u recomputed from x and w_in:
// float32, or for bf16 problems hi [M, 2F] and then lo [M, 2F], dz = hi + lo.
size_t gated_dz_bytes(bool is_bf16, int M, int F);
hipError_t launch_gated_dz(bool is_bf16, int M, int D, int F, int act, const void* x,
                           const void* w_in, const void* dh, void* dz, hipStream_t s);
// Partial sums of a product that runs its k in pieces (ws below): out [R, S] of
// K terms; tn: a weight gradient; split: with a_lo.
size_t dense_ws_bytes(bool is_bf16, bool split, bool tn, int R, int S, int K);
// out [M, S] = a [M, K] b [K, S]; with a_lo (bf16 problems) a is a + a_lo and
// out is float32, else out has the input type.
hipError_t launch_dense_nn(bool is_bf16, const char* name, int M, int K, int S, const void* a,
                           const void* a_lo, const void* b, void* out, void* ws, hipStream_t s);
// out [R, S] (float32) = (a + a_lo)^T b over M rows: a, a_lo [M, R] (a_lo may
// be null), b [M, S].
hipError_t launch_dense_tn(bool is_bf16, const char* name, int M, int R, int S, const void* a,
                           const void* a_lo, const void* b, float* out, void* ws, hipStream_t s);

}  // namespace swimba
