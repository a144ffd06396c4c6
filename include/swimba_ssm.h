/*
 * swimba_ssm.h - C ABI of the selective state space layer and its loss on
 * MI355X.
 *
 * The pages put the mixer into a hybrid stack of state space, attention and
 * feed-forward layers and fine-tune router and experts with the cross entropy
 * of next tokens (papernotes.org notes, Experiments). The scans of swimba.h
 * hold one decay per head; these calls are the layer with a decay of its own
 * per channel, state and token - the short causal convolution and the
 * selective scan, each for prompts, training and single tokens - and the cross
 * entropy over a vocabulary, with the gradients that enter the stack. The
 * layer itself is not on the pages: it is a neighbour of the mixer's scans.
 *
 * The conventions are those of swimba.h (device pointers, dense row-major
 * tensors unless a row stride is an argument, 16-byte alignment, caller-owned
 * workspaces, work on the given stream only, arguments validated before any
 * launch, bitwise repeatable results, swimba_last_error()). Sizes come from
 * swimba_dims:
 *   M = batch * seqlen tokens, C = nheads * headdim channels, N = dstate,
 *   G = ngroups (consecutive blocks of C / G channels), D = d_model,
 *   V = nheads * headdim rows of the vocabulary (cross entropy), dtype.
 * The other fields must be valid for swimba.h (1 will do) and are not used.
 * "dtype" below is the element type of activations and weights; sums, states,
 * decays and the gradients of weights and states are float32.
 * Row strides are elements from one row to the next; each is at least the row
 * and below 2^22.
 *   seq_lens  [batch] int32, or NULL: tokens of each sequence that are in use
 *             (a value outside [0, seqlen] counts as the nearest bound). Past
 *             them no input is looked at (they may hold anything), outputs per
 *             token are zeros, and the state is the one behind the last token
 *             in use.
 * An output must not overlap an input or another output unless the call says
 * that it may. Calls on one device that share a workspace, a state or an
 * output must be ordered by the caller.
 */
#ifndef SWIMBA_SSM_H
#define SWIMBA_SSM_H

#include "swimba.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum swimba_conv_act {
  SWIMBA_CONV_LINEAR = 0, /* the sum as it is */
  SWIMBA_CONV_SILU = 1    /* s sigmoid(s) */
} swimba_conv_act;

typedef enum swimba_ssm_call {
  SWIMBA_SSM_CONV_BACKWARD = 0,
  SWIMBA_SSM_SCAN = 1,
  SWIMBA_SSM_SCAN_BACKWARD = 2,
  SWIMBA_SSM_CROSS_ENTROPY = 3,
  SWIMBA_SSM_CROSS_ENTROPY_BACKWARD = 4
} swimba_ssm_call;

/* Workspace bytes that call `call` needs for `dims` (0 if none, and 0 for
 * invalid dims; the call itself then reports the error). Calls not in the
 * list need none. */
size_t swimba_ssm_workspace_size(const swimba_dims* dims, int32_t call);

/*
 * Causal convolution over the tokens of each channel:
 *   s_t = bias + sum_{k < width} weight[k] x_{t - width + 1 + k},   y_t = act(s_t),
 * x before the first token from state_in. Sums are float32.
 *   width     2, 3 or 4 (else SWIMBA_ERR_UNSUPPORTED)
 *   x         [M, C] dtype, rows ldx apart
 *   weight    [C, width] dtype;  bias [C] dtype, or NULL for zeros
 *   act       swimba_conv_act
 *   state_in  [batch, width - 1, C] dtype: the inputs before the first token,
 *             the oldest first; or NULL for zeros
 *   y         [M, C] dtype out
 *   state_out [batch, width - 1, C] dtype out, or NULL: the last width - 1
 *             inputs (of state_in where there are fewer tokens)
 */
swimba_status swimba_causal_conv(const swimba_dims* dims, int32_t width, const void* x,
                                 int64_t ldx, const void* weight, const void* bias, int32_t act,
                                 const int32_t* seq_lens, const void* state_in, void* y,
                                 void* state_out, hipStream_t stream);

/*
 * Backward of swimba_causal_conv. With ds_t = dy_t act'(s_t), s recomputed:
 *   dx_t = sum_k weight[k] ds_{t + width - 1 - k},   dweight[k] = sum_t ds_t x_{t - width + 1 + k},
 *   dbias = sum_t ds_t.
 * The sums over tokens run in a fixed order.
 *   x, ldx, weight, bias, act, seq_lens, state_in   as given to the forward
 *   dy        [M, C] dtype
 *   dstate_out [batch, width - 1, C] float32: gradient of state_out, or NULL
 *   dx        [M, C] dtype out, rows lddx apart
 *   dweight   [C, width] float32 out;  dbias [C] float32 out, or NULL (zeros
 *             without tokens)
 *   dstate_in [batch, width - 1, C] float32 out, or NULL
 *   ws        workspace of SWIMBA_SSM_CONV_BACKWARD
 */
swimba_status swimba_causal_conv_backward(const swimba_dims* dims, int32_t width, const void* x,
                                          int64_t ldx, const void* weight, const void* bias,
                                          int32_t act, const int32_t* seq_lens,
                                          const void* state_in, const void* dy,
                                          const float* dstate_out, void* dx, int64_t lddx,
                                          float* dweight, float* dbias, float* dstate_in,
                                          void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * One token of the convolution for `batch` sequences (dims->seqlen must be 1).
 *   x [batch, C] dtype, rows ldx apart;  weight, bias, act as above
 *   state_in  [batch, width - 1, C] dtype
 *   state_out [batch, width - 1, C] dtype out: state_in moved on by one token;
 *             may be state_in
 *   y         [batch, C] dtype out
 */
swimba_status swimba_causal_conv_step(const swimba_dims* dims, int32_t width, const void* x,
                                      int64_t ldx, const void* weight, const void* bias,
                                      int32_t act, const void* state_in, void* state_out, void* y,
                                      hipStream_t stream);

/*
 * Selective scan: N states per channel, the step and both vectors from the
 * token. For channel c of group g:
 *   delta_t = softplus(dt_t + dt_bias),   a_t[n] = exp(delta_t A[c, n]),
 *   h_t[n] = a_t[n] h_{t-1}[n] + delta_t B_t[g, n] x_t,
 *   u_t = sum_n C_t[g, n] h_t[n] + D[c] x_t,   y_t = u_t silu(z_t)   (u_t without z),
 *   h_{-1} = h_init.
 * States are held in float32. A is used as it is (a state decays where A < 0,
 * grows where A > 0 and is forgotten at every step above zero where A is -inf).
 *   x, dt, z  [M, C] dtype, rows ldx, lddt and ldz apart; z may be NULL
 *   B, C      [M, G * N] dtype, rows ldbc apart (both)
 *   A         [C, N] float32
 *   D         [C] float32, or NULL for zeros;  dt_bias [C] float32, or NULL
 *   h_init    [batch, C, N] float32, or NULL for zeros
 *   y         [M, C] dtype out
 *   h_final   [batch, C, N] float32 out, or NULL
 *   carry     float32 out of swimba_selective_scan_carry_size() bytes, or
 *             NULL: the states that the backward starts its blocks of tokens
 *             from
 *   ws        workspace of SWIMBA_SSM_SCAN
 * N at most 128 (else SWIMBA_ERR_UNSUPPORTED).
 */
swimba_status swimba_selective_scan(const swimba_dims* dims, const void* x, int64_t ldx,
                                    const void* dt, int64_t lddt, const void* z, int64_t ldz,
                                    const void* B, const void* C, int64_t ldbc, const float* A,
                                    const float* D, const float* dt_bias,
                                    const int32_t* seq_lens, const float* h_init, void* y,
                                    float* h_final, float* carry, void* ws, size_t ws_bytes,
                                    hipStream_t stream);

/* Bytes of the carry tensor for `dims` (0 for invalid dims or no tokens). */
size_t swimba_selective_scan_carry_size(const swimba_dims* dims);

/*
 * Backward of swimba_selective_scan. With v_t = dy_t silu(z_t) (dy_t without
 * z) and e_t = dl/dh_t,
 *   e_t[n] = C_t[n] v_t + a_{t+1}[n] e_{t+1}[n],   dh_final joining at the last token:
 *   dx_t = delta_t sum_n e_t[n] B_t[n] + D v_t,
 *   ddelta_t = sum_n e_t[n] (A[n] a_t[n] h_{t-1}[n] + B_t[n] x_t),
 *   ddt_t = ddelta_t sigmoid(dt_t + dt_bias),   dz_t = dy_t u_t silu'(z_t),
 *   dB_t[n] = sum_c e_t[c, n] delta_t x_t,   dC_t[n] = sum_c v_t h_t[c, n]   (the group's channels),
 *   dA[n] = sum_t e_t[n] delta_t a_t[n] h_{t-1}[n],   dD = sum_t v_t x_t,
 *   ddt_bias = sum_t ddt_t,   dh_init = a_0 e_0.
 * The states are recomputed from the forward's carry; sums over channels and
 * tokens run in a fixed order.
 *   x .. seq_lens  as given to the forward
 *   carry     as the forward wrote it for the same inputs
 *   dy        [M, C] dtype;  dh_final [batch, C, N] float32, or NULL for zeros
 *   dx, ddt, dz  [M, C] dtype out, rows lddx, ldddt and lddz apart; dz is
 *             required with z and ignored without
 *   dB, dC    [M, G * N] dtype out, rows lddbc apart (both)
 *   dA        [C, N] float32 out
 *   dD, ddt_bias  [C] float32 out, or NULL
 *   dh_init   [batch, C, N] float32 out, or NULL
 *   ws        workspace of SWIMBA_SSM_SCAN_BACKWARD
 */
swimba_status swimba_selective_scan_backward(
    const swimba_dims* dims, const void* x, int64_t ldx, const void* dt, int64_t lddt,
    const void* z, int64_t ldz, const void* B, const void* C, int64_t ldbc, const float* A,
    const float* D, const float* dt_bias, const int32_t* seq_lens, const float* carry,
    const void* dy, const float* dh_final, void* dx, int64_t lddx, void* ddt, int64_t ldddt,
    void* dz, int64_t lddz, void* dB, void* dC, int64_t lddbc, float* dA, float* dD,
    float* ddt_bias, float* dh_init, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * One token of the selective scan for `batch` sequences (dims->seqlen must be
 * 1), without a workspace.
 *   x, dt, z, B, C, A, D, dt_bias   as above with M = batch
 *   h_prev    [batch, C, N] float32;  h [batch, C, N] float32 out, may be h_prev
 *   y         [batch, C] dtype out
 */
swimba_status swimba_selective_step(const swimba_dims* dims, const void* x, int64_t ldx,
                                    const void* dt, int64_t lddt, const void* z, int64_t ldz,
                                    const void* B, const void* C, int64_t ldbc, const float* A,
                                    const float* D, const float* dt_bias, const float* h_prev,
                                    float* h, void* y, hipStream_t stream);

/*
 * Softmax cross entropy of each token over a vocabulary, without the logits:
 *   z = x w^T (float32),   lse = log sum_v exp(z_v),   loss = lse - z[target].
 * The loss is formed from the largest logit and the sum of exponentials below
 * it, so that a small one keeps its precision next to large logits.
 * A target outside [0, V) is no target: its loss is 0 and it gives no
 * gradient, whatever its row of x holds (its lse is that of the token). A
 * logit of +inf or NaN makes its token's lse infinite or NaN; one of -inf
 * counts for nothing, but where all are (lse -inf) or it is the target's
 * (loss +inf).
 *   x         [M, D] dtype;  w [V, D] dtype
 *   targets   [M] int32
 *   loss      [M] float32 out;  lse [M] float32 out
 *   ws        workspace of SWIMBA_SSM_CROSS_ENTROPY
 * D must be a multiple of 8 (else SWIMBA_ERR_UNSUPPORTED) and at most 2^20;
 * V at most 2^20, with (V + 2) D below 2^31; M V below some 2^37 (a launch's
 * threads), M below 2^28 (SWIMBA_ERR_DIMS otherwise).
 */
swimba_status swimba_cross_entropy(const swimba_dims* dims, const void* x, const void* w,
                                   const int32_t* targets, float* loss, float* lse, void* ws,
                                   size_t ws_bytes, hipStream_t stream);

/*
 * Backward of swimba_cross_entropy. The logits are computed again, a piece of
 * the vocabulary at a time:
 *   dz_v = (exp(z_v - lse) - [v = target]) dloss,   dx = dz w,   dw = dz^T x.
 * (An exponential is off by the rounding of its lse, up to 2^-24 |lse| of
 * itself.)
 * bf16 problems take dz into both products as the sum of three bf16 numbers,
 * all of its bits.
 *   x, w, targets  as given to the forward;  lse [M] float32 as it wrote it
 *   dloss     [M] float32: gradient of each token's loss (not looked at
 *             where there is no target)
 *   dx        [M, D] float32 out;  dw [V, D] float32 out (zeros without tokens)
 *   ws        workspace of SWIMBA_SSM_CROSS_ENTROPY_BACKWARD: x, dz of a piece of
 *             the vocabulary (for bf16 problems 6 bytes an element, 805 MB at most
 *             up to 2^17 tokens, 6 KB a token beyond; float32 two thirds of it)
 *             and partial sums of the products
 */
swimba_status swimba_cross_entropy_backward(const swimba_dims* dims, const void* x, const void* w,
                                            const int32_t* targets, const float* lse,
                                            const float* dloss, float* dx, float* dw, void* ws,
                                            size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SWIMBA_SSM_H */
