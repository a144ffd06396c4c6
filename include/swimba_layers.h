/*
 * swimba_layers.h - C ABI of the layers around the Swimba mixer on MI355X.
 *
 * The pages put the mixer into a hybrid stack of Mamba-2, attention and
 * feed-forward layers and fine-tune it (papernotes.org notes, Experiments).
 * These calls are what such a stack needs next to the mixer of swimba.h: a
 * layer norm with the residual add, the gated feed-forward projection, the
 * backward of each, and the backward of swimba_output_project (the mixer's
 * output projection and the feed-forward layer's down projection). The gated
 * linear recurrence over channels is not on the pages: it is a neighbour of
 * the scans of swimba.h, with a decay per channel and token and a backward.
 *
 * The conventions are those of swimba.h (device pointers, dense row-major
 * tensors unless a row stride is an argument, 16-byte alignment, caller-owned
 * workspaces, work on the given stream only, arguments validated before any
 * launch, bitwise repeatable results, swimba_last_error()). The sizes come
 * from swimba_dims as in swimba_output_project:
 *   M = batch * seqlen tokens, D = d_model, F = C = nheads * headdim, dtype.
 * The other fields must be valid for swimba.h (1 will do) and are not used.
 * "dtype" below is the element type of activations and weights; sums,
 * statistics, states and weight gradients are float32.
 * An output must not overlap an input or another output unless the call says
 * that it may. Calls on one device that share a workspace, a state or an
 * output must be ordered by the caller.
 */
#ifndef SWIMBA_LAYERS_H
#define SWIMBA_LAYERS_H

#include "swimba.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum swimba_activation {
  SWIMBA_ACT_SILU = 0, /* g sigmoid(g) */
  SWIMBA_ACT_GELU = 1  /* g Phi(g), Phi the normal distribution function (erf form) */
} swimba_activation;

typedef enum swimba_layer_call {
  SWIMBA_LAYER_NORM_BACKWARD = 0,
  SWIMBA_LAYER_GATED_SCAN = 1,
  SWIMBA_LAYER_GATED_SCAN_BACKWARD = 2,
  SWIMBA_LAYER_GATED_PROJECT_BACKWARD = 3,
  SWIMBA_LAYER_OUTPUT_PROJECT_BACKWARD = 4
} swimba_layer_call;

/* Workspace bytes that call `call` needs for `dims` (0 if none, and 0 for
 * invalid dims; the call itself then reports the error). Calls not in the
 * list need none. */
size_t swimba_layer_workspace_size(const swimba_dims* dims, int32_t call);

/*
 * Layer norm over rows of D, with an optional residual add before it:
 *   s = x + residual (rounded to dtype; s = x without a residual),
 *   mu = mean(s), rstd = (mean((s - mu)^2) + eps)^(-1/2),
 *   y = (s - mu) rstd weight + bias.
 * The statistics are of the stored (rounded) s, so that the backward, which
 * reads s, sees the same row. Values of magnitude above 1e18 overflow the
 * float32 variance; a row that holds an infinity or a NaN gives NaN in that
 * row only.
 *   x         [M, D] dtype
 *   residual  [M, D] dtype, or NULL
 *   weight    [D] dtype
 *   bias      [D] dtype, or NULL for zeros
 *   eps       finite and >= 0 (with 0 a constant row divides by zero)
 *   sum       [M, D] dtype out: s; required with a residual, ignored without;
 *             may be the same tensor as x or as residual
 *   y         [M, D] dtype out; may be the same tensor as x when there is no
 *             residual
 *   mean      [M] float32 out, or NULL;  rstd [M] float32 out, or NULL
 * D <= 32768 (else SWIMBA_ERR_UNSUPPORTED).
 */
swimba_status swimba_layer_norm(const swimba_dims* dims, const void* x, const void* residual,
                                const void* weight, const void* bias, float eps, void* sum,
                                void* y, float* mean, float* rstd, hipStream_t stream);

/*
 * Backward of swimba_layer_norm. With xh = (s - mean) rstd and g = dy weight:
 *   dx      = dres + rstd (g - mean(g) - xh mean(g xh))
 *   dweight = sum over rows of dy xh,   dbias = sum over rows of dy
 * dx is the gradient of s, that is of x and of the residual. The sums over
 * rows run in a fixed order.
 *   s         [M, D] dtype (the sum output, or x without a residual)
 *   weight    [D] dtype;  mean, rstd [M] float32 as the forward wrote them
 *   dy        [M, D] of dy_dtype: dims.dtype or SWIMBA_F32
 *   dres      [M, D] float32: the gradient that reaches s past the norm, or NULL
 *   dx        [M, D] float32 out; may be the same tensor as dres, or as a
 *             float32 dy
 *   dweight   [D] float32 out;  dbias [D] float32 out, or NULL
 *   ws        workspace of SWIMBA_LAYER_NORM_BACKWARD
 * Without tokens dweight and dbias are zeros.
 */
swimba_status swimba_layer_norm_backward(const swimba_dims* dims, const void* s,
                                         const void* weight, const float* mean, const float* rstd,
                                         const void* dy, int32_t dy_dtype, const float* dres,
                                         float* dx, float* dweight, float* dbias, void* ws,
                                         size_t ws_bytes, hipStream_t stream);

/*
 * Gated linear recurrence over C channels, each on its own:
 *   f_t = sigmoid(forget_t),  h_t = f_t h_{t-1} + (1 - f_t) x_t,
 *   y_t = h_t silu(gate_t)   (y_t = h_t without a gate),   h_{-1} = h_init.
 * h_t lies between h_{t-1} and x_t, so the state is bounded by its inputs
 * whatever the gates are. It is held in float32 and computed in the form that
 * keeps its relative precision for f near 0 and near 1 (an infinite x
 * therefore gives infinity or NaN from that token on, in that channel
 * of that sequence only).
 *   x, forget, gate  [M, C] dtype, gate may be NULL; rows `ld` elements apart
 *             (C <= ld < 2^22), so that all three may be column ranges of one
 *             projection's output
 *   seq_lens  [batch] int32, or NULL: tokens of each sequence that are in
 *             use (a value outside [0, seqlen] counts as the nearest bound).
 *             Past them x, forget and gate are not looked at (they may hold
 *             anything), y is zero and h_final is the state behind the last
 *             one (h_init for a length of 0)
 *   h_init    [batch, C] float32, or NULL for zeros
 *   y         [M, C] dtype out, dense
 *   h_final   [batch, C] float32 out, or NULL; may be the same tensor as h_init
 *   carry     float32 out of swimba_gated_scan_carry_size() bytes, or NULL:
 *             the states that the backward starts its chunks of tokens from
 *             (not written for chunks past a sequence's length)
 *   ws        workspace of SWIMBA_LAYER_GATED_SCAN. Chunks of tokens hand their
 *             states on through it: calls that use one workspace at the same
 *             time, which the conventions rule out, return SWIMBA_OK and give
 *             wrong results, NaN after some ten seconds of waiting among them
 */
swimba_status swimba_gated_scan(const swimba_dims* dims, const void* x, const void* forget,
                                const void* gate, int64_t ld, const int32_t* seq_lens,
                                const float* h_init, void* y, float* h_final, float* carry,
                                void* ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of the carry tensor for `dims` (0 for invalid dims or no tokens). */
size_t swimba_gated_scan_carry_size(const swimba_dims* dims);

/*
 * Backward of swimba_gated_scan. With e_t = dl/dh_t,
 *   e_t = dy_t silu(gate_t) + f_{t+1} e_{t+1},   dh_final joining at the last token:
 *   dx_t = (1 - f_t) e_t,   dforget_t = f_t (1 - f_t) e_t (h_{t-1} - x_t),
 *   dgate_t = dy_t h_t silu'(gate_t),   dh_init = f_0 e_0.
 * The states are recomputed from the forward's carry.
 *   x, forget, gate, ld, seq_lens   as given to the forward
 *   carry     as the forward wrote it for the same inputs
 *   dy        [M, C] dtype;  dh_final [batch, C] float32, or NULL for zeros
 *   dx, dforget, dgate  [M, C] dtype out, rows `ldd` elements apart (C <=
 *             ldd < 2^22), zeros past a sequence's length; dgate is required with a
 *             gate and ignored without
 *   dh_init   [batch, C] float32 out, or NULL; may be the same tensor as
 *             dh_final
 *   ws        workspace of SWIMBA_LAYER_GATED_SCAN_BACKWARD (used as the
 *             forward's)
 */
swimba_status swimba_gated_scan_backward(const swimba_dims* dims, const void* x,
                                         const void* forget, const void* gate, int64_t ld,
                                         const int32_t* seq_lens, const float* carry,
                                         const void* dy, const float* dh_final, void* dx,
                                         void* dforget, void* dgate, int64_t ldd, float* dh_init,
                                         void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * One token of the recurrence for `batch` sequences (dims->seqlen must be 1),
 * without a workspace:
 *   h = f h_prev + (1 - f) x,   y = h silu(gate).
 *   x, forget, gate  [batch, C] dtype, rows `ld` apart (C <= ld < 2^22); gate may be NULL
 *   h_prev    [batch, C] float32;  h [batch, C] float32 out, may be h_prev
 *   y         [batch, C] dtype out
 */
swimba_status swimba_gated_step(const swimba_dims* dims, const void* x, const void* forget,
                                const void* gate, int64_t ld, const float* h_prev, float* h,
                                void* y, hipStream_t stream);

/*
 * Gated feed-forward projection: both products, the activation and the gate
 * in one kernel (the down projection that follows is swimba_output_project).
 *   [g | u] = x w_in^T (float32 accumulation),   h = act(g) u
 *   x       [M, D] dtype
 *   w_in    [2 F, D] dtype: F rows for g, then F rows for u
 *   act     swimba_activation
 *   z       [M, 2 F] dtype out: [g | u], rounded, or NULL (the backward does
 *           not need it)
 *   h       [M, F] dtype out
 * D and F must be multiples of 8 (else SWIMBA_ERR_UNSUPPORTED); w_in at most
 * 2 GiB (else SWIMBA_ERR_DIMS).
 */
swimba_status swimba_gated_project(const swimba_dims* dims, const void* x, const void* w_in,
                                   int32_t act, void* z, void* h, hipStream_t stream);

/*
 * Backward of swimba_gated_project. g and u are recomputed in float32 from x
 * and w_in, so that the forward keeps nothing:
 *   dg = dh u act'(g),  du = dh act(g),  dz = [dg | du],
 *   dx = dz w_in,   dw_in = dz^T x.
 * bf16 problems take dz into both products as the sum of two bf16 numbers: an
 * element is off by at most 2^-16 of itself, where float32 would hold 2^-24 and
 * one bf16 2^-8, and dx by at most 2^-16 |dz| |w_in| from that (dw_in likewise).
 * An element of dz that bf16 rounds to infinity (above 3.39e38) gives NaN there.
 *   x, w_in, act as given to the forward
 *   dh      [M, F] dtype
 *   dx      [M, D] float32 out;  dw_in [2 F, D] float32 out (zeros without tokens)
 *   ws      workspace of SWIMBA_LAYER_GATED_PROJECT_BACKWARD
 */
swimba_status swimba_gated_project_backward(const swimba_dims* dims, const void* x,
                                            const void* w_in, const void* dh, int32_t act,
                                            float* dx, float* dw_in, void* ws, size_t ws_bytes,
                                            hipStream_t stream);

/*
 * Backward of swimba_output_project (out = y w_out^T):
 *   dy = dout w_out,   dw_out = dout^T y.
 *   y       [M, F] dtype;  w_out [D, F] dtype;  dout [M, D] dtype
 *   dy      [M, F] dtype out (what the backwards of the scans and of the
 *           gated projection take);  dw_out [D, F] float32 out (zeros without
 *           tokens)
 *   ws      workspace of SWIMBA_LAYER_OUTPUT_PROJECT_BACKWARD
 * D and F must be multiples of 8; w_out at most 2 GiB.
 */
swimba_status swimba_output_project_backward(const swimba_dims* dims, const void* y,
                                             const void* w_out, const void* dout, void* dy,
                                             float* dw_out, void* ws, size_t ws_bytes,
                                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SWIMBA_LAYERS_H */
