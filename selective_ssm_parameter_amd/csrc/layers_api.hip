// C ABI of the layers around the mixer (swimba_layers.h): argument
// validation, workspace carving, dispatch. Every check runs before the first
// launch; no HIP call is made on an invalid argument.
#include "swimba_layers.h"

#include <algorithm>
#include <cmath>

#include "api_common.hpp"
#include "layers.hpp"

using namespace swimba;

namespace {

// A grid's threads are counted in 32 bits.
constexpr int64_t kMaxThreads = int64_t(1) << 32;
constexpr int64_t kMaxLd = int64_t(1) << 22;
constexpr int64_t kMaxD = int64_t(1) << 20;

swimba_status read_layer_dims(const swimba_dims* dims, Dims& d) {
  const swimba_status st = read_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if (d.D > kMaxD) return fail(SWIMBA_ERR_DIMS, "d_model must be at most 2^20");
  return SWIMBA_OK;
}

int64_t elem(const Dims& d) { return d.bf16 ? 2 : 4; }

swimba_status check_norm(const Dims& d) {
  if (d.D > kNormMaxD)
    return fail(SWIMBA_ERR_UNSUPPORTED, "d_model %lld: the layer norm holds a row of at most %d",
                (long long)d.D, kNormMaxD);
  if (norm_fwd_threads(d.M, (int)d.D) >= kMaxThreads)
    return fail(SWIMBA_ERR_DIMS, "too many rows of this width for one launch");
  return SWIMBA_OK;
}

swimba_status check_gscan(const Dims& d, int64_t ld, int64_t ldd) {
  if (ld < d.HP || ldd < d.HP)
    return fail(SWIMBA_ERR_DIMS, "a row stride is smaller than nheads * headdim = %lld",
                (long long)d.HP);
  // a chunk's 128 rows are addressed through one buffer
  if (ld >= kMaxLd || ldd >= kMaxLd)
    return fail(SWIMBA_ERR_DIMS, "row strides must be below 2^22 elements");
  if (gscan_blocks(d.Bt, d.T, d.HP) * 512 >= kMaxThreads || d.Bt * d.HP >= kMaxThreads - 256)
    return fail(SWIMBA_ERR_DIMS, "too many chunks of tokens and channels for one launch");
  return SWIMBA_OK;
}

// weight_rows x weight_cols is the weight matrix read through one buffer.
swimba_status check_dense(const Dims& d, int64_t weight_rows, int64_t weight_cols) {
  if (d.D % 8 != 0 || d.HP % 8 != 0)
    return fail(SWIMBA_ERR_UNSUPPORTED,
                "d_model and nheads * headdim must be multiples of 8 for the matrix cores");
  if (weight_rows * weight_cols * elem(d) > kMaxRecord)
    return fail(SWIMBA_ERR_DIMS, "the weights (%lld bytes) exceed 2 GiB",
                (long long)(weight_rows * weight_cols * elem(d)));
  const int64_t tiles = ((d.M + 127) / 128 + 1) * ((2 * d.HP + d.D + 127) / 128 + 1);
  if (tiles * 512 >= kMaxThreads) return fail(SWIMBA_ERR_DIMS, "too many tiles for one launch");
  return SWIMBA_OK;
}

swimba_status check_act(int32_t act) {
  if (act != SWIMBA_ACT_SILU && act != SWIMBA_ACT_GELU)
    return fail(SWIMBA_ERR_DIMS, "act %d is not a swimba_activation", act);
  return SWIMBA_OK;
}

size_t gated_bwd_dz_bytes(const Dims& d) {
  return align256(gated_dz_bytes(d.bf16, (int)d.M, (int)d.HP));
}

size_t layer_ws(const Dims& d, int32_t call) {
  if (d.M == 0) return 0;
  const int M = (int)d.M, D = (int)d.D, F = (int)d.HP;
  switch (call) {
    case SWIMBA_LAYER_NORM_BACKWARD:
      return d.D > kNormMaxD ? 0
                             : sizeof(float) * 2 * (size_t)norm_bwd_parts((int)d.M, (int)d.D) * d.D;
    case SWIMBA_LAYER_GATED_SCAN:
    case SWIMBA_LAYER_GATED_SCAN_BACKWARD:
      return gscan_ws_bytes((int)d.Bt, (int)d.T, (int)d.HP);
    // dz, and behind it the partial sums of dx, then those of dw_in
    case SWIMBA_LAYER_GATED_PROJECT_BACKWARD:
      return gated_bwd_dz_bytes(d) +
             std::max(dense_ws_bytes(d.bf16, d.bf16, false, M, D, 2 * F),
                      dense_ws_bytes(d.bf16, d.bf16, true, 2 * F, D, M));
    case SWIMBA_LAYER_OUTPUT_PROJECT_BACKWARD:
      return std::max(dense_ws_bytes(d.bf16, false, false, M, F, D),
                      dense_ws_bytes(d.bf16, false, true, D, F, M));
    default: return 0;
  }
}

}  // namespace

extern "C" {

size_t swimba_layer_workspace_size(const swimba_dims* dims, int32_t call) {
  Dims d;
  if (!query_dims(dims, d) || d.D > kMaxD) return 0;
  return layer_ws(d, call);
}

size_t swimba_gated_scan_carry_size(const swimba_dims* dims) {
  Dims d;
  if (!query_dims(dims, d) || d.D > kMaxD) return 0;
  return sizeof(float) * (size_t)(d.Bt * gscan_chunks((int)d.T) * d.HP);
}

swimba_status swimba_layer_norm(const swimba_dims* dims, const void* x, const void* residual,
                                const void* weight, const void* bias, float eps, void* sum,
                                void* y, float* mean, float* rstd, hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if ((st = check_norm(d)) != SWIMBA_OK) return st;
  if (!(eps >= 0.f) || std::isinf(eps))
    return fail(SWIMBA_ERR_DIMS, "eps must be finite and >= 0");
  if (d.M == 0) return SWIMBA_OK;
  REQUIRE_PTR(x);
  OPTIONAL_PTR(residual);
  REQUIRE_PTR(weight);
  OPTIONAL_PTR(bias);
  if (residual) REQUIRE_PTR(sum);
  REQUIRE_PTR(y);
  OPTIONAL_PTR(mean);
  OPTIONAL_PTR(rstd);
  NormFwdArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.eps = eps;
  a.sum = sum; a.y = y; a.mean = mean; a.rstd = rstd; a.M = (int)d.M; a.D = (int)d.D;
  return hip_status(launch_norm_fwd(d.bf16, a, stream), "layer_norm launch");
}

swimba_status swimba_layer_norm_backward(const swimba_dims* dims, const void* s,
                                         const void* weight, const float* mean, const float* rstd,
                                         const void* dy, int32_t dy_dtype, const float* dres,
                                         float* dx, float* dweight, float* dbias, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if ((st = check_norm(d)) != SWIMBA_OK) return st;
  if (dy_dtype != SWIMBA_F32 && dy_dtype != dims->dtype)
    return fail(SWIMBA_ERR_UNSUPPORTED, "dy_dtype must be dims.dtype or SWIMBA_F32");
  REQUIRE_PTR(dweight);
  OPTIONAL_PTR(dbias);
  if (d.M == 0) {  // no tokens: the weight gradients are zero
    hipError_t e = launch_fill_zero(dweight, (size_t)d.D, stream);
    if (e == hipSuccess && dbias) e = launch_fill_zero(dbias, (size_t)d.D, stream);
    return hip_status(e, "layer_norm_backward launch");
  }
  REQUIRE_PTR(s);
  REQUIRE_PTR(weight);
  REQUIRE_PTR(mean);
  REQUIRE_PTR(rstd);
  REQUIRE_PTR(dy);
  OPTIONAL_PTR(dres);
  REQUIRE_PTR(dx);
  if ((st = check_ws(ws, ws_bytes, layer_ws(d, SWIMBA_LAYER_NORM_BACKWARD))) != SWIMBA_OK)
    return st;
  NormBwdArgs a{};
  a.s = s; a.weight = weight; a.mean = mean; a.rstd = rstd; a.dy = dy; a.dres = dres;
  a.dx = dx; a.dw = dweight; a.db = dbias; a.part = static_cast<float*>(ws);
  a.M = (int)d.M; a.D = (int)d.D;
  return hip_status(launch_norm_bwd(d.bf16, dy_dtype == SWIMBA_F32, a, stream),
                    "layer_norm_backward launch");
}

swimba_status swimba_gated_scan(const swimba_dims* dims, const void* x, const void* forget,
                                const void* gate, int64_t ld, const int32_t* seq_lens,
                                const float* h_init, void* y, float* h_final, float* carry,
                                void* ws, size_t ws_bytes, hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if ((st = check_gscan(d, ld, d.HP)) != SWIMBA_OK) return st;
  if (d.Bt == 0) return SWIMBA_OK;
  OPTIONAL_PTR(h_init);
  OPTIONAL_PTR(h_final);
  if (d.M == 0) {  // no tokens: the states pass through unchanged
    if (!h_final || h_final == h_init) return SWIMBA_OK;
    const size_t n = (size_t)(d.Bt * d.HP);
    return hip_status(h_init ? launch_state_copy(h_init, h_final, n, stream)
                             : launch_fill_zero(h_final, n, stream),
                      "gated_scan launch");
  }
  REQUIRE_PTR(x);
  REQUIRE_PTR(forget);
  OPTIONAL_PTR(gate);
  OPTIONAL_PTR(seq_lens);
  REQUIRE_PTR(y);
  OPTIONAL_PTR(carry);
  if ((st = check_ws(ws, ws_bytes, layer_ws(d, SWIMBA_LAYER_GATED_SCAN))) != SWIMBA_OK) return st;
  GScanArgs a{};
  a.x = x; a.f = forget; a.o = gate; a.ld = ld; a.lens = seq_lens; a.h_init = h_init;
  a.y = y; a.h_final = h_final; a.carry = carry; a.ws = ws;
  a.Bt = (int)d.Bt; a.T = (int)d.T; a.C = (int)d.HP;
  return hip_status(launch_gscan(d.bf16, a, stream), "gated_scan launch");
}

swimba_status swimba_gated_scan_backward(const swimba_dims* dims, const void* x,
                                         const void* forget, const void* gate, int64_t ld,
                                         const int32_t* seq_lens, const float* carry,
                                         const void* dy, const float* dh_final, void* dx,
                                         void* dforget, void* dgate, int64_t ldd, float* dh_init,
                                         void* ws, size_t ws_bytes, hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if ((st = check_gscan(d, ld, ldd)) != SWIMBA_OK) return st;
  if (d.Bt == 0) return SWIMBA_OK;
  OPTIONAL_PTR(dh_final);
  OPTIONAL_PTR(dh_init);
  if (d.M == 0) {  // no tokens: the state's gradient passes through unchanged
    if (!dh_init || dh_init == dh_final) return SWIMBA_OK;
    const size_t n = (size_t)(d.Bt * d.HP);
    return hip_status(dh_final ? launch_state_copy(dh_final, dh_init, n, stream)
                               : launch_fill_zero(dh_init, n, stream),
                      "gated_scan_backward launch");
  }
  REQUIRE_PTR(x);
  REQUIRE_PTR(forget);
  OPTIONAL_PTR(gate);
  OPTIONAL_PTR(seq_lens);
  REQUIRE_PTR(carry);
  REQUIRE_PTR(dy);
  REQUIRE_PTR(dx);
  REQUIRE_PTR(dforget);
  if (gate) REQUIRE_PTR(dgate);
  if ((st = check_ws(ws, ws_bytes, layer_ws(d, SWIMBA_LAYER_GATED_SCAN_BACKWARD))) != SWIMBA_OK)
    return st;
  GScanArgs a{};
  a.x = x; a.f = forget; a.o = gate; a.ld = ld; a.lens = seq_lens; a.carry_in = carry;
  a.dy = dy; a.dh_final = dh_final; a.dx = dx; a.df = dforget; a.d_o = dgate; a.ldd = ldd;
  a.dh_init = dh_init; a.ws = ws;
  a.Bt = (int)d.Bt; a.T = (int)d.T; a.C = (int)d.HP;
  return hip_status(launch_gscan_backward(d.bf16, a, stream), "gated_scan_backward launch");
}

swimba_status swimba_gated_step(const swimba_dims* dims, const void* x, const void* forget,
                                const void* gate, int64_t ld, const float* h_prev, float* h,
                                void* y, hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if (d.T != 1) return fail(SWIMBA_ERR_DIMS, "gated_step takes one token: seqlen must be 1");
  if (ld < d.HP || ld >= kMaxLd)
    return fail(SWIMBA_ERR_DIMS, "the row stride must lie in [nheads * headdim, 2^22)");
  if (d.Bt * d.HP >= kMaxThreads - 256) return fail(SWIMBA_ERR_DIMS, "too many channels for one launch");
  if (d.Bt == 0) return SWIMBA_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(forget);
  OPTIONAL_PTR(gate);
  REQUIRE_PTR(h_prev);
  REQUIRE_PTR(h);
  REQUIRE_PTR(y);
  return hip_status(launch_gscan_step(d.bf16, x, forget, gate, ld, h_prev, h, y, (int)d.Bt,
                                      (int)d.HP, stream),
                    "gated_step launch");
}

swimba_status swimba_gated_project(const swimba_dims* dims, const void* x, const void* w_in,
                                   int32_t act, void* z, void* h, hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if ((st = check_dense(d, 2 * d.HP, d.D)) != SWIMBA_OK) return st;
  if ((st = check_act(act)) != SWIMBA_OK) return st;
  if (d.M == 0) return SWIMBA_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w_in);
  OPTIONAL_PTR(z);
  REQUIRE_PTR(h);
  return hip_status(launch_gated_project(d.bf16, (int)d.M, (int)d.D, (int)d.HP, act, x, w_in, z, h,
                                         stream),
                    "gated_project launch");
}

swimba_status swimba_gated_project_backward(const swimba_dims* dims, const void* x,
                                            const void* w_in, const void* dh, int32_t act,
                                            float* dx, float* dw_in, void* ws, size_t ws_bytes,
                                            hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if ((st = check_dense(d, 2 * d.HP, d.D)) != SWIMBA_OK) return st;
  if ((st = check_act(act)) != SWIMBA_OK) return st;
  REQUIRE_PTR(dw_in);
  if (d.M == 0)
    return hip_status(launch_fill_zero(dw_in, (size_t)(2 * d.HP * d.D), stream),
                      "gated_project_backward launch");
  REQUIRE_PTR(x);
  REQUIRE_PTR(w_in);
  REQUIRE_PTR(dh);
  REQUIRE_PTR(dx);
  if ((st = check_ws(ws, ws_bytes, layer_ws(d, SWIMBA_LAYER_GATED_PROJECT_BACKWARD))) != SWIMBA_OK)
    return st;
  const int M = (int)d.M, D = (int)d.D, F = (int)d.HP;
  unsigned char* w8 = static_cast<unsigned char*>(ws);
  unsigned char* part = w8 + gated_bwd_dz_bytes(d);
  const void* lo = d.bf16 ? w8 + (size_t)M * 2 * F * 2 : nullptr;
  hipError_t e = launch_gated_dz(d.bf16, M, D, F, act, x, w_in, dh, ws, stream);
  if (e != hipSuccess) return hip_status(e, "gated_project_backward dz launch");
  e = launch_dense_nn(d.bf16, "gated_dx", M, 2 * F, D, ws, lo, w_in, dx, part, stream);
  if (e != hipSuccess) return hip_status(e, "gated_project_backward dx launch");
  return hip_status(launch_dense_tn(d.bf16, "gated_dw", M, 2 * F, D, ws, lo, x, dw_in, part,
                                    stream),
                    "gated_project_backward dw launch");
}

swimba_status swimba_output_project_backward(const swimba_dims* dims, const void* y,
                                             const void* w_out, const void* dout, void* dy,
                                             float* dw_out, void* ws, size_t ws_bytes,
                                             hipStream_t stream) {
  Dims d;
  swimba_status st = read_layer_dims(dims, d);
  if (st != SWIMBA_OK) return st;
  if ((st = check_dense(d, d.D, d.HP)) != SWIMBA_OK) return st;
  REQUIRE_PTR(dw_out);
  if (d.M == 0)
    return hip_status(launch_fill_zero(dw_out, (size_t)(d.D * d.HP), stream),
                      "output_project_backward launch");
  REQUIRE_PTR(y);
  REQUIRE_PTR(w_out);
  REQUIRE_PTR(dout);
  REQUIRE_PTR(dy);
  if ((st = check_ws(ws, ws_bytes, layer_ws(d, SWIMBA_LAYER_OUTPUT_PROJECT_BACKWARD))) != SWIMBA_OK)
    return st;
  const int M = (int)d.M, D = (int)d.D, F = (int)d.HP;
  hipError_t e = launch_dense_nn(d.bf16, "output_project_dy", M, D, F, dout, nullptr, w_out, dy, ws, stream);
  if (e != hipSuccess) return hip_status(e, "output_project_backward dy launch");
  return hip_status(launch_dense_tn(d.bf16, "output_project_dw", M, D, F, dout, nullptr, y, dw_out, ws,
                                    stream),
                    "output_project_backward dw launch");
}

}  // extern "C"
