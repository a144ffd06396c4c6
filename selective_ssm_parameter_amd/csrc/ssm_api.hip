// C ABI of the selective state space layer and its loss (swimba_ssm.h):
// argument validation, workspace carving, dispatch. Every check runs before the
// first launch; no HIP call is made on an invalid argument.
#include "swimba_ssm.h"

#include <algorithm>

#include "api_common.hpp"
#include "layers.hpp"
#include "ssm.hpp"

using namespace swimba;

namespace {

constexpr int64_t kMaxThreads = int64_t(1) << 32;  // a grid's threads are counted in 32 bits
constexpr int64_t kMaxLd = int64_t(1) << 22;
constexpr int64_t kMaxD = int64_t(1) << 20;

swimba_status check_ld(int64_t ld, int64_t row, const char* what) {
  if (ld < row || ld >= kMaxLd)
    return fail(SWIMBA_ERR_DIMS, "%s %lld: row strides must lie in [%lld, 2^22)", what,
                (long long)ld, (long long)row);
  return SWIMBA_OK;
}
#define CHECK_LD(ld, row)                                                    \
  do {                                                                       \
    const swimba_status e = check_ld(ld, row, #ld);                          \
    if (e != SWIMBA_OK) return e;                                            \
  } while (0)
#define CHECK(call)                                                          \
  do {                                                                       \
    const swimba_status e = (call);                                          \
    if (e != SWIMBA_OK) return e;                                            \
  } while (0)

swimba_status check_conv(const Dims& d, int32_t width, int32_t act) {
  if (width < 2 || width > 4)
    return fail(SWIMBA_ERR_UNSUPPORTED, "width %d: the convolution takes 2, 3 or 4", width);
  if (act != SWIMBA_CONV_LINEAR && act != SWIMBA_CONV_SILU)
    return fail(SWIMBA_ERR_DIMS, "act %d is not a swimba_conv_act", act);
  // (a thread per channel and 8 tokens, at most)
  if (d.Bt * ((d.T + 7) / 8 + 1) >= kMaxThreads / d.HP)
    return fail(SWIMBA_ERR_DIMS, "too many tokens and channels for one launch");
  return SWIMBA_OK;
}

swimba_status check_scan(const Dims& d) {
  if (d.N > kScanMaxN)
    return fail(SWIMBA_ERR_UNSUPPORTED, "dstate %lld: the selective scan holds at most %d states",
                (long long)d.N, kScanMaxN);
  if (d.GN >= kMaxLd) return fail(SWIMBA_ERR_DIMS, "ngroups * dstate must be below 2^22");
  if (d.Bt > 0 && sscan_threads(d.Bt, d.T, d.HP, d.N, d.G) >= kMaxThreads)
    return fail(SWIMBA_ERR_DIMS, "too many tokens and channels for one launch");
  return SWIMBA_OK;
}

swimba_status check_loss(const Dims& d) {
  if (d.D > kMaxD) return fail(SWIMBA_ERR_DIMS, "d_model must be at most 2^20");
  if (d.D % 8 != 0)
    return fail(SWIMBA_ERR_UNSUPPORTED, "d_model must be a multiple of 8 for the matrix cores");
  // (smaller tiles are taken where there are few; the statistics' second kernel has 16
  // threads a token)
  const int64_t tiles = ((d.M + 127) / 128 + 1) * ((d.HP + 127) / 128 + 1);
  if (tiles * 512 >= kMaxThreads || d.M * 16 >= kMaxThreads - 256)
    return fail(SWIMBA_ERR_DIMS, "too many tokens and words for one launch");
  return SWIMBA_OK;
}

// The backward's pieces of the vocabulary: dz of one (three bf16 numbers or one float32
// an element) has 2^27 elements at most, 805 or 537 MB, in whole tiles (half of that: 4
// to 12 % slower, a quarter 7 to 15 %, at 16384 x 768 over 32768, 65536 x 512 over 32768
// and 8192 x 768 over 131072 words, but 2 % faster at 4096 x 1024 over 131072); but past
// 131072 tokens 1024 words, whatever that takes (6 KB a token). Each piece but the first
// reads and writes dx once more, so they are as few as that allows, and then equally
// large. A piece's weights are read through one buffer.
int64_t xent_piece(const Dims& d) {
  const int64_t cols = (int64_t(1) << 27) / std::max<int64_t>(1, d.M) / 256 * 256;
  const int64_t rows = kMaxRecord / (d.D * (d.bf16 ? 2 : 4)) / 256 * 256;
  const int64_t most = std::min({d.HP, rows, std::max<int64_t>(1024, cols)});
  const int64_t pieces = (d.HP + most - 1) / most;
  return std::min(most, ((d.HP + pieces - 1) / pieces + 255) / 256 * 256);
}
int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

// bf16 problems take dz through both products as three bf16 numbers, all of its 24
// bits. Two would be off by up to 2^-17 = 7.6e-6 in the 2-norm, whatever the sums'
// lengths (all of it where every target's dz has the same value), and are by 1.0 to
// 4.3e-6 with the mean over the tokens as the loss; three are off by what the sums in
// float32 are, 2e-7 at 246 tokens to 8e-7 at 16384 x 768 over 32768 words (elementary
// float32 products: 2e-7 to 3.2e-6). Neither dx, whose sums run over the words, nor dw,
// over the tokens, has a usual length at which two would not be the larger part. The
// third costs nothing at 246 x 480 over 832 words (36 us), 1570 against 1210 us at 8192 x
// 768 over 16000 and 6400 against 4750 at 16384 x 768 over 32768.
int xent_numbers(const Dims& d) { return d.bf16 ? 3 : 1; }

size_t xent_dz_bytes(const Dims& d, int64_t nv) {
  return align256((d.bf16 ? 6 : 4) * (size_t)(d.M * round8(nv)));
}

// x without the rows of tokens that have no target, behind dz.
size_t xent_rows_bytes(const Dims& d) { return align256((size_t)(d.M * d.D) * (d.bf16 ? 2 : 4)); }

size_t xent_bwd_ws(const Dims& d) {
  const int M = (int)d.M, D = (int)d.D;
  const int64_t piece = xent_piece(d);
  size_t sums = 0;
  for (int64_t nv : {piece, d.HP % piece}) {
    if (nv == 0) continue;
    sums = std::max({sums, dense_ws_bytes(d.bf16, xent_numbers(d), false, M, D, (int)round8(nv)),
                     dense_ws_bytes(d.bf16, xent_numbers(d), true, (int)nv, D, M)});
  }
  return xent_dz_bytes(d, piece) + xent_rows_bytes(d) + sums;
}

size_t ssm_ws(const Dims& d, int32_t call) {
  if (d.M == 0) return 0;
  const int Bt = (int)d.Bt, T = (int)d.T, C = (int)d.HP, N = (int)d.N, G = (int)d.G;
  switch (call) {
    case SWIMBA_SSM_CONV_BACKWARD: return conv_bwd_ws_bytes(Bt, T, C);
    case SWIMBA_SSM_SCAN: return N > kScanMaxN ? 0 : sscan_ws_bytes(Bt, T, C, N, G);
    case SWIMBA_SSM_SCAN_BACKWARD: return N > kScanMaxN ? 0 : sscan_bwd_ws_bytes(Bt, T, C, N, G);
    // (d_model is theirs alone)
    case SWIMBA_SSM_CROSS_ENTROPY:
      return d.D > kMaxD ? 0 : xent_ws_bytes(d.bf16, (int)d.M, (int)d.D, C);
    case SWIMBA_SSM_CROSS_ENTROPY_BACKWARD: return d.D > kMaxD ? 0 : xent_bwd_ws(d);
    default: return 0;
  }
}

// Copies (or clears) states where there are no tokens.
hipError_t pass_states(const float* from, float* to, size_t n, hipStream_t s) {
  if (!to || to == from || n == 0) return hipSuccess;
  return from ? launch_state_copy(from, to, n, s) : launch_fill_zero(to, n, s);
}

}  // namespace

extern "C" {

size_t swimba_ssm_workspace_size(const swimba_dims* dims, int32_t call) {
  Dims d;
  if (!query_dims(dims, d)) return 0;
  return ssm_ws(d, call);
}

size_t swimba_selective_scan_carry_size(const swimba_dims* dims) {
  Dims d;
  if (!query_dims(dims, d) || d.N > kScanMaxN) return 0;
  return sscan_carry_bytes((int)d.Bt, (int)d.T, (int)d.HP, (int)d.N);
}

swimba_status swimba_causal_conv(const swimba_dims* dims, int32_t width, const void* x,
                                 int64_t ldx, const void* weight, const void* bias, int32_t act,
                                 const int32_t* seq_lens, const void* state_in, void* y,
                                 void* state_out, hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  CHECK(check_conv(d, width, act));
  CHECK_LD(ldx, d.HP);
  if (d.Bt == 0) return SWIMBA_OK;
  OPTIONAL_PTR(state_in);
  OPTIONAL_PTR(state_out);
  if (state_out && state_out == state_in)
    return fail(SWIMBA_ERR_DIMS, "state_out must not be state_in (a step's may)");
  if (d.M == 0) {  // no tokens: the state passes through unchanged
    const size_t n = (size_t)(d.Bt * (width - 1) * d.HP);
    if (!state_out) return SWIMBA_OK;
    return hip_status(launch_conv_state(d.bf16, state_in, state_out, n, stream),
                      "causal_conv launch");
  }
  REQUIRE_PTR(x);
  REQUIRE_PTR(weight);
  OPTIONAL_PTR(bias);
  OPTIONAL_PTR(seq_lens);
  REQUIRE_PTR(y);
  ConvArgs a{};
  a.x = x; a.ldx = ldx; a.w = weight; a.bias = bias; a.lens = seq_lens; a.state_in = state_in;
  a.y = y; a.state_out = state_out;
  a.Bt = (int)d.Bt; a.T = (int)d.T; a.C = (int)d.HP; a.W = width; a.silu = act;
  return hip_status(launch_conv(d.bf16, a, stream), "causal_conv launch");
}

swimba_status swimba_causal_conv_backward(const swimba_dims* dims, int32_t width, const void* x,
                                          int64_t ldx, const void* weight, const void* bias,
                                          int32_t act, const int32_t* seq_lens,
                                          const void* state_in, const void* dy,
                                          const float* dstate_out, void* dx, int64_t lddx,
                                          float* dweight, float* dbias, float* dstate_in,
                                          void* ws, size_t ws_bytes, hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  CHECK(check_conv(d, width, act));
  CHECK_LD(ldx, d.HP);
  CHECK_LD(lddx, d.HP);
  REQUIRE_PTR(dweight);
  OPTIONAL_PTR(dbias);
  OPTIONAL_PTR(dstate_out);
  OPTIONAL_PTR(dstate_in);
  if (dstate_in && dstate_in == dstate_out)
    return fail(SWIMBA_ERR_DIMS, "dstate_in must not be dstate_out");
  if (d.M == 0) {  // no tokens: zeros, the state's gradient passes through unchanged
    hipError_t e = launch_fill_zero(dweight, (size_t)(d.HP * width), stream);
    if (e == hipSuccess && dbias) e = launch_fill_zero(dbias, (size_t)d.HP, stream);
    if (e == hipSuccess)
      e = pass_states(dstate_out, dstate_in, (size_t)(d.Bt * (width - 1) * d.HP), stream);
    return hip_status(e, "causal_conv_backward launch");
  }
  REQUIRE_PTR(x);
  REQUIRE_PTR(weight);
  OPTIONAL_PTR(bias);
  OPTIONAL_PTR(seq_lens);
  OPTIONAL_PTR(state_in);
  REQUIRE_PTR(dy);
  REQUIRE_PTR(dx);
  CHECK(check_ws(ws, ws_bytes, ssm_ws(d, SWIMBA_SSM_CONV_BACKWARD)));
  ConvArgs a{};
  a.x = x; a.ldx = ldx; a.w = weight; a.bias = bias; a.lens = seq_lens; a.state_in = state_in;
  a.dy = dy; a.dstate_out = dstate_out; a.dx = dx; a.lddx = lddx; a.dw = dweight; a.db = dbias;
  a.dstate_in = dstate_in; a.part = static_cast<float*>(ws);
  a.Bt = (int)d.Bt; a.T = (int)d.T; a.C = (int)d.HP; a.W = width; a.silu = act;
  return hip_status(launch_conv_backward(d.bf16, a, stream), "causal_conv_backward launch");
}

swimba_status swimba_causal_conv_step(const swimba_dims* dims, int32_t width, const void* x,
                                      int64_t ldx, const void* weight, const void* bias,
                                      int32_t act, const void* state_in, void* state_out, void* y,
                                      hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  if (d.T != 1) return fail(SWIMBA_ERR_DIMS, "causal_conv_step takes one token: seqlen must be 1");
  CHECK(check_conv(d, width, act));
  CHECK_LD(ldx, d.HP);
  if (d.Bt == 0) return SWIMBA_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(weight);
  OPTIONAL_PTR(bias);
  REQUIRE_PTR(state_in);
  REQUIRE_PTR(state_out);
  REQUIRE_PTR(y);
  ConvArgs a{};
  a.x = x; a.ldx = ldx; a.w = weight; a.bias = bias; a.state_in = state_in; a.y = y;
  a.state_out = state_out;
  a.Bt = (int)d.Bt; a.T = 1; a.C = (int)d.HP; a.W = width; a.silu = act;
  return hip_status(launch_conv_step(d.bf16, a, stream), "causal_conv_step launch");
}

swimba_status swimba_selective_scan(const swimba_dims* dims, const void* x, int64_t ldx,
                                    const void* dt, int64_t lddt, const void* z, int64_t ldz,
                                    const void* B, const void* C, int64_t ldbc, const float* A,
                                    const float* D, const float* dt_bias,
                                    const int32_t* seq_lens, const float* h_init, void* y,
                                    float* h_final, float* carry, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  CHECK(check_scan(d));
  CHECK_LD(ldx, d.HP);
  CHECK_LD(lddt, d.HP);
  if (z) CHECK_LD(ldz, d.HP);
  CHECK_LD(ldbc, d.GN);
  if (d.Bt == 0) return SWIMBA_OK;
  OPTIONAL_PTR(h_init);
  OPTIONAL_PTR(h_final);
  if (d.M == 0)  // no tokens: the states pass through unchanged
    return hip_status(pass_states(h_init, h_final, (size_t)(d.Bt * d.HP * d.N), stream),
                      "selective_scan launch");
  if (h_final && h_final == h_init)
    return fail(SWIMBA_ERR_DIMS, "h_final must not be h_init (a step's may)");
  REQUIRE_PTR(x);
  REQUIRE_PTR(dt);
  OPTIONAL_PTR(z);
  REQUIRE_PTR(B);
  REQUIRE_PTR(C);
  REQUIRE_PTR(A);
  OPTIONAL_PTR(D);
  OPTIONAL_PTR(dt_bias);
  OPTIONAL_PTR(seq_lens);
  REQUIRE_PTR(y);
  OPTIONAL_PTR(carry);
  CHECK(check_ws(ws, ws_bytes, ssm_ws(d, SWIMBA_SSM_SCAN)));
  SScanArgs a{};
  a.x = x; a.dt = dt; a.z = z; a.ldx = ldx; a.lddt = lddt; a.ldz = ldz; a.B = B; a.C = C;
  a.ldbc = ldbc; a.A = A; a.D = D; a.bias = dt_bias; a.lens = seq_lens; a.h_init = h_init;
  a.y = y; a.h_final = h_final; a.carry = carry; a.ws = ws;
  a.Bt = (int)d.Bt; a.T = (int)d.T; a.Ch = (int)d.HP; a.N = (int)d.N; a.G = (int)d.G;
  return hip_status(launch_sscan(d.bf16, a, stream), "selective_scan launch");
}

swimba_status swimba_selective_scan_backward(
    const swimba_dims* dims, const void* x, int64_t ldx, const void* dt, int64_t lddt,
    const void* z, int64_t ldz, const void* B, const void* C, int64_t ldbc, const float* A,
    const float* D, const float* dt_bias, const int32_t* seq_lens, const float* carry,
    const void* dy, const float* dh_final, void* dx, int64_t lddx, void* ddt, int64_t ldddt,
    void* dz, int64_t lddz, void* dB, void* dC, int64_t lddbc, float* dA, float* dD,
    float* ddt_bias, float* dh_init, void* ws, size_t ws_bytes, hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  CHECK(check_scan(d));
  CHECK_LD(ldx, d.HP);
  CHECK_LD(lddt, d.HP);
  if (z) CHECK_LD(ldz, d.HP);
  CHECK_LD(ldbc, d.GN);
  CHECK_LD(lddx, d.HP);
  CHECK_LD(ldddt, d.HP);
  if (z) CHECK_LD(lddz, d.HP);
  CHECK_LD(lddbc, d.GN);
  REQUIRE_PTR(dA);
  OPTIONAL_PTR(dD);
  OPTIONAL_PTR(ddt_bias);
  OPTIONAL_PTR(dh_final);
  OPTIONAL_PTR(dh_init);
  if (d.M == 0) {  // no tokens: zeros, the state's gradient passes through unchanged
    hipError_t e = launch_fill_zero(dA, (size_t)(d.HP * d.N), stream);
    if (e == hipSuccess && dD) e = launch_fill_zero(dD, (size_t)d.HP, stream);
    if (e == hipSuccess && ddt_bias) e = launch_fill_zero(ddt_bias, (size_t)d.HP, stream);
    if (e == hipSuccess)
      e = pass_states(dh_final, dh_init, (size_t)(d.Bt * d.HP * d.N), stream);
    return hip_status(e, "selective_scan_backward launch");
  }
  if (dh_init && dh_init == dh_final)
    return fail(SWIMBA_ERR_DIMS, "dh_init must not be dh_final");
  REQUIRE_PTR(x);
  REQUIRE_PTR(dt);
  OPTIONAL_PTR(z);
  REQUIRE_PTR(B);
  REQUIRE_PTR(C);
  REQUIRE_PTR(A);
  OPTIONAL_PTR(D);
  OPTIONAL_PTR(dt_bias);
  OPTIONAL_PTR(seq_lens);
  REQUIRE_PTR(carry);
  REQUIRE_PTR(dy);
  REQUIRE_PTR(dx);
  REQUIRE_PTR(ddt);
  if (z) REQUIRE_PTR(dz);
  REQUIRE_PTR(dB);
  REQUIRE_PTR(dC);
  CHECK(check_ws(ws, ws_bytes, ssm_ws(d, SWIMBA_SSM_SCAN_BACKWARD)));
  SScanArgs a{};
  a.x = x; a.dt = dt; a.z = z; a.ldx = ldx; a.lddt = lddt; a.ldz = ldz; a.B = B; a.C = C;
  a.ldbc = ldbc; a.A = A; a.D = D; a.bias = dt_bias; a.lens = seq_lens; a.carry_in = carry;
  a.dy = dy; a.dh_final = dh_final; a.dx = dx; a.lddx = lddx; a.ddt = ddt; a.ldddt = ldddt;
  a.dz = dz; a.lddz = lddz; a.dB = dB; a.dC = dC; a.lddbc = lddbc; a.dA = dA; a.dD = dD;
  a.dbias = ddt_bias; a.dh_init = dh_init; a.ws = ws;
  a.Bt = (int)d.Bt; a.T = (int)d.T; a.Ch = (int)d.HP; a.N = (int)d.N; a.G = (int)d.G;
  return hip_status(launch_sscan_backward(d.bf16, a, stream), "selective_scan_backward launch");
}

swimba_status swimba_selective_step(const swimba_dims* dims, const void* x, int64_t ldx,
                                    const void* dt, int64_t lddt, const void* z, int64_t ldz,
                                    const void* B, const void* C, int64_t ldbc, const float* A,
                                    const float* D, const float* dt_bias, const float* h_prev,
                                    float* h, void* y, hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  if (d.T != 1) return fail(SWIMBA_ERR_DIMS, "selective_step takes one token: seqlen must be 1");
  CHECK(check_scan(d));
  CHECK_LD(ldx, d.HP);
  CHECK_LD(lddt, d.HP);
  if (z) CHECK_LD(ldz, d.HP);
  CHECK_LD(ldbc, d.GN);
  if (d.Bt == 0) return SWIMBA_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(dt);
  OPTIONAL_PTR(z);
  REQUIRE_PTR(B);
  REQUIRE_PTR(C);
  REQUIRE_PTR(A);
  OPTIONAL_PTR(D);
  OPTIONAL_PTR(dt_bias);
  REQUIRE_PTR(h_prev);
  REQUIRE_PTR(h);
  REQUIRE_PTR(y);
  SScanArgs a{};
  a.x = x; a.dt = dt; a.z = z; a.ldx = ldx; a.lddt = lddt; a.ldz = ldz; a.B = B; a.C = C;
  a.ldbc = ldbc; a.A = A; a.D = D; a.bias = dt_bias; a.h_prev = h_prev; a.h = h; a.y = y;
  a.Bt = (int)d.Bt; a.T = 1; a.Ch = (int)d.HP; a.N = (int)d.N; a.G = (int)d.G;
  return hip_status(launch_sscan_step(d.bf16, a, stream), "selective_step launch");
}

swimba_status swimba_cross_entropy(const swimba_dims* dims, const void* x, const void* w,
                                   const int32_t* targets, float* loss, float* lse, void* ws,
                                   size_t ws_bytes, hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  CHECK(check_loss(d));
  if (d.M == 0) return SWIMBA_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w);
  REQUIRE_PTR(targets);
  REQUIRE_PTR(loss);
  REQUIRE_PTR(lse);
  CHECK(check_ws(ws, ws_bytes, ssm_ws(d, SWIMBA_SSM_CROSS_ENTROPY)));
  return hip_status(launch_xent(d.bf16, (int)d.M, (int)d.D, (int)d.HP, x, w, targets, loss, lse,
                                ws, stream),
                    "cross_entropy launch");
}

swimba_status swimba_cross_entropy_backward(const swimba_dims* dims, const void* x, const void* w,
                                            const int32_t* targets, const float* lse,
                                            const float* dloss, float* dx, float* dw, void* ws,
                                            size_t ws_bytes, hipStream_t stream) {
  Dims d;
  CHECK(read_dims(dims, d));
  CHECK(check_loss(d));
  REQUIRE_PTR(dw);
  if (d.M == 0)
    return hip_status(launch_fill_zero(dw, (size_t)(d.HP * d.D), stream),
                      "cross_entropy_backward launch");
  REQUIRE_PTR(x);
  REQUIRE_PTR(w);
  REQUIRE_PTR(targets);
  REQUIRE_PTR(lse);
  REQUIRE_PTR(dloss);
  REQUIRE_PTR(dx);
  CHECK(check_ws(ws, ws_bytes, ssm_ws(d, SWIMBA_SSM_CROSS_ENTROPY_BACKWARD)));
  const int M = (int)d.M, D = (int)d.D, V = (int)d.HP, piece = (int)xent_piece(d);
  const size_t es = d.bf16 ? 2 : 4;
  const int numbers = xent_numbers(d);
  unsigned char* dz = static_cast<unsigned char*>(ws);
  unsigned char* rows = dz + xent_dz_bytes(d, piece);
  unsigned char* part = rows + xent_rows_bytes(d);
  hipError_t e = launch_xent_rows(d.bf16, M, D, V, x, targets, rows, stream);
  if (e != hipSuccess) return hip_status(e, "cross_entropy_backward rows launch");
  for (int v0 = 0; v0 < V; v0 += piece) {
    const int nv = std::min(piece, V - v0), ld = (int)round8(nv);
    const void* wp = static_cast<const unsigned char*>(w) + (size_t)v0 * D * es;
    e = launch_xent_dz(d.bf16, M, D, V, v0, nv, x, wp, targets, lse, dloss, dz, stream);
    if (e != hipSuccess) return hip_status(e, "cross_entropy_backward dz launch");
    e = launch_dense_nn(d.bf16, "cross_entropy_dx", M, ld, D, dz, numbers, wp, dx, part, stream, nv,
                        v0 > 0);
    if (e != hipSuccess) return hip_status(e, "cross_entropy_backward dx launch");
    e = launch_dense_tn(d.bf16, "cross_entropy_dw", M, nv, D, dz, numbers, rows, dw + (size_t)v0 * D,
                        part, stream, ld);
    if (e != hipSuccess) return hip_status(e, "cross_entropy_backward dw launch");
  }
  return SWIMBA_OK;
}

}  // extern "C"
