// Causal convolution over the tokens of each channel (swimba_ssm.h), forward,
// backward and one token:
//   s_t = bias + sum_k w[k] x_{t-W+1+k},  y = act(s);
//   ds = dy act'(s),  dx_t = sum_k w[k] ds_{t+W-1-k},  dw[k] = sum_t ds_t x_{t-W+1+k}.
// Bound by HBM: a thread owns 16 bytes of channels (backward: 8; one element where
// rows do not allow it) and walks a run of tokens with the last W inputs (backward:
// and the last W ds) in registers, the next 8 (4) rows requested while as many are
// computed; only the W - 1 rows at the ends of a run are read twice. The backward recomputes s,
// so the forward keeps nothing. Sums over tokens: a run's in registers, the runs'
// in a second kernel, in order. bf16, W = 4: 4 x 8192 x 4096 forward 108 us (5.0 TB/s),
// padded 8 x 2048 x 1536 forward 16, backward 30, sums 5 us; 256 x 4096 one token 5 us.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "ssm.hpp"
#include "ssm_plan.hpp"

namespace swimba {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

template <typename T, int VEC> struct Raw {
  typedef T t __attribute__((ext_vector_type(VEC)));
};
template <typename T> struct Raw<T, 1> {
  struct t {
    T v;
    __device__ T& operator[](int) { return v; }
    __device__ T operator[](int) const { return v; }
  };
};
template <typename T, int VEC> using Vt = typename Raw<T, VEC>::t;
template <typename T, int VEC>
__device__ __forceinline__ Vt<T, VEC> load_raw(const T* p) {
  return *reinterpret_cast<const Vt<T, VEC>*>(p);
}
// NT: past the L2's reuse order, where rows start on 128-byte lines (nothing here
// reads them again; a hint only): 8 x 2048 x 1536 forward 19.5 -> 16.7 us, backward
// 41 -> 38 when it was measured. (As a test at each store it gained nothing.)
template <typename T, int VEC, bool NT = false>
__device__ __forceinline__ void store_raw(T* p, const float* v) {
  Vt<T, VEC> r;
#pragma unroll
  for (int j = 0; j < VEC; ++j) r[j] = from_f32<T>(v[j]);
  if constexpr (NT && VEC > 1) __builtin_nontemporal_store(r, reinterpret_cast<Vt<T, VEC>*>(p));
  else *reinterpret_cast<Vt<T, VEC>*>(p) = r;
}
template <typename T, int VEC>
__device__ __forceinline__ Vt<T, VEC> zero_raw() {
  Vt<T, VEC> r;
#pragma unroll
  for (int j = 0; j < VEC; ++j) r[j] = from_f32<T>(0.f);
  return r;
}
template <int VEC>
__device__ __forceinline__ void store_f32(float* p, const float* v) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) p[j] = v[j];
}

__device__ __forceinline__ float sigm(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// What a thread of a pass over runs of tokens works on.
struct Run {
  int b, t0, len, c;
  size_t index;
};
template <int VEC>
__device__ __forceinline__ bool run_of(const ConvArgs& A, Run& r) {
  const unsigned nv = A.C / VEC, runs = (A.T + A.run - 1) / A.run;
  const size_t q = (size_t)blockIdx.x * 256 + threadIdx.x;
  r.index = q / nv;
  if (r.index >= (size_t)A.Bt * runs) return false;
  r.c = (int)(q - r.index * nv) * VEC;
  r.b = (int)(r.index / runs);
  r.t0 = (int)(r.index - (size_t)r.b * runs) * A.run;
  r.len = A.lens ? min(max(A.lens[r.b], 0), A.T) : A.T;
  return true;
}

// The weights [C, W] of a thread's channels (VEC * W elements in a row) and bias.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_weights(const ConvArgs& A, int c, float (&w)[W][VEC],
                                             float (&bias)[VEC]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const Vt<T, VEC> v = load_raw<T, VEC>(static_cast<const T*>(A.w) + (size_t)c * W + i * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[(i * VEC + j) % W][(i * VEC + j) / W] = to_f32(v[j]);
  }
  Vt<T, VEC> b = zero_raw<T, VEC>();
  if (A.bias) b = load_raw<T, VEC>(static_cast<const T*>(A.bias) + c);
#pragma unroll
  for (int j = 0; j < VEC; ++j) bias[j] = to_f32(b[j]);
}

// Input t of sequence b: x, before it the state, zeros past `len`.
template <typename T, int VEC, int W>
__device__ __forceinline__ Vt<T, VEC> input_at(const ConvArgs& A, int b, int c, int t, int len) {
  if (t >= len) return zero_raw<T, VEC>();
  if (t >= 0) return load_raw<T, VEC>(static_cast<const T*>(A.x) + ((size_t)b * A.T + t) * A.ldx + c);
  if (!A.state_in) return zero_raw<T, VEC>();
  return load_raw<T, VEC>(static_cast<const T*>(A.state_in) +
                          ((size_t)b * (W - 1) + (t + W - 1)) * A.C + c);
}

template <typename T, int VEC, int W, bool NT>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs A) {
  Run r;
  if (!run_of<VEC>(A, r)) return;
  T* y = static_cast<T*>(A.y) + (size_t)r.b * A.T * A.C + r.c;
  if (r.t0 == 0 && A.state_out) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const Vt<T, VEC> v = input_at<T, VEC, W>(A, r.b, r.c, r.len - (W - 1) + j, r.len);
      *reinterpret_cast<Vt<T, VEC>*>(static_cast<T*>(A.state_out) +
                                     ((size_t)r.b * (W - 1) + j) * A.C + r.c) = v;
    }
  }
  const int t1 = min(A.T, r.t0 + A.run), live = min(t1, r.len);
  float zeros[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) zeros[j] = 0.f;
  int t = r.t0;
  if (t < live) {
    float w[W][VEC], bias[VEC], win[W][VEC];  // win[k]: input t - W + 1 + k
    load_weights<T, VEC, W>(A, r.c, w, bias);
    Vt<T, VEC> nxt[kStep];
#pragma unroll
    for (int i = 0; i < kStep; ++i) nxt[i] = input_at<T, VEC, W>(A, r.b, r.c, t + i, live);
#pragma unroll
    for (int k = 1; k < W; ++k) {
      const Vt<T, VEC> v = input_at<T, VEC, W>(A, r.b, r.c, t - W + k, r.len);
#pragma unroll
      for (int j = 0; j < VEC; ++j) win[k][j] = to_f32(v[j]);
    }
    for (; t < live; t += kStep) {
      Vt<T, VEC> cur[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        cur[i] = nxt[i];
        nxt[i] = input_at<T, VEC, W>(A, r.b, r.c, t + kStep + i, live);
      }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        float out[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
#pragma unroll
          for (int k = 0; k + 1 < W; ++k) win[k][j] = win[k + 1][j];
          win[W - 1][j] = to_f32(cur[i][j]);
          float s = bias[j];
#pragma unroll
          for (int k = 0; k < W; ++k) s = __builtin_fmaf(w[k][j], win[k][j], s);
          out[j] = A.silu ? s * sigm(s) : s;
        }
        if (t + i < live) store_raw<T, VEC, NT>(y + (size_t)(t + i) * A.C, out);
      }
    }
  }
  for (t = max(r.t0, live); t < t1; ++t)
    store_raw<T, VEC, NT>(y + (size_t)t * A.C, zeros);
}

template <typename T, int VEC, int W, bool NT>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs A) {
  Run r;
  if (!run_of<VEC>(A, r)) return;
  const T* dy = static_cast<const T*>(A.dy) + (size_t)r.b * A.T * A.C + r.c;
  T* dx = static_cast<T*>(A.dx) + (size_t)r.b * A.T * A.lddx + r.c;
  const int t1 = min(A.T, r.t0 + A.run);
  float w[W][VEC], bias[VEC], win[W][VEC], ds[W][VEC];  // ds[k]: that of token t - W + 1 + k
  float dw[W][VEC], db[VEC];
  load_weights<T, VEC, W>(A, r.c, w, bias);
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[k][j] = ds[k][j] = db[j] = 0.f;
  // tokens of the run in use; its outputs are complete W - 1 tokens behind their end
  const int live = max(min(t1, r.len), r.t0), end = live + W - 1, last = min(r.len, end);
  const T* x = static_cast<const T*>(A.x) + (size_t)r.b * A.T * A.ldx + r.c;
  Vt<T, VEC> nx[kStepBwd], nd[kStepBwd];
  auto fetch = [&](int t) {
    if (t + kStepBwd <= last) {
#pragma unroll
      for (int i = 0; i < kStepBwd; ++i) {
        nx[i] = load_raw<T, VEC>(x + (size_t)(t + i) * A.ldx);
        nd[i] = load_raw<T, VEC>(dy + (size_t)(t + i) * A.C);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kStepBwd; ++i) {
        nx[i] = nd[i] = zero_raw<T, VEC>();
        if (t + i < last) {
          nx[i] = load_raw<T, VEC>(x + (size_t)(t + i) * A.ldx);
          nd[i] = load_raw<T, VEC>(dy + (size_t)(t + i) * A.C);
        }
      }
    }
  };
  fetch(r.t0);
#pragma unroll
  for (int k = 1; k < W; ++k) {
    const Vt<T, VEC> v = input_at<T, VEC, W>(A, r.b, r.c, r.t0 - W + k, r.len);
#pragma unroll
    for (int j = 0; j < VEC; ++j) win[k][j] = to_f32(v[j]);
  }
  // One token: INNER where it and the output that it completes lie within the run and
  // before the inputs that the state behind the sequence holds.
  auto token = [&](int tt, const Vt<T, VEC>& xv, const Vt<T, VEC>& dv, auto inner) {
    constexpr bool INNER = decltype(inner)::value;
    const int out = tt - (W - 1);  // ds of tt completes the gradient of input out
    const bool in = INNER || tt < r.len, mine = INNER || (tt < t1 && tt < r.len);
    float g[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
#pragma unroll
      for (int k = 0; k + 1 < W; ++k) {
        win[k][j] = win[k + 1][j];
        ds[k][j] = ds[k + 1][j];
      }
      win[W - 1][j] = to_f32(xv[j]);
      float s = bias[j];
#pragma unroll
      for (int k = 0; k < W; ++k) s = __builtin_fmaf(w[k][j], win[k][j], s);
      float d = to_f32(dv[j]);
      if (A.silu) {
        const float sg = sigm(s);
        d *= sg * __builtin_fmaf(s, 1.f - sg, 1.f);
      }
      if constexpr (!INNER) d = in ? d : 0.f;
      ds[W - 1][j] = d;
      if (mine) {
        db[j] += d;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][j] = __builtin_fmaf(d, win[k][j], dw[k][j]);
      }
      g[j] = w[0][j] * ds[W - 1][j];
#pragma unroll
      for (int k = 1; k < W; ++k) g[j] = __builtin_fmaf(w[k][j], ds[W - 1 - k][j], g[j]);
    }
    if constexpr (INNER) {
      store_raw<T, VEC, NT>(dx + (size_t)out * A.lddx, g);
      return;
    }
    // the state behind the last token holds inputs len - W + 1 .. len - 1
    const int js = out - (r.len - (W - 1));
    if (A.dstate_out && js >= 0 && js < W - 1 && tt < end) {
      const float* p = A.dstate_out + ((size_t)r.b * (W - 1) + js) * A.C + r.c;
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[j] += p[j];
    }
    if (out >= r.t0 && out < live) {
      store_raw<T, VEC, NT>(dx + (size_t)out * A.lddx, g);
    } else if (r.t0 == 0 && out < 0 && A.dstate_in) {
      store_f32<VEC>(A.dstate_in + ((size_t)r.b * (W - 1) + tt) * A.C + r.c, g);
    }
  };
  // (a run past the length has nothing but zeros to write, the first its state besides)
  if (live > r.t0 || r.t0 == 0) {
    for (int t = r.t0; t < end; t += kStepBwd) {
      Vt<T, VEC> cx[kStepBwd], cd[kStepBwd];
#pragma unroll
      for (int i = 0; i < kStepBwd; ++i) {
        cx[i] = nx[i];
        cd[i] = nd[i];
      }
      fetch(t + kStepBwd);
      if (t >= r.t0 + W - 1 && t + kStepBwd <= live) {
#pragma unroll
        for (int i = 0; i < kStepBwd; ++i) token(t + i, cx[i], cd[i], std::true_type());
      } else {
#pragma unroll
        for (int i = 0; i < kStepBwd; ++i) token(t + i, cx[i], cd[i], std::false_type());
      }
    }
  }
  float zeros[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) zeros[j] = 0.f;
  for (int t = live; t < t1; ++t) store_raw<T, VEC, NT>(dx + (size_t)t * A.lddx, zeros);
  float* part = A.part + r.index * (W + 1) * A.C + r.c;
#pragma unroll
  for (int k = 0; k < W; ++k) store_f32<VEC>(part + (size_t)k * A.C, dw[k]);
  store_f32<VEC>(part + (size_t)W * A.C, db);
}

// dw and db: the runs' sums added in order, 64 columns a workgroup, a sixteenth of
// the runs each wave.
__global__ __launch_bounds__(1024) void conv_sum_kernel(ConvArgs A, size_t runs) {
  __shared__ float sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const size_t cols = (size_t)(A.W + 1) * A.C, q = (size_t)blockIdx.x * 64 + lane;
  const size_t per = (runs + 15) / 16, r1 = min(runs, (wave + 1) * per);
  float v = 0.f;
  if (q < cols) {
#pragma unroll 8
    for (size_t r = wave * per; r < r1; ++r) v += A.part[r * cols + q];
  }
  sum[wave][lane] = v;
  __syncthreads();
  if (wave || q >= cols) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) v += sum[w][lane];
  const int k = (int)(q / A.C), c = (int)(q - (size_t)k * A.C);
  if (k < A.W) A.dw[(size_t)c * A.W + k] = v;
  else if (A.db) A.db[c] = v;
}

template <typename T, int VEC, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs A) {
  const unsigned nv = A.C / VEC;
  const size_t q = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t b = q / nv;
  if (b >= (size_t)A.Bt) return;
  const int c = (int)(q - b * nv) * VEC;
  Vt<T, VEC> in[W];
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
    in[k] = load_raw<T, VEC>(static_cast<const T*>(A.state_in) + (b * (W - 1) + k) * A.C + c);
  in[W - 1] = load_raw<T, VEC>(static_cast<const T*>(A.x) + b * A.ldx + c);
  float w[W][VEC], bias[VEC], out[VEC];
  load_weights<T, VEC, W>(A, c, w, bias);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    float s = bias[j];
#pragma unroll
    for (int k = 0; k < W; ++k) s = __builtin_fmaf(w[k][j], to_f32(in[k][j]), s);
    out[j] = A.silu ? s * sigm(s) : s;
  }
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
    *reinterpret_cast<Vt<T, VEC>*>(static_cast<T*>(A.state_out) + (b * (W - 1) + k) * A.C + c) =
        in[k + 1];
  store_raw<T, VEC>(static_cast<T*>(A.y) + b * A.C + c, out);
}

// The state where there are no tokens: state_in, or zeros.
template <typename T>
__global__ __launch_bounds__(256) void conv_state_kernel(const T* from, T* to, size_t n) {
  for (size_t q = (size_t)blockIdx.x * 256 + threadIdx.x; q < n; q += (size_t)gridDim.x * 256)
    to[q] = from ? from[q] : from_f32<T>(0.f);
}

// f(element type, channels per thread, width)
template <int VB, int VF, class F>
hipError_t with_kernel(bool is_bf16, int vec, int W, F f) {
  auto width = [&](auto t, auto v) {
    if (W == 2) return f(t, v, std::integral_constant<int, 2>());
    if (W == 3) return f(t, v, std::integral_constant<int, 3>());
    return f(t, v, std::integral_constant<int, 4>());
  };
  const std::integral_constant<int, 1> one{};
  if (is_bf16)
    return vec == 1 ? width(bf16(), one) : width(bf16(), std::integral_constant<int, VB>());
  return vec == 1 ? width(0.f, one) : width(0.f, std::integral_constant<int, VF>());
}

// Whether rows so many bytes apart start on 128-byte lines.
bool whole_lines(const void* p, size_t pitch) {
  return (reinterpret_cast<uintptr_t>(p) | pitch) % 128 == 0;
}

dim3 blocks_of(size_t threads) { return dim3((unsigned)((threads + 255) / 256)); }

size_t runs_of(const ConvArgs& A) { return (size_t)A.Bt * ((A.T + A.run - 1) / A.run); }

}  // namespace

size_t conv_bwd_ws_bytes(int Bt, int T, int C) {
  // the shortest runs that any strides lead to
  size_t runs = 0;
  for (int v : {1, 2, 4}) {
    const int run = run_length(Bt, T, std::max(1, C / v), kBwdThreads);
    runs = std::max(runs, (size_t)Bt * ((T + run - 1) / run));
  }
  return sizeof(float) * runs * 5 * C;
}

hipError_t launch_conv(bool is_bf16, const ConvArgs& a, hipStream_t s) {
  const int vec = vec_of(vec_fwd(is_bf16), a.C, a.ldx, 0);
  ConvArgs A = a;
  A.run = run_length(A.Bt, A.T, A.C / vec, kFwdThreads);
  return with_kernel<8, 4>(is_bf16, vec, A.W, [&](auto t, auto v, auto w) {
    auto run = [&](auto nt) {
      return launch("causal_conv", conv_kernel<decltype(t), v(), w(), nt()>,
                    blocks_of(runs_of(A) * (A.C / vec)), dim3(256), 0, s, A);
    };
    return whole_lines(A.y, A.C * sizeof(t)) ? run(std::true_type()) : run(std::false_type());
  });
}

hipError_t launch_conv_backward(bool is_bf16, const ConvArgs& a, hipStream_t s) {
  const int vec = vec_of(vec_bwd(is_bf16), a.C, a.ldx, a.lddx);
  ConvArgs A = a;
  A.run = run_length(A.Bt, A.T, A.C / vec, kBwdThreads);
  const hipError_t e = with_kernel<4, 2>(is_bf16, vec, A.W, [&](auto t, auto v, auto w) {
    auto run = [&](auto nt) {
      return launch("causal_conv_bwd", conv_bwd_kernel<decltype(t), v(), w(), nt()>,
                    blocks_of(runs_of(A) * (A.C / vec)), dim3(256), 0, s, A);
    };
    return whole_lines(A.dx, A.lddx * sizeof(t)) ? run(std::true_type()) : run(std::false_type());
  });
  if (e != hipSuccess) return e;
  const size_t cols = (size_t)(A.W + 1) * A.C;
  return launch("causal_conv_sum", conv_sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024),
                0, s, A, runs_of(A));
}

hipError_t launch_conv_state(bool is_bf16, const void* from, void* to, size_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<size_t>((n + 255) / 256, 4096));
  if (is_bf16)
    return launch("causal_conv_state", conv_state_kernel<bf16>, grid, dim3(256), 0, s,
                  (const bf16*)from, (bf16*)to, n);
  return launch("causal_conv_state", conv_state_kernel<float>, grid, dim3(256), 0, s,
                (const float*)from, (float*)to, n);
}

hipError_t launch_conv_step(bool is_bf16, const ConvArgs& A, hipStream_t s) {
  const int vec = vec_of(vec_fwd(is_bf16), A.C, A.ldx, 0);
  return with_kernel<8, 4>(is_bf16, vec, A.W, [&](auto t, auto v, auto w) {
    return launch("causal_conv_step", conv_step_kernel<decltype(t), v(), w()>,
                  blocks_of((size_t)A.Bt * (A.C / vec)), dim3(256), 0, s, A);
  });
}

}  // namespace swimba
