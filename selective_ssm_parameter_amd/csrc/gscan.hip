// Gated linear recurrence over channels (swimba_layers.h), forward, backward
// and one token:
//   f = sigmoid(forget), g = 1 - f, h_t = f h_{t-1} + g x_t, y = h silu(gate);
//   e_t = dy silu(gate) + f_{t+1} e_{t+1},  dx = g e,  dforget = f g e (h_{t-1} - x),
//   dgate = dy h silu'(gate).
// A run of tokens maps the state that enters it to P h + S, with P the product
// of its f: runs are composed as (P_a P_b, S_b + P_b S_a), which is how threads,
// waves and chunks are joined (chunks of 256 tokens x 64 channels per
// workgroup; a thread holds 32 elements, so a chunk is read once per pass and
// its tokens are walked in registers).
//
// The steps keep their relative precision where f is near 1 (a memory of many
// tokens) and near 0 (a reset): with small = min(f, g) = t / (1 + t), t =
// exp(-|forget|), a step is h + g (x - h) while g is the smaller one and
// x - f (x - h) otherwise; the pair is kept as k = small with forget's sign.
// P is kept the same way: 1 - P (as G) next to P, and the one that is not
// close to 1 is used.
#include "common.hpp"
#include "layers.hpp"

namespace swimba {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kChunk = 256;   // tokens per chunk
constexpr int kCh = 64;       // channels per workgroup
constexpr int kTh = 512;      // threads per workgroup
constexpr int kEl = kChunk * kCh / kTh;  // elements per thread

// Thread layout for VEC channels per access: LC lanes cover the workgroup's 64
// channels, TG groups of TPT consecutive tokens cover the chunk.
template <int VEC>
struct Lay {
  static constexpr int LC = kCh / VEC, TG = kTh / LC, TPT = kChunk / TG, GW = 64 / LC;
  static_assert(TPT * VEC == kEl, "elements per thread");
};

template <typename T, int VEC> struct Raw {
  typedef T t __attribute__((ext_vector_type(VEC)));
};
template <typename T> struct Raw<T, 1> {
  struct t {
    T v;
    __device__ T operator[](int) const { return v; }
  };
};
template <typename T, int VEC>
__device__ __forceinline__ typename Raw<T, VEC>::t load_raw(const T* p) {
  return *reinterpret_cast<const typename Raw<T, VEC>::t*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T* p, const float* v) {
  if constexpr (VEC == 1) {
    p[0] = from_f32<T>(v[0]);
  } else {
    typename Raw<T, VEC>::t r;
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] = from_f32<T>(v[j]);
    *reinterpret_cast<typename Raw<T, VEC>::t*>(p) = r;
  }
}

// small = min(f, 1 - f) with the sign of the logit: + where g = 1 - f is small.
__device__ __forceinline__ float gate_of(float fl) {
  const float t = __builtin_amdgcn_exp2f(-fabsf(fl) * kLog2e);
  return __builtin_copysignf(t * __builtin_amdgcn_rcpf(1.f + t), fl);
}
__device__ __forceinline__ bool neg(float k) { return __builtin_signbit(k); }
// h <- f h + g x
__device__ __forceinline__ float step(float k, float x, float h) {
  return __builtin_fmaf(k, x - h, neg(k) ? x : h);
}
__device__ __forceinline__ float forget_of(float k) { return neg(k) ? -k : 1.f - k; }
// f e: e - g e while g is the smaller one
__device__ __forceinline__ float decay(float k, float e) {
  return __builtin_fmaf(-k, e, neg(k) ? 0.f : e);
}
// g e
__device__ __forceinline__ float inject(float k, float e) {
  return __builtin_fmaf(k, e, neg(k) ? e : 0.f);
}
__device__ __forceinline__ float sigm(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// A run of tokens as a map of the state entering it: h -> P h + S, G = 1 - P.
struct Run {
  float G, P, S;
};
__device__ __forceinline__ Run identity() { return Run{0.f, 1.f, 0.f}; }
__device__ __forceinline__ float apply(const Run& r, float h) {
  return r.S + (r.G <= 0.5f ? __builtin_fmaf(-r.G, h, h) : r.P * h);
}
// a, then b
__device__ __forceinline__ Run join(const Run& a, const Run& b) {
  return Run{__builtin_fmaf(-a.G, b.G, a.G + b.G), a.P * b.P, apply(b, a.S)};
}
__device__ __forceinline__ Run shfl_up(const Run& r, int d) {
  return Run{__shfl_up(r.G, d), __shfl_up(r.P, d), __shfl_up(r.S, d)};
}
__device__ __forceinline__ Run shfl_down(const Run& r, int d) {
  return Run{__shfl_down(r.G, d), __shfl_down(r.P, d), __shfl_down(r.S, d)};
}

__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int T) {
  if (!lens) return T;
  const int n = lens[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// What precedes this thread's tokens within the chunk (exclusive run), per
// channel, and the whole chunk's run. REV: runs are joined from the last token
// backwards (the backward's direction).
template <int VEC, bool REV>
__device__ __forceinline__ void chunk_runs(const Run (&own)[VEC], Run (&excl)[VEC],
                                           Run (&total)[VEC], float (&sh)[3][8][kCh]) {
  typedef Lay<VEC> L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cl = lane % L::LC;
  Run incl[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) incl[j] = own[j];
#pragma unroll
  for (int d = L::LC; d < 64; d *= 2) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const Run o = REV ? shfl_down(incl[j], d) : shfl_up(incl[j], d);
      const bool ok = REV ? lane + d < 64 : lane >= d;
      const Run n = join(o, incl[j]);
      if (ok) incl[j] = n;
    }
  }
  // the wave's run is in its last (REV: first) token group
  const bool last = REV ? lane < L::LC : lane >= 64 - L::LC;
  __syncthreads();  // sh is no longer read
  if (last) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      sh[0][wave][cl * VEC + j] = incl[j].G;
      sh[1][wave][cl * VEC + j] = incl[j].P;
      sh[2][wave][cl * VEC + j] = incl[j].S;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    Run ex = identity();
    if constexpr (L::GW > 1) {
      const Run o = REV ? shfl_down(incl[j], L::LC) : shfl_up(incl[j], L::LC);
      const bool first = REV ? lane >= 64 - L::LC : lane < L::LC;
      if (!first) ex = o;
    }
    Run before = identity(), all = identity();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int w = REV ? 7 - q : q;
      const Run r{sh[0][w][cl * VEC + j], sh[1][w][cl * VEC + j], sh[2][w][cl * VEC + j]};
      if (w == wave) before = all;
      all = join(all, r);
    }
    excl[j] = join(before, ex);
    total[j] = all;
  }
}

// Tokens of the chunk that this thread holds and whether its channels exist.
template <int VEC>
struct Place {
  int b, chunk, c, t0, len;  // c: first channel; t0: first token within the sequence
  size_t cw;                 // row of the chunk among all sequences' chunks
  bool on;
  __device__ Place(const GScanArgs& A) {
    typedef Lay<VEC> L;
    const unsigned ncb = (A.C + kCh - 1) / kCh;  // chunks run slowest, then sequences
    const unsigned q = blockIdx.x / ncb;
    b = q % A.Bt;
    chunk = q / A.Bt;
    cw = (size_t)b * ((A.T + kChunk - 1) / kChunk) + chunk;
    c = (blockIdx.x - q * ncb) * kCh + (threadIdx.x % L::LC) * VEC;
    t0 = chunk * kChunk + (threadIdx.x / L::LC) * L::TPT;
    len = seq_len(A.lens, b, A.T);
    on = c < A.C;
  }
};

// ---------------------------------------------------------------- forward

// Pass 1: each chunk's run, to ws [Bt][chunks][3][C].
template <typename T, int VEC>
__global__ __launch_bounds__(kTh) void gscan_runs_kernel(GScanArgs A) {
  typedef Lay<VEC> L;
  __shared__ float sh[3][8][kCh];
  const Place<VEC> p(A);
  const T* x = static_cast<const T*>(A.x);
  const T* f = static_cast<const T*>(A.f);
  Run own[VEC], excl[VEC], total[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) own[j] = identity();
#pragma unroll
  for (int i = 0; i < L::TPT; ++i) {
    if (p.on && p.t0 + i < p.len) {
      const size_t off = ((size_t)p.b * A.T + p.t0 + i) * A.ld + p.c;
      const auto xr = load_raw<T, VEC>(x + off);
      const auto fr = load_raw<T, VEC>(f + off);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float k = gate_of(to_f32(fr[j]));
        const float g = neg(k) ? 1.f + k : k;
        own[j].G = __builtin_fmaf(g, 1.f - own[j].G, own[j].G);
        own[j].P *= forget_of(k);
        own[j].S = step(k, to_f32(xr[j]), own[j].S);
      }
    }
  }
  chunk_runs<VEC, false>(own, excl, total, sh);
  if (p.on && threadIdx.x < L::LC) {
    float* w = static_cast<float*>(A.ws) + p.cw * 3 * A.C + p.c;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[j] = total[j].G;
      w[A.C + j] = total[j].P;
      w[2 * (size_t)A.C + j] = total[j].S;
    }
  }
}

// Pass 2: the state entering each chunk (REV: the gradient leaving it), by
// walking the chunks' runs; written over the runs' S.
template <bool REV>
__global__ __launch_bounds__(64) void gscan_carry_kernel(float* ws, int nc, int C,
                                                         const float* init, float* final_out,
                                                         float* carry) {
  const int ncb = (C + 63) / 64, b = blockIdx.x / ncb;
  const int c = (blockIdx.x - b * ncb) * 64 + threadIdx.x;
  if (c >= C) return;
  float h = init ? init[(size_t)b * C + c] : 0.f;
  for (int q = 0; q < nc; ++q) {
    const int i = REV ? nc - 1 - q : q;
    float* w = ws + ((size_t)b * nc + i) * 3 * C + c;
    const Run r{w[0], w[C], w[2 * (size_t)C]};
    w[2 * (size_t)C] = h;
    if (carry) carry[((size_t)b * nc + i) * C + c] = h;
    h = apply(r, h);
  }
  if (final_out) final_out[(size_t)b * C + c] = h;
}

// Pass 3: the outputs of each chunk from the state entering it.
template <typename T, int VEC>
__global__ __launch_bounds__(kTh) void gscan_out_kernel(GScanArgs A) {
  typedef Lay<VEC> L;
  __shared__ float sh[3][8][kCh];
  const Place<VEC> p(A);
  const T* x = static_cast<const T*>(A.x);
  const T* f = static_cast<const T*>(A.f);
  const T* o = static_cast<const T*>(A.o);
  T* y = static_cast<T*>(A.y);
  float k[L::TPT][VEC], xv[L::TPT][VEC];
  Run own[VEC], excl[VEC], total[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) own[j] = identity();
#pragma unroll
  for (int i = 0; i < L::TPT; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) k[i][j] = xv[i][j] = 0.f;
    if (p.on && p.t0 + i < p.len) {
      const size_t off = ((size_t)p.b * A.T + p.t0 + i) * A.ld + p.c;
      const auto xr = load_raw<T, VEC>(x + off);
      const auto fr = load_raw<T, VEC>(f + off);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        k[i][j] = gate_of(to_f32(fr[j]));
        xv[i][j] = to_f32(xr[j]);
        const float g = neg(k[i][j]) ? 1.f + k[i][j] : k[i][j];
        own[j].G = __builtin_fmaf(g, 1.f - own[j].G, own[j].G);
        own[j].P *= forget_of(k[i][j]);
        own[j].S = step(k[i][j], xv[i][j], own[j].S);
      }
    }
  }
  chunk_runs<VEC, false>(own, excl, total, sh);
  if (!p.on) return;
  const float* w = static_cast<const float*>(A.ws) + p.cw * 3 * A.C + p.c;
  float h[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) h[j] = apply(excl[j], w[2 * (size_t)A.C + j]);
#pragma unroll
  for (int i = 0; i < L::TPT; ++i) {
    if (p.t0 + i >= A.T) continue;
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = 0.f;
    if (p.t0 + i < p.len) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = h[j] = step(k[i][j], xv[i][j], h[j]);
      if (o) {
        const auto orow = load_raw<T, VEC>(o + ((size_t)p.b * A.T + p.t0 + i) * A.ld + p.c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float ov = to_f32(orow[j]);
          v[j] *= ov * sigm(ov);
        }
      }
    }
    store_raw<T, VEC>(y + ((size_t)p.b * A.T + p.t0 + i) * A.C + p.c, v);
  }
}

// ---------------------------------------------------------------- backward

// The gradient that reaches h_t from y_t, dy silu(gate), for one row.
template <typename T, int VEC>
__device__ __forceinline__ void dh_of(const T* dy, const T* o, float* u) {
  const auto dr = load_raw<T, VEC>(dy);
#pragma unroll
  for (int j = 0; j < VEC; ++j) u[j] = to_f32(dr[j]);
  if (o) {
    const auto orow = load_raw<T, VEC>(o);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float ov = to_f32(orow[j]);
      u[j] *= ov * sigm(ov);
    }
  }
}

// Walking back, c = f_t e_t is the gradient that leaves token t for the state
// before it: c <- f (u + c).
template <typename T, int VEC>
__global__ __launch_bounds__(kTh) void gscan_bwd_runs_kernel(GScanArgs A) {
  typedef Lay<VEC> L;
  __shared__ float sh[3][8][kCh];
  const Place<VEC> p(A);
  const T* f = static_cast<const T*>(A.f);
  const T* o = static_cast<const T*>(A.o);
  const T* dy = static_cast<const T*>(A.dy);
  Run own[VEC], excl[VEC], total[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) own[j] = identity();
#pragma unroll
  for (int i = L::TPT - 1; i >= 0; --i) {
    if (p.on && p.t0 + i < p.len) {
      const size_t row = (size_t)p.b * A.T + p.t0 + i;
      const auto fr = load_raw<T, VEC>(f + row * A.ld + p.c);
      float u[VEC];
      dh_of<T, VEC>(dy + row * A.C + p.c, o ? o + row * A.ld + p.c : nullptr, u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float k = gate_of(to_f32(fr[j]));
        const float g = neg(k) ? 1.f + k : k;
        own[j].G = __builtin_fmaf(g, 1.f - own[j].G, own[j].G);
        own[j].P *= forget_of(k);
        own[j].S = decay(k, u[j] + own[j].S);
      }
    }
  }
  chunk_runs<VEC, true>(own, excl, total, sh);
  if (p.on && threadIdx.x < L::LC) {
    float* w = static_cast<float*>(A.ws) + p.cw * 3 * A.C + p.c;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[j] = total[j].G;
      w[A.C + j] = total[j].P;
      w[2 * (size_t)A.C + j] = total[j].S;
    }
  }
}

template <typename T, int VEC>
__global__ __launch_bounds__(kTh) void gscan_bwd_out_kernel(GScanArgs A) {
  typedef Lay<VEC> L;
  __shared__ float sh[3][8][kCh];
  const Place<VEC> p(A);
  const T* x = static_cast<const T*>(A.x);
  const T* f = static_cast<const T*>(A.f);
  const T* o = static_cast<const T*>(A.o);
  const T* dy = static_cast<const T*>(A.dy);
  T* dx = static_cast<T*>(A.dx);
  T* df = static_cast<T*>(A.df);
  T* d_o = static_cast<T*>(A.d_o);
  float k[L::TPT][VEC], xv[L::TPT][VEC], u[L::TPT][VEC];
  Run fw[VEC], bw[VEC], fex[VEC], bex[VEC], total[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) fw[j] = bw[j] = identity();
#pragma unroll
  for (int i = 0; i < L::TPT; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) k[i][j] = xv[i][j] = u[i][j] = 0.f;
    if (p.on && p.t0 + i < p.len) {
      const size_t row = (size_t)p.b * A.T + p.t0 + i;
      const auto xr = load_raw<T, VEC>(x + row * A.ld + p.c);
      const auto fr = load_raw<T, VEC>(f + row * A.ld + p.c);
      dh_of<T, VEC>(dy + row * A.C + p.c, o ? o + row * A.ld + p.c : nullptr, u[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        k[i][j] = gate_of(to_f32(fr[j]));
        xv[i][j] = to_f32(xr[j]);
        const float g = neg(k[i][j]) ? 1.f + k[i][j] : k[i][j];
        fw[j].G = __builtin_fmaf(g, 1.f - fw[j].G, fw[j].G);
        fw[j].P *= forget_of(k[i][j]);
        fw[j].S = step(k[i][j], xv[i][j], fw[j].S);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    bw[j].G = fw[j].G;
    bw[j].P = fw[j].P;
  }
#pragma unroll
  for (int i = L::TPT - 1; i >= 0; --i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) bw[j].S = decay(k[i][j], u[i][j] + bw[j].S);
  chunk_runs<VEC, false>(fw, fex, total, sh);
  chunk_runs<VEC, true>(bw, bex, total, sh);
  if (!p.on) return;
  const float* w = static_cast<const float*>(A.ws) + p.cw * 3 * A.C + p.c;
  float h[VEC], c[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    h[j] = apply(fex[j], A.carry_in[p.cw * A.C + p.c + j]);
    c[j] = apply(bex[j], w[2 * (size_t)A.C + j]);
  }
  // e_t backwards: u becomes e
#pragma unroll
  for (int i = L::TPT - 1; i >= 0; --i) {
    if (p.t0 + i < p.len) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        u[i][j] += c[j];
        c[j] = decay(k[i][j], u[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < L::TPT; ++i) {
    if (p.t0 + i >= A.T) continue;
    const size_t row = (size_t)p.b * A.T + p.t0 + i;
    float vx[VEC], vf[VEC], vo[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) vx[j] = vf[j] = vo[j] = 0.f;
    if (p.t0 + i < p.len) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float kk = k[i][j], a = fabsf(kk), e = u[i][j];
        vx[j] = inject(kk, e);
        vf[j] = __builtin_fmaf(-a, a, a) * e * (h[j] - xv[i][j]);
        h[j] = step(kk, xv[i][j], h[j]);
      }
      if (o) {
        const auto orow = load_raw<T, VEC>(o + row * A.ld + p.c);
        const auto dr = load_raw<T, VEC>(dy + row * A.C + p.c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float ov = to_f32(orow[j]), sg = sigm(ov);
          vo[j] = to_f32(dr[j]) * h[j] * (sg * __builtin_fmaf(ov, 1.f - sg, 1.f));
        }
      }
    }
    store_raw<T, VEC>(dx + row * A.ldd + p.c, vx);
    store_raw<T, VEC>(df + row * A.ldd + p.c, vf);
    if (o) store_raw<T, VEC>(d_o + row * A.ldd + p.c, vo);
  }
}

// ---------------------------------------------------------------- one token

template <typename T, int VEC>
__global__ __launch_bounds__(256) void gscan_step_kernel(const T* __restrict__ x,
                                                         const T* __restrict__ f,
                                                         const T* __restrict__ o, int64_t ld,
                                                         const float* h_prev, float* h,
                                                         T* __restrict__ y, int Bt, int C) {
  const int ng = C / VEC;
  const size_t q = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t b = q / ng;
  if (b >= (size_t)Bt) return;
  const int c = (int)(q - b * ng) * VEC;
  const auto xr = load_raw<T, VEC>(x + b * ld + c);
  const auto fr = load_raw<T, VEC>(f + b * ld + c);
  typename Raw<T, VEC>::t orow = xr;
  if (o) orow = load_raw<T, VEC>(o + b * ld + c);
  float hv[VEC], v[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) hv[j] = h_prev[b * C + c + j];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    v[j] = hv[j] = step(gate_of(to_f32(fr[j])), to_f32(xr[j]), hv[j]);
    if (o) {
      const float ov = to_f32(orow[j]);
      v[j] *= ov * sigm(ov);
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) h[b * C + c + j] = hv[j];
  store_raw<T, VEC>(y + b * C + c, v);
}

// ---------------------------------------------------------------- launch

// 16-byte accesses need rows that start on 16 bytes and whole groups of channels.
template <typename T>
bool rows_aligned(int C, int64_t ld, int64_t ldd) {
  constexpr int V = 16 / (int)sizeof(T);
  return C % V == 0 && ld % V == 0 && ldd % V == 0;
}

template <typename T, int VEC>
hipError_t fwd_t(const GScanArgs& A, hipStream_t s) {
  const int nc = gscan_chunks(A.T);
  const unsigned ncb = (unsigned)((A.C + kCh - 1) / kCh);
  const dim3 grid(ncb * (unsigned)nc * (unsigned)A.Bt);
  hipEvent_t e0, e1;
  prof_kernel("gated_scan_runs", &e0, &e1);
  hipExtLaunchKernelGGL((gscan_runs_kernel<T, VEC>), grid, dim3(kTh), 0, s, e0, e1, 0, A);
  prof_kernel("gated_scan_carry", &e0, &e1);
  hipExtLaunchKernelGGL(gscan_carry_kernel<false>, dim3(ncb * (unsigned)A.Bt), dim3(64), 0, s,
                        e0, e1, 0, (float*)A.ws, nc, A.C, A.h_init, A.h_final, A.carry);
  prof_kernel("gated_scan", &e0, &e1);
  hipExtLaunchKernelGGL((gscan_out_kernel<T, VEC>), grid, dim3(kTh), 0, s, e0, e1, 0, A);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t bwd_t(const GScanArgs& A, hipStream_t s) {
  const int nc = gscan_chunks(A.T);
  const unsigned ncb = (unsigned)((A.C + kCh - 1) / kCh);
  const dim3 grid(ncb * (unsigned)nc * (unsigned)A.Bt);
  hipEvent_t e0, e1;
  prof_kernel("gated_scan_bwd_runs", &e0, &e1);
  hipExtLaunchKernelGGL((gscan_bwd_runs_kernel<T, VEC>), grid, dim3(kTh), 0, s, e0, e1, 0, A);
  prof_kernel("gated_scan_bwd_carry", &e0, &e1);
  hipExtLaunchKernelGGL(gscan_carry_kernel<true>, dim3(ncb * (unsigned)A.Bt), dim3(64), 0, s,
                        e0, e1, 0, (float*)A.ws, nc, A.C, A.dh_final, A.dh_init, (float*)nullptr);
  prof_kernel("gated_scan_bwd", &e0, &e1);
  hipExtLaunchKernelGGL((gscan_bwd_out_kernel<T, VEC>), grid, dim3(kTh), 0, s, e0, e1, 0, A);
  return hipGetLastError();
}

}  // namespace

int gscan_chunks(int T) { return (T + kChunk - 1) / kChunk; }

int64_t gscan_blocks(int64_t Bt, int64_t T, int64_t C) {
  return Bt * ((T + kChunk - 1) / kChunk) * ((C + kCh - 1) / kCh);
}

size_t gscan_ws_bytes(int Bt, int T, int C) {
  return sizeof(float) * 3 * (size_t)Bt * gscan_chunks(T) * C;
}

hipError_t launch_gscan(bool is_bf16, const GScanArgs& a, hipStream_t s) {
  if (is_bf16)
    return rows_aligned<bf16>(a.C, a.ld, 0) ? fwd_t<bf16, 8>(a, s) : fwd_t<bf16, 1>(a, s);
  return rows_aligned<float>(a.C, a.ld, 0) ? fwd_t<float, 4>(a, s) : fwd_t<float, 1>(a, s);
}

hipError_t launch_gscan_backward(bool is_bf16, const GScanArgs& a, hipStream_t s) {
  if (is_bf16)
    return rows_aligned<bf16>(a.C, a.ld, a.ldd) ? bwd_t<bf16, 8>(a, s) : bwd_t<bf16, 1>(a, s);
  return rows_aligned<float>(a.C, a.ld, a.ldd) ? bwd_t<float, 4>(a, s) : bwd_t<float, 1>(a, s);
}

hipError_t launch_gscan_step(bool is_bf16, const void* x, const void* f, const void* o, int64_t ld,
                             const float* h_prev, float* h, void* y, int Bt, int C,
                             hipStream_t s) {
  hipEvent_t e0, e1;
  prof_kernel("gated_step", &e0, &e1);
  auto go = [&](auto tag, auto vec) {
    typedef decltype(tag) T;
    constexpr int VEC = decltype(vec)::value;
    const dim3 grid((unsigned)(((size_t)Bt * (C / VEC) + 255) / 256));
    hipExtLaunchKernelGGL((gscan_step_kernel<T, VEC>), grid, dim3(256), 0, s, e0, e1, 0,
                          (const T*)x, (const T*)f, (const T*)o, ld, h_prev, h, (T*)y, Bt, C);
  };
  if (is_bf16) {
    if (rows_aligned<bf16>(C, ld, 0)) go(bf16(), std::integral_constant<int, 4>());
    else go(bf16(), std::integral_constant<int, 1>());
  } else {
    if (rows_aligned<float>(C, ld, 0)) go(0.f, std::integral_constant<int, 4>());
    else go(0.f, std::integral_constant<int, 1>());
  }
  return hipGetLastError();
}

}  // namespace swimba
