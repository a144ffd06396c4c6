// Layer norm over rows of D, forward and backward (swimba_layers.h).
//
// Forward, per row: s = x + residual (rounded to the stored type), mu =
// mean(s), var = mean((s - mu)^2), y = (s - mu) (var + eps)^(-1/2) w + b.
// Backward, per row, with xh = (s - mu) rstd and g = dy w: dx = dres + rstd
// (g - mean(g) - xh mean(g xh)); over the rows dw = sum dy xh, db = sum dy.
// Both are bound by HBM: a row is read once, held in registers and written
// once; the variance is a second pass over the registers, so that an offset
// common to the row does not cancel. A row takes 4 to 1024 threads, 8 elements
// each in the forward (one 16-byte access of bf16; 32768 x 2048: 91 us with 256
// threads a row, 102 with 64) and 16 in the backward, whose weight gradients
// stay in registers over all rows that a workgroup takes, with the next row's
// loads in flight; one partial row per workgroup goes to the workspace, and a
// second kernel adds the partial rows in order.
#include <algorithm>

#include "common.hpp"
#include "layers.hpp"

namespace swimba {

namespace {

// VEC consecutive elements as floats: one 16-byte access (two for 8 floats),
// or single elements where rows are not 16-byte aligned.
template <typename T, int VEC>
__device__ __forceinline__ void loadv(const T* p, float* v) {
  if constexpr (VEC == 1) {
    v[0] = to_f32(p[0]);
  } else if constexpr (VEC == 8) {
    const typename Vec<T>::x8 r = load8<T>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(r[i]);
  } else {
    const typename Vec<T>::x4 r = *reinterpret_cast<const typename Vec<T>::x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_f32(r[i]);
  }
}
// Stored past the L2's reuse order: nothing here reads it again, and the next
// kernel sees the values as those of any store (61 -> 57 us for the forward and
// backward of 16384 x 768).
template <typename T, int VEC>
__device__ __forceinline__ void storev(T* p, const float* v) {
  if constexpr (VEC == 1) {
    p[0] = from_f32<T>(v[0]);
  } else if constexpr (VEC == 8) {
    typename Vec<T>::x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = from_f32<T>(v[i]);
    if constexpr (sizeof(T) == 2) {
      __builtin_nontemporal_store(__builtin_bit_cast(int4v, r), reinterpret_cast<int4v*>(p));
    } else {
      const floatx4 lo = {r[0], r[1], r[2], r[3]}, hi = {r[4], r[5], r[6], r[7]};
      __builtin_nontemporal_store(lo, reinterpret_cast<floatx4*>(p));
      __builtin_nontemporal_store(hi, reinterpret_cast<floatx4*>(p) + 1);
    }
  } else {
    typename Vec<T>::x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = from_f32<T>(v[i]);
    __builtin_nontemporal_store(r, reinterpret_cast<typename Vec<T>::x4*>(p));
  }
}

// Sum over the NT threads of a row, in a butterfly within a wave.
template <int NT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = (NT < 64 ? NT : 64) / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = lanes_sum<NT>(v);
  if constexpr (NT > 64) {
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += red[w];
  }
  return v;
}

// Threads and rows per workgroup.
template <int NT>
struct RowCfg {
  static constexpr int TH = NT <= 64 ? 256 : NT;
  static constexpr int RP = TH / NT;
  static constexpr int NW = NT < 64 ? 1 : NT / 64;  // waves per row
};

template <typename T, int VEC, int NT, int EPT>
__global__ __launch_bounds__(RowCfg<NT>::TH) void norm_fwd_kernel(
    const T* x, const T* residual, const T* __restrict__ weight, const T* __restrict__ bias,
    float eps, T* sum, T* y, float* __restrict__ mean, float* __restrict__ rstd, int M, int D) {
  constexpr int VPT = EPT / VEC;
  __shared__ float red[RowCfg<NT>::NW];
  const int tid = threadIdx.x % NT;
  const int m = blockIdx.x * RowCfg<NT>::RP + threadIdx.x / NT;
  if (m >= M) return;  // all threads of the row, and of the workgroup where a row has it alone
  const size_t base = (size_t)m * D;
  float v[VPT][VEC];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
    if (c < D) loadv<T, VEC>(x + base + c, v[i]);
  }
  if (residual) {
    float r[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) loadv<T, VEC>(residual + base + c, r[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) {
        // the norm is of the sum as it is stored
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = to_f32(from_f32<T>(v[i][j] + r[i][j]));
        storev<T, VEC>(sum + base + c, v[i]);
      }
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += v[i][j];
  const float inv = 1.f / (float)D;
  const float mu = row_sum<NT>(s, red) * inv;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * VEC;
    if (c < D) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] -= mu;
        q += v[i][j] * v[i][j];
      }
    }
  }
  const float rs = 1.f / sqrtf(row_sum<NT>(q, red) * inv + eps);
  if (tid == 0) {
    if (mean) mean[m] = mu;
    if (rstd) rstd[m] = rs;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * VEC;
    if (c < D) {
      float w[VEC], b[VEC];
      loadv<T, VEC>(weight + c, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) b[j] = 0.f;
      if (bias) loadv<T, VEC>(bias + c, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = v[i][j] * rs * w[j] + b[j];
      storev<T, VEC>(y + base + c, v[i]);
    }
  }
}

// Workgroup wg takes rows wg RP + sub, then every nwg RP-th row further on.
template <typename T, typename TG, int VEC, int NT, int EPT>
__global__ __launch_bounds__(RowCfg<NT>::TH) void norm_bwd_kernel(
    const T* __restrict__ s, const T* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, const TG* dy, const float* dres, float* dx,
    float* __restrict__ part, int M, int D) {
  constexpr int VPT = EPT / VEC, RP = RowCfg<NT>::RP, TH = RowCfg<NT>::TH, NW = RowCfg<NT>::NW;
  __shared__ float red[2 * NW];
  extern __shared__ float acc_sh[];  // [2][D] where several rows share the workgroup
  const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
  float w[VPT][VEC], dw[VPT][VEC], db[VPT][VEC];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = dw[i][j] = db[i][j] = 0.f;
    if (c < D) loadv<T, VEC>(weight + c, w[i]);
  }
  const float inv = 1.f / (float)D;
  struct Row {
    float s[VPT][VEC], g[VPT][VEC], r[VPT][VEC], mu, rs;
  };
  auto load = [&](Row& q, int m) {
    const size_t base = (size_t)m * D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) q.s[i][j] = q.g[i][j] = q.r[i][j] = 0.f;
      if (c < D) {
        loadv<T, VEC>(s + base + c, q.s[i]);
        loadv<TG, VEC>(dy + base + c, q.g[i]);
        if (dres) loadv<float, VEC>(dres + base + c, q.r[i]);
      }
    }
    q.mu = mean[m];
    q.rs = rstd[m];
  };
  const int step = gridDim.x * RP;
  int m = blockIdx.x * RP + sub;
  // 1024 threads have 128 registers each: no room for the next row
  constexpr bool AHEAD = NT < 1024;
  Row cur, nxt;
  if (AHEAD && m < M) load(cur, m);
  for (; m < M; m += step) {
    if constexpr (!AHEAD) load(cur, m);
    else if (m + step < M) load(nxt, m + step);
    float sg = 0.f, sx = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          cur.s[i][j] = (cur.s[i][j] - cur.mu) * cur.rs;
          dw[i][j] += cur.g[i][j] * cur.s[i][j];
          db[i][j] += cur.g[i][j];
          cur.g[i][j] *= w[i][j];
          sg += cur.g[i][j];
          sx += cur.g[i][j] * cur.s[i][j];
        }
      }
    }
    sg = lanes_sum<NT>(sg);
    sx = lanes_sum<NT>(sx);
    if constexpr (NT > 64) {
      __syncthreads();  // the previous row's sums have been read
      if ((threadIdx.x & 63) == 0) {
        red[2 * (threadIdx.x >> 6)] = sg;
        red[2 * (threadIdx.x >> 6) + 1] = sx;
      }
      __syncthreads();
      sg = sx = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        sg += red[2 * q];
        sx += red[2 * q + 1];
      }
    }
    const float mg = sg * inv, mx = sx * inv;
    const size_t base = (size_t)m * D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          cur.r[i][j] += cur.rs * (cur.g[i][j] - mg - cur.s[i][j] * mx);
        storev<float, VEC>(dx + base + c, cur.r[i]);
      }
    }
    if constexpr (AHEAD) cur = nxt;
  }
  // one partial row of dw and of db per workgroup: the rows of a wave in a
  // butterfly, then the waves (or the rows of wider groups) in order
#pragma unroll
  for (int off = NT; off < 64; off *= 2) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dw[i][j] += __shfl_xor(dw[i][j], off);
        db[i][j] += __shfl_xor(db[i][j], off);
      }
  }
  float* pw = part + (size_t)blockIdx.x * 2 * D;
  if constexpr (RP == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          pw[c + j] = dw[i][j];
          pw[D + c + j] = db[i][j];
        }
      }
    }
  } else {
    for (int r = 0; r < TH / 64; ++r) {
      if ((int)(threadIdx.x >> 6) == r && (threadIdx.x & 63) < NT) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = (i * NT + tid) * VEC;
          if (c < D) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              acc_sh[c + j] = r ? acc_sh[c + j] + dw[i][j] : dw[i][j];
              acc_sh[D + c + j] = r ? acc_sh[D + c + j] + db[i][j] : db[i][j];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * D; c += TH) pw[c] = acc_sh[c];
  }
}

// dw and db: the np partial rows added in a fixed order (32 interleaved sums
// per column, joined in order).
constexpr int kDwSums = 32;
__global__ __launch_bounds__(32 * kDwSums) void norm_dw_kernel(const float* __restrict__ part,
                                                               int np, int D,
                                                               float* __restrict__ dw,
                                                               float* __restrict__ db) {
  __shared__ float sh[kDwSums][32];
  const int cl = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cl;  // column of [dw | db]
  float a = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int p = grp; p < np; p += kDwSums) a += part[(size_t)p * 2 * D + c];
  }
  sh[grp][cl] = a;
  __syncthreads();
  if (grp == 0 && c < 2 * D) {
#pragma unroll
    for (int q = 1; q < kDwSums; ++q) a += sh[q][cl];
    if (c < D) dw[c] = a;
    else if (db) db[c - D] = a;
  }
}

template <typename T, int VEC, int NT, int EPT>
hipError_t fwd_cfg(const NormFwdArgs& a, hipStream_t s) {
  constexpr int RP = RowCfg<NT>::RP;
  return launch("layer_norm", norm_fwd_kernel<T, VEC, NT, EPT>,
                dim3((unsigned)((a.M + RP - 1) / RP)), dim3(RowCfg<NT>::TH), 0, s, (const T*)a.x,
                (const T*)a.residual, (const T*)a.weight, (const T*)a.bias, a.eps, (T*)a.sum,
                (T*)a.y, a.mean, a.rstd, a.M, a.D);
}

template <typename T, typename TG, int VEC, int NT, int EPT>
hipError_t bwd_cfg(const NormBwdArgs& a, hipStream_t s) {
  constexpr int RP = RowCfg<NT>::RP;
  const int np = norm_bwd_parts(a.M, a.D);
  const hipError_t e =
      launch("layer_norm_backward", norm_bwd_kernel<T, TG, VEC, NT, EPT>, dim3((unsigned)np),
             dim3(RowCfg<NT>::TH), RP > 1 ? 2 * a.D * sizeof(float) : 0, s, (const T*)a.s,
             (const T*)a.weight, a.mean, a.rstd, (const TG*)a.dy, a.dres, a.dx, a.part, a.M, a.D);
  if (e != hipSuccess) return e;
  return launch("layer_norm_dw", norm_dw_kernel, dim3((unsigned)((2 * a.D + 31) / 32)),
                dim3(32 * kDwSums), 0, s, a.part, np, a.D, a.dw, a.db);
}

// Threads per row for E elements each; 1024 threads then take up to 32 each.
int row_threads(int D, int E) {
  for (int nt : {4, 16, 64, 128, 256, 512})
    if (D <= nt * E) return nt;
  return 1024;
}

// CALL(threads, elements per thread) for E elements per thread.
#define SWIMBA_NORM_CFG(E, CALL)             \
  switch (row_threads(a.D, E)) {             \
    case 4: return CALL(4, E);               \
    case 16: return CALL(16, E);             \
    case 64: return CALL(64, E);             \
    case 128: return CALL(128, E);           \
    case 256: return CALL(256, E);           \
    case 512: return CALL(512, E);           \
    default: break;                          \
  }                                          \
  if (a.D <= 8192) return CALL(1024, 8);     \
  if (a.D <= 16384) return CALL(1024, 16);   \
  return CALL(1024, 32)

constexpr int kFwdE = 8, kBwdE = 16;

template <typename T, int VEC>
hipError_t fwd_t(const NormFwdArgs& a, hipStream_t s) {
#define CALL(NT, EPT) fwd_cfg<T, VEC, NT, EPT>(a, s)
  SWIMBA_NORM_CFG(kFwdE, CALL);
#undef CALL
}
template <typename T, typename TG, int VEC>
hipError_t bwd_t(const NormBwdArgs& a, hipStream_t s) {
#define CALL(NT, EPT) bwd_cfg<T, TG, VEC, NT, EPT>(a, s)
  SWIMBA_NORM_CFG(kBwdE, CALL);
#undef CALL
}

}  // namespace

// Workgroups of the backward, each with one partial row: as many as the chip
// holds at once (8 waves per CU), or fewer with at least four rows each.
int norm_bwd_parts(int M, int D) {
  const int nt = row_threads(D, kBwdE), th = nt <= 64 ? 256 : nt, rp = th / nt;
  const int64_t wgs = (M + 4 * rp - 1) / (4 * rp);
  return (int)std::min<int64_t>(std::max<int64_t>(wgs, 1), 256 * 512 / th);
}

int64_t norm_fwd_threads(int64_t M, int D) {
  const int nt = row_threads(D, kFwdE), th = nt <= 64 ? 256 : nt, rp = th / nt;
  return (M + rp - 1) / rp * th;
}

hipError_t launch_norm_fwd(bool is_bf16, const NormFwdArgs& a, hipStream_t s) {
  if (is_bf16) return a.D % 8 == 0 ? fwd_t<bf16, 8>(a, s) : fwd_t<bf16, 1>(a, s);
  return a.D % 4 == 0 ? fwd_t<float, 4>(a, s) : fwd_t<float, 1>(a, s);
}

hipError_t launch_norm_bwd(bool is_bf16, bool dy_f32, const NormBwdArgs& a, hipStream_t s) {
  if (!is_bf16)
    return a.D % 4 == 0 ? bwd_t<float, float, 4>(a, s) : bwd_t<float, float, 1>(a, s);
  if (dy_f32)
    return a.D % 8 == 0 ? bwd_t<bf16, float, 8>(a, s) : bwd_t<bf16, float, 1>(a, s);
  return a.D % 8 == 0 ? bwd_t<bf16, bf16, 8>(a, s) : bwd_t<bf16, bf16, 1>(a, s);
}

}  // namespace swimba
