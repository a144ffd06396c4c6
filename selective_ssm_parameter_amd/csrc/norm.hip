// Layer norm over rows of D, forward and backward (swimba_layers.h).
//
// Forward, per row: s = x + residual (rounded to the stored type), mu =
// mean(s), var = mean((s - mu)^2), y = (s - mu) (var + eps)^(-1/2) w + b.
// Backward, per row, with xh = (s - mu) rstd and g = dy w: dx = dres + rstd
// (g - mean(g) - xh mean(g xh)); over the rows dw = sum dy xh, db = sum dy.
// Both are bound by HBM: a row is read once, held in registers (32 elements
// per thread at most) and written once; the variance is a second pass over
// the registers, so that an offset common to the row does not cancel. The
// weight gradients stay in registers over all rows that a workgroup takes,
// one partial row per workgroup goes to the workspace, and a second kernel
// adds the partial rows in order.
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
template <typename T, int VEC>
__device__ __forceinline__ void storev(T* p, const float* v) {
  if constexpr (VEC == 1) {
    p[0] = from_f32<T>(v[0]);
  } else if constexpr (VEC == 8) {
    typename Vec<T>::x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = from_f32<T>(v[i]);
    store8<T>(p, r);
  } else {
    typename Vec<T>::x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = from_f32<T>(v[i]);
    *reinterpret_cast<typename Vec<T>::x4*>(p) = r;
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Sum over the NT threads of a row (NT = 64: one wave; else the workgroup).
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
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

// Rows per workgroup of the forward and the backward.
template <int NT>
struct RowCfg {
  static constexpr int TH = NT < 256 ? 256 : NT;  // threads per workgroup
  static constexpr int RP = TH / NT;
};

template <typename T, int VEC, int NT, int EPT>
__global__ __launch_bounds__(RowCfg<NT>::TH) void norm_fwd_kernel(
    const T* x, const T* residual, const T* __restrict__ weight, const T* __restrict__ bias,
    float eps, T* sum, T* y, float* __restrict__ mean, float* __restrict__ rstd, int M, int D) {
  constexpr int VPT = EPT / VEC;
  __shared__ float red[NT / 64];
  const int tid = threadIdx.x % NT;
  const int m = blockIdx.x * RowCfg<NT>::RP + threadIdx.x / NT;
  if (m >= M) return;  // whole waves, and whole workgroups where they share a row
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
  constexpr int VPT = EPT / VEC, RP = RowCfg<NT>::RP, TH = RowCfg<NT>::TH;
  __shared__ float red[2 * (NT / 64)];
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
  for (int m = blockIdx.x * RP + sub; m < M; m += gridDim.x * RP) {
    const size_t base = (size_t)m * D;
    float xh[VPT][VEC], g[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) xh[i][j] = g[i][j] = 0.f;
      if (c < D) {
        loadv<T, VEC>(s + base + c, xh[i]);
        loadv<TG, VEC>(dy + base + c, g[i]);
      }
    }
    const float mu = mean[m], rs = rstd[m];
    float sg = 0.f, sx = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] = (xh[i][j] - mu) * rs;
          dw[i][j] += g[i][j] * xh[i][j];
          db[i][j] += g[i][j];
          g[i][j] *= w[i][j];
          sg += g[i][j];
          sx += g[i][j] * xh[i][j];
        }
      }
    }
    sg = wave_sum(sg);
    sx = wave_sum(sx);
    if constexpr (NT > 64) {
      __syncthreads();  // the previous row's sums have been read
      if ((threadIdx.x & 63) == 0) {
        red[2 * (threadIdx.x >> 6)] = sg;
        red[2 * (threadIdx.x >> 6) + 1] = sx;
      }
      __syncthreads();
      sg = sx = 0.f;
#pragma unroll
      for (int q = 0; q < NT / 64; ++q) {
        sg += red[2 * q];
        sx += red[2 * q + 1];
      }
    }
    const float mg = sg * inv, mx = sx * inv;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) {
        float r[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) r[j] = 0.f;
        if (dres) loadv<float, VEC>(dres + base + c, r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) r[j] += rs * (g[i][j] - mg - xh[i][j] * mx);
        storev<float, VEC>(dx + base + c, r);
      }
    }
  }
  // one partial row of dw and of db per workgroup: the row groups in order
  float* pw = part + (size_t)blockIdx.x * 2 * D;
  if constexpr (RP == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c < D) {
        storev<float, VEC>(pw + c, dw[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) pw[D + c + j] = db[i][j];
      }
    }
  } else {
    for (int r = 0; r < RP; ++r) {
      if (sub == r) {
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

// dw and db: the np partial rows added in a fixed order (8 interleaved sums
// per column, joined in order).
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* __restrict__ part, int np,
                                                      int D, float* __restrict__ dw,
                                                      float* __restrict__ db) {
  __shared__ float sh[8][32];
  const int cl = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cl;  // column of [dw | db]
  float a = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int p = grp; p < np; p += 8) a += part[(size_t)p * 2 * D + c];
  }
  sh[grp][cl] = a;
  __syncthreads();
  if (grp == 0 && c < 2 * D) {
#pragma unroll
    for (int q = 1; q < 8; ++q) a += sh[q][cl];
    if (c < D) dw[c] = a;
    else if (db) db[c - D] = a;
  }
}

template <typename T, int VEC, int NT, int EPT>
hipError_t fwd_cfg(const NormFwdArgs& a, hipStream_t s) {
  constexpr int RP = RowCfg<NT>::RP;
  hipEvent_t e0, e1;
  prof_kernel("layer_norm", &e0, &e1);
  hipExtLaunchKernelGGL((norm_fwd_kernel<T, VEC, NT, EPT>), dim3((unsigned)((a.M + RP - 1) / RP)),
                        dim3(RowCfg<NT>::TH), 0, s, e0, e1, 0, (const T*)a.x,
                        (const T*)a.residual, (const T*)a.weight, (const T*)a.bias, a.eps,
                        (T*)a.sum, (T*)a.y, a.mean, a.rstd, a.M, a.D);
  return hipGetLastError();
}

template <typename T, typename TG, int VEC, int NT, int EPT>
hipError_t bwd_cfg(const NormBwdArgs& a, hipStream_t s) {
  constexpr int RP = RowCfg<NT>::RP;
  const int np = norm_bwd_parts(a.M, a.D);
  hipEvent_t e0, e1;
  prof_kernel("layer_norm_backward", &e0, &e1);
  hipExtLaunchKernelGGL((norm_bwd_kernel<T, TG, VEC, NT, EPT>), dim3((unsigned)np),
                        dim3(RowCfg<NT>::TH), RP > 1 ? 2 * a.D * sizeof(float) : 0, s, e0, e1, 0,
                        (const T*)a.s, (const T*)a.weight, a.mean, a.rstd, (const TG*)a.dy, a.dres,
                        a.dx, a.part, a.M, a.D);
  prof_kernel("layer_norm_dw", &e0, &e1);
  hipExtLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((2 * a.D + 31) / 32)), dim3(256), 0, s, e0,
                        e1, 0, a.part, np, a.D, a.dw, a.db);
  return hipGetLastError();
}

// Threads per row: one wave up to 64 x 32 elements, then a workgroup of 256
// or 1024.
int row_threads(int D) { return D <= 2048 ? 64 : (D <= 8192 ? 256 : 1024); }

#define SWIMBA_NORM_CFG(CALL)                                   \
  const int nt = row_threads(a.D), ept = (a.D + nt - 1) / nt;   \
  if (nt == 64) {                                               \
    if (ept <= 8) return CALL(64, 8);                           \
    if (ept <= 16) return CALL(64, 16);                         \
    return CALL(64, 32);                                        \
  }                                                             \
  if (nt == 256) {                                              \
    if (ept <= 16) return CALL(256, 16);                        \
    return CALL(256, 32);                                       \
  }                                                             \
  if (ept <= 16) return CALL(1024, 16);                         \
  return CALL(1024, 32)

template <typename T, int VEC>
hipError_t fwd_t(const NormFwdArgs& a, hipStream_t s) {
#define CALL(NT, EPT) fwd_cfg<T, VEC, NT, EPT>(a, s)
  SWIMBA_NORM_CFG(CALL);
#undef CALL
}
template <typename T, typename TG, int VEC>
hipError_t bwd_t(const NormBwdArgs& a, hipStream_t s) {
#define CALL(NT, EPT) bwd_cfg<T, TG, VEC, NT, EPT>(a, s)
  SWIMBA_NORM_CFG(CALL);
#undef CALL
}

}  // namespace

int norm_bwd_parts(int M, int D) {
  const int rp = row_threads(D) == 64 ? 4 : 1;
  const int wgs = (M + rp - 1) / rp;
  return wgs < 512 ? wgs : 512;
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
