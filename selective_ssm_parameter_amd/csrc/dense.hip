// Dense products around the mixer on the matrix cores (swimba_layers.h): the
// gated feed-forward projection with its activation in the epilogue, and the
// products of the projections' backward.
//
//   out(r, s) = sum_k a(r, k) b(s, k)
//
// Each operand lies in HBM either with k contiguous ("rows") or with r or s
// contiguous and k as the row ("columns"); a columns operand is read from LDS
// with the transposing read, so no operand is ever transposed in HBM:
//   gated projection  [g | u] = x w_in^T        rows x rows
//   dx = dz w_in,  dy = dout w_out               rows x columns
//   dw_in = dz^T x,  dw_out = dout^T y           columns x columns, k = tokens
// Tiles of 256 x 256 (8 waves), 128 x 128 (4 waves), k steps of 32; four LDS stages, filled three steps ahead by buffer-to-LDS copies that
// are waited for with a fixed count; fp32 accumulation in the matrix cores.
// Bound by the matrix cores for many tokens.
#include <type_traits>

#include "common.hpp"
#include "layers.hpp"
#include "lds_tiles.hpp"
#include "swimba_layers.h"

namespace swimba {

namespace {

template <int BM_, int BN_, int WM_, int WN_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, NTH = 64 * NW;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
};
typedef Cfg<256, 256, 2, 4> Big;
typedef Cfg<128, 128, 2, 2> Mid;

enum Mode { kGated, kNN, kTN };

struct DenseArgs {
  const void *a, *b;
  void* out;      // kGated: h
  void* z;        // kGated: [g | u] or null
  int R, S, K;    // kGated: S = F, the columns of h
  int act;
  int splits;     // kTN: k is cut into this many runs of ksplit rows
  int ksplit;
};

constexpr int kBK = 32, kStages = 4;

template <typename T, class C, Mode MODE>
struct DLay {
  static constexpr int ES = sizeof(T), EPC = 16 / ES;
  static constexpr bool ACOL = MODE == kTN, BCOL = MODE != kGated;
  // tile in LDS: rows of CPR 16-byte chunks
  static constexpr int AROWS = ACOL ? kBK : C::BM, ACPR = (ACOL ? C::BM : kBK) / EPC;
  static constexpr int BROWS = BCOL ? kBK : C::BN, BCPR = (BCOL ? C::BN : kBK) / EPC;
  static constexpr int AB = AROWS * ACPR * 16, BB = BROWS * BCPR * 16, STAGE = AB + BB;
  static constexpr int MA = AB / 1024 / C::NW, MB = BB / 1024 / C::NW;  // copies per wave
  static_assert(AB % (1024 * C::NW) == 0 && BB % (1024 * C::NW) == 0, "whole copies per wave");
};

// sigmoid(g), and Phi(g) from erfc, which keeps its relative precision for
// negative g (1 + erf would cancel)
__device__ __forceinline__ float sigm(float g) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-g));
}
__device__ __forceinline__ float normal_cdf(float g) {
  return 0.5f * erfcf(g * -0.70710678118654752f);
}
__device__ __forceinline__ float act_of(int act, float g) {
  return g * (act == SWIMBA_ACT_SILU ? sigm(g) : normal_cdf(g));
}
// act(g) and act'(g)
__device__ __forceinline__ void act_grad(int act, float g, float& v, float& d) {
  if (act == SWIMBA_ACT_SILU) {
    const float s = sigm(g);
    v = g * s;
    d = s * (1.f + g * (1.f - s));
  } else {
    const float phi = normal_cdf(g);
    v = g * phi;
    d = phi + g * 0.39894228040143268f * __expf(-0.5f * g * g);
  }
}

// XCD-aware order: workgroups are dealt round-robin to the 8 XCDs, so XCD x
// takes the contiguous range [x per, (x + 1) per) of the units, which run in
// groups of GR row tiles, column tile by column tile within a group.
__device__ __forceinline__ bool unit_of(int nr, int nc, int& tr, int& tc) {
  constexpr int GR = 4;
  const int units = nr * nc, per = (units + 7) / 8, slot = blockIdx.x / 8;
  if (slot >= per) return false;
  const int logical = (blockIdx.x % 8) * per + slot;
  if (logical >= units) return false;
  const int group = logical / (GR * nc), rem = logical - group * (GR * nc);
  const int gm = min(GR, nr - group * GR);
  tc = rem / gm;
  tr = group * GR + (rem - tc * gm);
  return true;
}

template <typename T, class C, Mode MODE, typename TO>
__global__ __launch_bounds__(C::NTH) void dense_kernel(DenseArgs A) {
  typedef DLay<T, C, MODE> L;
  typedef typename Vec<T>::x8 F;
  constexpr int BM = C::BM, BN = C::BN, NW = C::NW, TM = C::TM, TN = C::TN;
  constexpr int MA = L::MA, MB = L::MB, EPC = L::EPC;
  constexpr uint32_t ES = L::ES;
  // columns of out per tile: the gated tile holds BN / 2 of g and the same of u
  constexpr int SN = MODE == kGated ? BN / 2 : BN;

  // four stage arrays: copies into one are known not to touch the others
  __shared__ __align__(16) unsigned char stg0[L::STAGE];
  __shared__ __align__(16) unsigned char stg1[L::STAGE];
  __shared__ __align__(16) unsigned char stg2[L::STAGE];
  __shared__ __align__(16) unsigned char stg3[L::STAGE];

  const int nr = (A.R + BM - 1) / BM, nc = (A.S + SN - 1) / SN;
  int tr, tc, split = 0;
  if constexpr (MODE == kTN) {
    // the splits of one unit follow each other
    if (!unit_of(nr, nc * A.splits, tr, tc)) return;
    split = tc % A.splits;
    tc /= A.splits;
  } else {
    if (!unit_of(nr, nc, tr, tc)) return;
  }
  const int r0 = tr * BM, s0 = tc * SN;
  const int nrows = min(BM, A.R - r0);
  const int kbeg = MODE == kTN ? split * A.ksplit : 0;
  const int K = MODE == kTN ? min(A.ksplit, A.K - kbeg) : A.K;

  const int lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;

  // ---- copy plan: instruction m of this wave fills the 64 LDS chunks from
  // 64 (wave + NW m) on; every lane's offset in HBM is that of k = 0, a k step
  // enters as the copy's scalar offset. Buffers start at this tile's rows (or
  // this split's tokens), so that only a weight matrix or one tile's or
  // split's rows have to stay below 2 GiB.
  const T* ap = static_cast<const T*>(A.a);
  const T* bp = static_cast<const T*>(A.b);
  BufRes rA, rB;
  uint32_t aoff[MA], boff[MB];
  int akc[MA], bkc[MB];  // rows operands: the chunk's first k, to cut at K
  uint32_t astep, bstep;
  if constexpr (L::ACOL) {
    rA = make_rsrc(ap + (size_t)kbeg * A.R, (uint64_t)K * A.R * ES);
    astep = kBK * (uint32_t)A.R * ES;
  } else {
    rA = make_rsrc(ap + (size_t)r0 * A.K, (uint64_t)nrows * A.K * ES);
    astep = kBK * ES;
  }
  if constexpr (L::BCOL) {
    rB = make_rsrc(bp + (size_t)kbeg * A.S, (uint64_t)K * A.S * ES);
    bstep = kBK * (uint32_t)A.S * ES;
  } else {
    rB = make_rsrc(bp, (uint64_t)2 * A.S * A.K * ES);
    bstep = kBK * ES;
  }
#pragma unroll
  for (int m = 0; m < MA; ++m) {
    const int slot = 64 * (wave + NW * m) + lane;
    const int r = slot / L::ACPR, pc = slot % L::ACPR;
    if constexpr (L::ACOL) {
      const int col = r0 + (pc ^ swz_tr<T, L::ACPR>(r)) * EPC;
      aoff[m] = col < A.R ? ((uint32_t)r * A.R + col) * ES : kOOB;
      akc[m] = r;
    } else {
      akc[m] = (pc ^ swz_row<T, L::ACPR>(r)) * EPC;
      aoff[m] = r < nrows ? ((uint32_t)r * A.K + akc[m]) * ES : kOOB;
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int slot = 64 * (wave + NW * m) + lane;
    const int r = slot / L::BCPR, pc = slot % L::BCPR;
    if constexpr (L::BCOL) {
      const int col = s0 + (pc ^ swz_tr<T, L::BCPR>(r)) * EPC;
      boff[m] = col < A.S ? ((uint32_t)r * A.S + col) * ES : kOOB;
      bkc[m] = r;
    } else {
      // 64 tile rows are 32 columns of g and the same 32 of u
      const int col = s0 + (r >> 6) * 32 + (r & 31);
      bkc[m] = (pc ^ swz_row<T, L::BCPR>(r)) * EPC;
      boff[m] = col < A.S
                    ? ((uint32_t)(((r >> 5) & 1 ? A.S : 0) + col) * A.K + bkc[m]) * ES
                    : kOOB;
    }
  }
  // Steps past K read zeros: a columns operand's rows end with its buffer, a
  // rows operand's chunks past K are cut one by one.
  auto fetch = [&](unsigned char* st, int kt) {
    const int k0 = kt * kBK;
#pragma unroll
    for (int m = 0; m < MA; ++m) {
      const uint32_t off = k0 + akc[m] < K && aoff[m] != kOOB ? aoff[m] + kt * astep : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rA, (__attribute__((address_space(3))) void*)(st + 1024 * (wave + NW * m)), 16, off, 0, 0,
          0);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const uint32_t off = k0 + bkc[m] < K && boff[m] != kOOB ? boff[m] + kt * bstep : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rB, (__attribute__((address_space(3))) void*)(st + L::AB + 1024 * (wave + NW * m)), 16,
          off, 0, 0, 0);
    }
  };

  // ---- fragments. acc[i][j] holds, in lane (g, c), row 16 i + c and columns
  // 16 j + 4 g .. + 3 of this wave's block (b is the matrix cores' A operand);
  // the gated tile's columns are permuted within pairs of tiles so that a
  // lane's 8 values of a pair are consecutive columns 8 g .. 8 g + 7.
  auto afrag = [&](const unsigned char* st, int i) -> F {
    const int row = wm * TM * 16 + 16 * i;
    if constexpr (L::ACOL) {
      return load_kmajor<T, L::ACPR>(st, 0, row, lane);
    } else {
      const int r = row + c;
      if constexpr (ES == 2)
        return load8<T>(reinterpret_cast<const T*>(
            st + (r * L::ACPR + (g ^ swz_row<T, L::ACPR>(r))) * 16));
      else
        return load8<T>(reinterpret_cast<const T*>(st + r * L::ACPR * 16 + 32 * g));
    }
  };
  auto bfrag = [&](const unsigned char* st, int j) -> F {
    if constexpr (L::BCOL) {
      return load_kmajor<T, L::BCPR>(st + L::AB, 0, wn * TN * 16 + 16 * j, lane);
    } else {
      const int r = wn * TN * 16 + 32 * (j >> 1) + 8 * (c >> 2) + 4 * (j & 1) + (c & 3);
      if constexpr (ES == 2)
        return load8<T>(reinterpret_cast<const T*>(
            st + L::AB + (r * L::BCPR + (g ^ swz_row<T, L::BCPR>(r))) * 16));
      else
        return load8<T>(reinterpret_cast<const T*>(st + L::AB + r * L::BCPR * 16 + 32 * g));
    }
  };

  floatx4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const unsigned char* st) {
    F bf[TN], af[TM];
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[j] = bfrag(st, j);
#pragma unroll
    for (int i = 0; i < TM; ++i) af[i] = afrag(st, i);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma16(bf[j], af[i], acc[i][j]);
  };

  // whole turns of the four stages, every copy unconditional (steps past K
  // multiply zeros)
  const int nk4 = ((K + kBK - 1) / kBK + kStages - 1) / kStages * kStages;
  fetch(stg0, 0);
  fetch(stg1, 1);
  fetch(stg2, 2);
  auto iter = [&](int kt, const unsigned char* cur, unsigned char* far) {
    wait_vm<2 * (MA + MB)>();  // step kt landed (steps kt + 1, kt + 2 may be in flight)
    stage_barrier();           // step kt visible to all waves; step kt - 1 no longer read
    fetch(far, kt + 3);
    compute(cur);
  };
  for (int kt = 0; kt < nk4; kt += kStages) {
    iter(kt, stg0, stg3);
    iter(kt + 1, stg1, stg0);
    iter(kt + 2, stg2, stg1);
    iter(kt + 3, stg3, stg2);
  }
  wait_vm<0>();  // the copies past the end land before the workgroup's LDS is released

  // ---- epilogue
  if constexpr (MODE == kGated) {
    static_assert(TN % 4 == 0, "a pair of g tiles and the pair of u tiles per wave");
    TO* h = static_cast<TO*>(A.out);
    TO* z = static_cast<TO*>(A.z);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm * TM * 16 + 16 * i + c;
#pragma unroll
      for (int jj = 0; jj < TN / 4; ++jj) {
        const int col = s0 + (wn * (TN / 4) + jj) * 32 + 8 * g;
        if (r >= nrows || col >= A.S) continue;
        typename Vec<TO>::x8 og, ou, oh;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float gv = acc[i][4 * jj + (q >> 2)][q & 3];
          const float uv = acc[i][4 * jj + 2 + (q >> 2)][q & 3];
          og[q] = from_f32<TO>(gv);
          ou[q] = from_f32<TO>(uv);
          oh[q] = from_f32<TO>(act_of(A.act, gv) * uv);
        }
        const size_t row = (size_t)(r0 + r);
        store8<TO>(h + row * A.S + col, oh);
        if (z) {
          store8<TO>(z + row * 2 * A.S + col, og);
          store8<TO>(z + row * 2 * A.S + A.S + col, ou);
        }
      }
    }
  } else {
    typedef typename Vec<TO>::x4 O4;
    TO* out = static_cast<TO*>(A.out) + (MODE == kTN ? (size_t)split * A.R * A.S : 0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm * TM * 16 + 16 * i + c;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int col = s0 + wn * TN * 16 + 16 * j + 4 * g;
        if (r >= nrows || col >= A.S) continue;
        O4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = from_f32<TO>(acc[i][j][q]);
        *reinterpret_cast<O4*>(out + (size_t)(r0 + r) * A.S + col) = o;
      }
    }
  }
}

// dz = [dh u act'(g) | dh act(g)], 8 columns per thread.
template <typename T>
__global__ __launch_bounds__(256) void gated_dz_kernel(const T* __restrict__ z,
                                                       const T* __restrict__ dh,
                                                       T* __restrict__ dz, int M, int F, int act) {
  const int f8 = F / 8;
  const size_t n = (size_t)M * f8;
  for (size_t q = (size_t)blockIdx.x * 256 + threadIdx.x; q < n; q += (size_t)gridDim.x * 256) {
    const size_t m = q / f8;
    const int c = (int)(q - m * f8) * 8;
    const typename Vec<T>::x8 gv = load8<T>(z + m * 2 * F + c);
    const typename Vec<T>::x8 uv = load8<T>(z + m * 2 * F + F + c);
    const typename Vec<T>::x8 dv = load8<T>(dh + m * F + c);
    typename Vec<T>::x8 og, ou;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v, d;
      act_grad(act, to_f32(gv[j]), v, d);
      const float dd = to_f32(dv[j]);
      og[j] = from_f32<T>(dd * to_f32(uv[j]) * d);
      ou[j] = from_f32<T>(dd * v);
    }
    store8<T>(dz + m * 2 * F + c, og);
    store8<T>(dz + m * 2 * F + F + c, ou);
  }
}

// out = the splits' partial products added in split order.
__global__ __launch_bounds__(256) void dense_sum_kernel(const float* __restrict__ part, int splits,
                                                        size_t n4, float* __restrict__ out) {
  for (size_t q = (size_t)blockIdx.x * 256 + threadIdx.x; q < n4; q += (size_t)gridDim.x * 256) {
    floatx4 s = reinterpret_cast<const floatx4*>(part)[q];
    for (int p = 1; p < splits; ++p) s = s + reinterpret_cast<const floatx4*>(part)[p * n4 + q];
    reinterpret_cast<floatx4*>(out)[q] = s;
  }
}

template <typename T, class C, Mode MODE, typename TO>
hipError_t go(const char* name, const DenseArgs& A, hipStream_t s) {
  constexpr int SN = MODE == kGated ? C::BN / 2 : C::BN;
  const int64_t units = (int64_t)((A.R + C::BM - 1) / C::BM) * ((A.S + SN - 1) / SN) *
                        (MODE == kTN ? A.splits : 1);
  hipEvent_t e0, e1;
  prof_kernel(name, &e0, &e1);
  hipExtLaunchKernelGGL((dense_kernel<T, C, MODE, TO>), dim3((unsigned)((units + 7) / 8 * 8)),
                        dim3(C::NTH), 0, s, e0, e1, 0, A);
  return hipGetLastError();
}

unsigned grid_1d(size_t threads) {
  const size_t b = (threads + 255) / 256;
  return (unsigned)(b < 4096 ? b : 4096);
}

// k runs of a weight gradient: enough workgroups to fill the chip, at least
// 512 tokens each, and every run's operand rows below 2 GiB.
void tn_splits(bool is_bf16, int M, int R, int S, int& splits, int& ksplit) {
  const int bt = is_bf16 && (int64_t)R * S >= 256 * 256 * 16 ? 256 : 128;
  const int64_t units = (int64_t)((R + bt - 1) / bt) * ((S + bt - 1) / bt);
  int64_t n = (256 + units - 1) / units;
  const int64_t most = (M + 511) / 512;
  if (n > most) n = most;
  const int64_t row = (int64_t)(R > S ? R : S) * (is_bf16 ? 2 : 4);
  const int64_t least = (M * row + (1ll << 30) - 1) >> 30;
  if (n < least) n = least;
  if (n < 1) n = 1;
  ksplit = (int)(((M + n - 1) / n + kBK - 1) / kBK * kBK);
  splits = (M + ksplit - 1) / ksplit;
}

}  // namespace

hipError_t launch_gated_project(bool is_bf16, int M, int D, int F, int act, const void* x,
                                const void* w_in, void* z, void* h, hipStream_t s) {
  DenseArgs A{};
  A.a = x; A.b = w_in; A.out = h; A.z = z; A.R = M; A.S = F; A.K = D; A.act = act;
  if (is_bf16) {
    if (M >= 2048) return go<bf16, Big, kGated, bf16>("gated_project", A, s);
    return go<bf16, Mid, kGated, bf16>("gated_project", A, s);
  }
  return go<float, Mid, kGated, float>("gated_project", A, s);
}

hipError_t launch_gated_dz(bool is_bf16, int M, int F, int act, const void* z, const void* dh,
                           void* dz, hipStream_t s) {
  hipEvent_t e0, e1;
  prof_kernel("gated_dz", &e0, &e1);
  const dim3 grid(grid_1d((size_t)M * (F / 8)));
  if (is_bf16)
    hipExtLaunchKernelGGL(gated_dz_kernel<bf16>, grid, dim3(256), 0, s, e0, e1, 0, (const bf16*)z,
                          (const bf16*)dh, (bf16*)dz, M, F, act);
  else
    hipExtLaunchKernelGGL(gated_dz_kernel<float>, grid, dim3(256), 0, s, e0, e1, 0,
                          (const float*)z, (const float*)dh, (float*)dz, M, F, act);
  return hipGetLastError();
}

hipError_t launch_dense_nn(bool is_bf16, bool out_f32, const char* name, int M, int K, int S,
                           const void* a, const void* b, void* out, hipStream_t s) {
  DenseArgs A{};
  A.a = a; A.b = b; A.out = out; A.R = M; A.S = S; A.K = K;
  if (!is_bf16) return go<float, Mid, kNN, float>(name, A, s);
  const bool big = M >= 4096 && S >= 192;
  if (out_f32)
    return big ? go<bf16, Big, kNN, float>(name, A, s) : go<bf16, Mid, kNN, float>(name, A, s);
  return big ? go<bf16, Big, kNN, bf16>(name, A, s) : go<bf16, Mid, kNN, bf16>(name, A, s);
}

size_t dense_tn_ws_bytes(bool is_bf16, int M, int R, int S) {
  int splits, ksplit;
  tn_splits(is_bf16, M, R, S, splits, ksplit);
  return splits > 1 ? sizeof(float) * (size_t)splits * R * S : 0;
}

hipError_t launch_dense_tn(bool is_bf16, const char* name, int M, int R, int S, const void* a,
                           const void* b, float* out, void* ws, hipStream_t s) {
  DenseArgs A{};
  A.a = a; A.b = b; A.R = R; A.S = S; A.K = M;
  tn_splits(is_bf16, M, R, S, A.splits, A.ksplit);
  A.out = A.splits > 1 ? ws : (void*)out;
  hipError_t e;
  if (!is_bf16) e = go<float, Mid, kTN, float>(name, A, s);
  else if ((int64_t)R * S >= 256 * 256 * 16) e = go<bf16, Big, kTN, float>(name, A, s);
  else e = go<bf16, Mid, kTN, float>(name, A, s);
  if (e != hipSuccess || A.splits == 1) return e;
  hipEvent_t e0, e1;
  prof_kernel("dense_sum", &e0, &e1);
  const size_t n4 = (size_t)R * S / 4;
  hipExtLaunchKernelGGL(dense_sum_kernel, dim3(grid_1d(n4)), dim3(256), 0, s, e0, e1, 0,
                        (const float*)ws, A.splits, n4, out);
  return hipGetLastError();
}

}  // namespace swimba
