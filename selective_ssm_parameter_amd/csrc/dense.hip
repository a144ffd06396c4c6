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
// Tiles of 256 x 256 and 256 x 192 (8 waves), 128 x 128, 64 x 64, 32 x 64 and,
// for gated products, 64 x 128 and 32 x 128 (4 waves), k steps of 32; two to
// four LDS stages (DLay::NS), all but one filled ahead by buffer-to-LDS copies
// that are waited for with a fixed count; fp32 accumulation in the matrix cores.
// The gated projection's backward recomputes g and u with the forward's product
// and turns them into dz in the epilogue, in fp32; for bf16 problems dz then
// goes through both products as hi + lo, two bf16 numbers: 16 bits of dz, an
// element off by at most 2^-16 of itself, where one bf16 rounding is off by
// 2^-8 (16384 x 768 -> 2 x 2048: dx and dw_in 2.5e-6 off in the 2-norm, against
// 2.5e-3 with one and 1.2e-6 with an fp32 product): each LDS stage holds both,
// three stages of them, and a fragment of the other operand serves both.
// Bound by the matrix cores for many tokens.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "dense_plan.hpp"
#include "layers.hpp"
#include "lds_tiles.hpp"
#include "swimba_layers.h"

namespace swimba {

namespace {

// BM x BN tiles by WM x WN waves.
template <int BM_, int BN_, int WM_, int WN_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, NTH = 64 * NW;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
};
typedef Cfg<256, 256, 2, 4> Big;
typedef Cfg<256, 192, 2, 4> Wide;  // not for gated products
typedef Cfg<128, 128, 2, 2> Mid;
typedef Cfg<64, 128, 2, 2> Small;   // gated products (32 columns of g and of u per wave)
typedef Cfg<64, 64, 2, 2> Small64;  // the others
typedef Cfg<32, 64, 2, 2> Tiny;
typedef Cfg<32, 128, 2, 2> TinyGated;  // fp32 gated products: 100 x 512 x 1024
                                         // 21.8 -> 15.2 us, 300 x 2048 x 4096 142 -> 113

// kGated: h; kGatedBwd: the same product, dz in the epilogue
enum Mode { kGated, kGatedBwd, kNN, kTN };
constexpr bool is_gated(Mode m) { return m == kGated || m == kGatedBwd; }

struct DenseArgs {
  const void *a, *b;
  const void* a_lo;  // split operands: a = a (bf16) + a_lo (bf16)
  void* out;         // kGated: h; kGatedBwd: dz (its lo half behind it for bf16)
  void* z;           // kGated: [g | u] or null
  const void* dh;    // kGatedBwd
  int R, S, K;       // gated: S = F, the columns of h
  int act;
  int splits;     // kNN, kTN: k is cut into this many runs of ksplit, their
                  // partial products [splits][R][S] float32 in out
  int ksplit;
};

template <typename T, class C, Mode MODE, bool SPLIT>
struct DLay {
  static constexpr int ES = sizeof(T), EPC = 16 / ES;
  // (fp32 128 x 128 gated tiles: two stages, so that two workgroups share a CU,
  // 114 against 90 TFLOP/s at 12000 x 320 x 512; no gain for columns tiles)
  // (32 x 128: three, also for two workgroups a CU)
  static constexpr int NS =
      SPLIT ? 3 : !(is_gated(MODE) && ES == 4) ? 4 : C::BM == 128 ? 2 : C::BM == 32 ? 3 : 4;
  static constexpr bool ACOL = MODE == kTN, BCOL = !is_gated(MODE);
  // tile in LDS: rows of CPR 16-byte chunks
  static constexpr int AROWS = ACOL ? kBK : C::BM, ACPR = (ACOL ? C::BM : kBK) / EPC;
  static constexpr int BROWS = BCOL ? kBK : C::BN, BCPR = (BCOL ? C::BN : kBK) / EPC;
  static constexpr int AB = AROWS * ACPR * 16, BB = BROWS * BCPR * 16, STAGE = AB * (SPLIT ? 2 : 1) + BB;
  static constexpr int BOFF = STAGE - BB;  // a (, a_lo), b
  static constexpr int NA = AB / 1024, NB = BB / 1024;  // copies of 64 chunks
  static constexpr int MA = (NA + C::NW - 1) / C::NW, MB = (NB + C::NW - 1) / C::NW;  // per wave
  static constexpr int CPW = MA * (SPLIT ? 2 : 1) + MB;
  static_assert(AB % 1024 == 0 && BB % 1024 == 0, "whole copies");
};

// Copy m of a wave among n: where the copies do not divide by the waves, the
// waves past the last one repeat an earlier copy (the same bytes to the same
// place), so that every wave waits for the same count.
template <int NCOPY, int NW>
__device__ __forceinline__ int copy_of(int m, int wave) {
  const int i = wave + NW * m;
  return NCOPY % NW == 0 || i < NCOPY ? i : i - NCOPY;
}

// Fragments from LDS. The contraction index of element e in lane group g is
// 8 g + e for 2-byte types and 4 g + e % 4 + 16 (e / 4) for fp32, for rows and
// columns tiles alike.
//
// Rows tiles: chunk ch of row r lies at ch ^ swz_rows(r).
template <typename T, int CPR>
__device__ __forceinline__ int swz_rows(int r) {
  if constexpr (sizeof(T) == 2) return swz_row<T, CPR>(r);
  else return r & 7;  // 8 chunks a row: 8 lanes reading one chunk of 8 rows take all of them
}
template <typename T, int CPR>
__device__ __forceinline__ typename Vec<T>::x8 load_row(const unsigned char* tile, int r, int g) {
  const unsigned char* row = tile + r * CPR * 16;
  const int x = swz_rows<T, CPR>(r);
  if constexpr (sizeof(T) == 2)
    return load8<T>(reinterpret_cast<const T*>(row + 16 * (g ^ x)));
  else
    return load4x2<T>(reinterpret_cast<const T*>(row + 16 * (g ^ x)),
                      reinterpret_cast<const T*>(row + 16 * ((g + 4) ^ x)));
}
// Columns tiles ([k][column]), 2-byte types: transposing reads, chunks swizzled
// as swz_tr; rows of 24 chunks keep the swizzle within aligned groups of 8.
// fp32 tiles are not swizzled: a lane reads N neighbouring columns of a row at
// once, one for each of N matrix-core tiles, whose columns are then N apart
// (tile n, index m: column col0 + N m + n).
template <typename T, int CPR>
__device__ __forceinline__ int swz_cols(int r) {
  if constexpr (sizeof(T) == 4) return 0;
  else if constexpr (CPR % 16 == 0 || CPR < 16) return swz_tr<T, CPR>(r);
  else return swz_tr<T, 8>(r);
}
template <typename T, int CPR, int N>
__device__ __forceinline__ void load_cols(const unsigned char* tile, int col0, int lane,
                                          typename Vec<T>::x8 (&f)[N]) {
  const int g = lane >> 4, c = lane & 15;
  if constexpr (sizeof(T) == 2) {
    typedef short s4 __attribute__((__vector_size__(8)));
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = 8 * g + 4 * hh + (c >> 2), col = col0 + 16 * n + 4 * (c & 3);
        const unsigned char* p =
            tile + (r * CPR + ((col >> 3) ^ swz_cols<T, CPR>(r))) * 16 + 8 * ((col >> 2) & 1);
        const typename Vec<T>::x4 w4 = __builtin_bit_cast(
            typename Vec<T>::x4,
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)(p)));
#pragma unroll
        for (int m = 0; m < 4; ++m) f[n][4 * hh + m] = w4[m];
      }
    }
  } else {
    typedef float FN __attribute__((ext_vector_type(N)));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = 4 * g + (e & 3) + 16 * (e >> 2);
      const FN v = *reinterpret_cast<const FN*>(tile + k * CPR * 16 + (col0 + N * c) * 4);
#pragma unroll
      for (int n = 0; n < N; ++n) f[n][e] = v[n];
    }
  }
}

__device__ __forceinline__ float sigm(float g) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-g));
}
// e = exp(-g^2 / 2) and Phi(g), from the upper tail Q(|g|) = e erfcx(|g| / sqrt 2) / 2,
// so that it keeps its relative precision for negative g. erfcx (e^(x^2) erfc x)
// is a polynomial of degree 9 in t = 1 / (1 + 0.3 x) without constant term,
// fitted for this file by reweighted least squares on 0 <= x <= 10: relative
// error 2e-8, 4.4e-7 evaluated in fp32. (The library's erfcf took 30 us more
// of a 16384 x 2048 projection of 768.)
__device__ __forceinline__ float normal_cdf(float g, float& e) {
  const float a = fabsf(g);
  e = __builtin_amdgcn_exp2f(-0.72134752044f * g * g);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.21213203436f, a, 1.f));
  float c = -0.12952312601577864f;
  c = __builtin_fmaf(c, t, 0.4855643722941682f);
  c = __builtin_fmaf(c, t, -0.5122806874687891f);
  c = __builtin_fmaf(c, t, 0.5477232538943848f);
  c = __builtin_fmaf(c, t, -0.09465315028525317f);
  c = __builtin_fmaf(c, t, 0.21492718641342054f);
  c = __builtin_fmaf(c, t, 0.14833885369157157f);
  c = __builtin_fmaf(c, t, 0.17071527585634538f);
  c = __builtin_fmaf(c, t, 0.16918800203758264f);
  const float tail = 0.5f * c * t * e;
  return g > 0.f ? 1.f - tail : tail;
}
__device__ __forceinline__ float act_of(int act, float g) {
  float e;
  return g * (act == SWIMBA_ACT_SILU ? sigm(g) : normal_cdf(g, e));
}
// act(g) and act'(g)
__device__ __forceinline__ void act_grad(int act, float g, float& v, float& d) {
  if (act == SWIMBA_ACT_SILU) {
    const float s = sigm(g);
    v = g * s;
    d = s * (1.f + g * (1.f - s));
  } else {
    float e;
    const float phi = normal_cdf(g, e);
    v = g * phi;
    d = __builtin_fmaf(g * 0.39894228040143268f, e, phi);
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

// 8 elements of a gated output, past the L2's reuse order where its rows start on
// 128-byte lines (through): 32768 x 8192 x 2048 2 % faster. (The order is a hint:
// the next kernel sees the values as those of any store.)
template <typename T>
__device__ __forceinline__ void store_gated(T* p, typename Vec<T>::x8 v, bool through) {
  if constexpr (sizeof(T) == 2) {
    if (through) {
      __builtin_nontemporal_store(__builtin_bit_cast(int4v, v), reinterpret_cast<int4v*>(p));
      return;
    }
  }
  store8<T>(p, v);
}

template <typename T, class C, Mode MODE, typename TO, bool SPLIT>
__global__ __launch_bounds__(C::NTH) void dense_kernel(DenseArgs A) {
  typedef DLay<T, C, MODE, SPLIT> L;
  typedef typename Vec<T>::x8 F;
  constexpr int BM = C::BM, BN = C::BN, NW = C::NW, TM = C::TM, TN = C::TN;
  constexpr int MA = L::MA, MB = L::MB, EPC = L::EPC;
  constexpr uint32_t ES = L::ES;
  // columns of out per tile: the gated tile holds BN / 2 of g and the same of u
  constexpr int SN = is_gated(MODE) ? BN / 2 : BN;

  // an array per stage: copies into one are known not to touch the others
  __shared__ __align__(16) unsigned char stg0[L::STAGE];
  __shared__ __align__(16) unsigned char stg1[L::STAGE];
  __shared__ __align__(16) unsigned char stg2[L::NS > 2 ? L::STAGE : 16];
  __shared__ __align__(16) unsigned char stg3[L::NS > 3 ? L::STAGE : 16];

  const int nr = (A.R + BM - 1) / BM, nc = (A.S + SN - 1) / SN;
  int tr, tc, split = 0;
  if constexpr (!is_gated(MODE)) {
    // the splits of one unit follow each other
    if (!unit_of(nr, nc * A.splits, tr, tc)) return;
    split = tc % A.splits;
    tc /= A.splits;
  } else {
    if (!unit_of(nr, nc, tr, tc)) return;
  }
  const int r0 = tr * BM, s0 = tc * SN;
  const int nrows = min(BM, A.R - r0);
  const int kbeg = split * A.ksplit;
  const int K = is_gated(MODE) ? A.K : min(A.ksplit, A.K - kbeg);

  const int lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;

  // ---- copy plan: instruction m of this wave fills the 64 LDS chunks from
  // 64 (wave + NW m) on; every lane's offset in HBM is that of k = 0; fetch
  // adds the k step, or takes the out-of-range offset past the end. Buffers start at this tile's rows (or
  // this split's tokens), so that only a weight matrix or one tile's or
  // split's rows have to stay below 2 GiB.
  const T* ap = static_cast<const T*>(A.a);
  const T* bp = static_cast<const T*>(A.b);
  const T* lp = static_cast<const T*>(A.a_lo);
  BufRes rA, rL, rB;
  uint32_t aoff[MA], boff[MB];
  int akc[MA], bkc[MB];  // rows operands: the chunk's first k, to cut at K
  uint32_t astep, bstep;
  if constexpr (L::ACOL) {
    rA = make_rsrc(ap + (size_t)kbeg * A.R, (uint64_t)K * A.R * ES);
    if constexpr (SPLIT) rL = make_rsrc(lp + (size_t)kbeg * A.R, (uint64_t)K * A.R * ES);
    astep = kBK * (uint32_t)A.R * ES;
  } else {
    const uint64_t bytes = ((uint64_t)nrows * A.K - kbeg) * ES;
    rA = make_rsrc(ap + (size_t)r0 * A.K + kbeg, bytes);
    if constexpr (SPLIT) rL = make_rsrc(lp + (size_t)r0 * A.K + kbeg, bytes);
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
    const int slot = 64 * copy_of<L::NA, NW>(m, wave) + lane;
    const int r = slot / L::ACPR, pc = slot % L::ACPR;
    if constexpr (L::ACOL) {
      const int col = r0 + (pc ^ swz_cols<T, L::ACPR>(r)) * EPC;
      aoff[m] = col < A.R ? ((uint32_t)r * A.R + col) * ES : kOOB;
      akc[m] = r;
    } else {
      akc[m] = (pc ^ swz_rows<T, L::ACPR>(r)) * EPC;
      aoff[m] = r < nrows ? ((uint32_t)r * A.K + akc[m]) * ES : kOOB;
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int slot = 64 * copy_of<L::NB, NW>(m, wave) + lane;
    const int r = slot / L::BCPR, pc = slot % L::BCPR;
    if constexpr (L::BCOL) {
      const int col = s0 + (pc ^ swz_cols<T, L::BCPR>(r)) * EPC;
      boff[m] = col < A.S ? ((uint32_t)r * A.S + col) * ES : kOOB;
      bkc[m] = r;
    } else {
      // 64 tile rows are 32 columns of g and the same 32 of u
      const int col = s0 + (r >> 6) * 32 + (r & 31);
      bkc[m] = (pc ^ swz_rows<T, L::BCPR>(r)) * EPC;
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
          rA, (__attribute__((address_space(3))) void*)(st + 1024 * copy_of<L::NA, NW>(m, wave)), 16,
          off, 0, 0, 0);
      if constexpr (SPLIT)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rL, (__attribute__((address_space(3))) void*)(st + L::AB + 1024 * copy_of<L::NA, NW>(m, wave)),
            16, off, 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const uint32_t off = k0 + bkc[m] < K && boff[m] != kOOB ? boff[m] + kt * bstep : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rB, (__attribute__((address_space(3))) void*)(st + L::BOFF + 1024 * copy_of<L::NB, NW>(m, wave)),
          16, off, 0, 0, 0);
    }
  };

  // ---- fragments. acc[i][j] holds, in lane (g, c), index c of row tile i and
  // indexes 4 g .. + 3 of column tile j of this wave's block (b is the matrix
  // cores' A operand). The gated tile's columns are permuted within pairs of
  // tiles so that a lane's 8 values of a pair are consecutive columns
  // 8 g .. 8 g + 7.
  auto load_a = [&](const unsigned char* st, F (&f)[TM]) __attribute__((always_inline)) {
    const int row = wm * TM * 16;
    if constexpr (L::ACOL) {
      load_cols<T, L::ACPR, TM>(st, row, lane, f);
    } else {
#pragma unroll
      for (int i = 0; i < TM; ++i) f[i] = load_row<T, L::ACPR>(st, row + 16 * i + c, g);
    }
  };
  auto load_b = [&](const unsigned char* st, F (&f)[TN]) __attribute__((always_inline)) {
    const int col = wn * TN * 16;
    if constexpr (L::BCOL) {
      load_cols<T, L::BCPR, TN>(st + L::BOFF, col, lane, f);
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        f[j] = load_row<T, L::BCPR>(
            st + L::BOFF, col + 32 * (j >> 1) + 8 * (c >> 2) + 4 * (j & 1) + (c & 3), g);
    }
  };

  floatx4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  // DEFER (the gated products on the largest tile): the products of a step's
  // last row of fragments are issued after the reads of the next step (past its
  // barrier), so that they cover the wait for those reads: 1 to 3 %.
  constexpr bool DEFER = is_gated(MODE) && TM == 8;
  F bd[DEFER ? TN : 1], ad = zero8<T>();
  if constexpr (DEFER) {
#pragma unroll
    for (int j = 0; j < TN; ++j) bd[j] = zero8<T>();
  }
  auto compute = [&](const unsigned char* st) {
    F bf[TN], af[TM];
    load_b(st, bf);
    load_a(st, af);
    if constexpr (DEFER) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[TM - 1][j] = mma16(bd[j], ad, acc[TM - 1][j]);
#pragma unroll
      for (int j = 0; j < TN; ++j) bd[j] = bf[j];
      ad = af[TM - 1];
    }
#pragma unroll
    for (int i = 0; i < (DEFER ? TM - 1 : TM); ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma16(bf[j], af[i], acc[i][j]);
    if constexpr (SPLIT) {
      load_a(st + L::AB, af);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mma16(bf[j], af[i], acc[i][j]);
    }
  };

  // whole turns of the stages, every copy unconditional (steps past K
  // multiply zeros)
  const int nks = ((K + kBK - 1) / kBK + L::NS - 1) / L::NS * L::NS;
  auto iter = [&](int kt, const unsigned char* cur, unsigned char* far) {
    wait_vm<(L::NS - 2) * L::CPW>();  // step kt landed (the steps after it may be in flight)
    stage_barrier();                  // step kt visible to all waves; step kt - 1 no longer read
    fetch(far, kt + L::NS - 1);
    compute(cur);
  };
  fetch(stg0, 0);
  if constexpr (L::NS > 2) fetch(stg1, 1);
  if constexpr (L::NS == 2) {
    for (int kt = 0; kt < nks; kt += 2) {
      iter(kt, stg0, stg1);
      iter(kt + 1, stg1, stg0);
    }
  } else if constexpr (L::NS == 4) {
    fetch(stg2, 2);
    for (int kt = 0; kt < nks; kt += 4) {
      iter(kt, stg0, stg3);
      iter(kt + 1, stg1, stg0);
      iter(kt + 2, stg2, stg1);
      iter(kt + 3, stg3, stg2);
    }
  } else {
    for (int kt = 0; kt < nks; kt += 3) {
      iter(kt, stg0, stg2);
      iter(kt + 1, stg1, stg0);
      iter(kt + 2, stg2, stg1);
    }
  }
  if constexpr (DEFER) {
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[TM - 1][j] = mma16(bd[j], ad, acc[TM - 1][j]);
  }
  wait_vm<0>();  // the copies past the end land before the workgroup's LDS is released

  // ---- epilogue
  if constexpr (is_gated(MODE)) {
    static_assert(TN % 4 == 0, "a pair of g tiles and the pair of u tiles per wave");
    TO* h = static_cast<TO*>(A.out);
    TO* z = static_cast<TO*>(A.z);
    const bool through = A.S % 64 == 0;
    // the gradients of h for this lane's rows, all requested before the first use
    typename Vec<T>::x8 dv[MODE == kGatedBwd ? TM * (TN / 4) : 1];
    if constexpr (MODE == kGatedBwd) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int jj = 0; jj < TN / 4; ++jj) {
          const int r = min(wm * TM * 16 + 16 * i + c, nrows - 1);
          const int col = min(s0 + (wn * (TN / 4) + jj) * 32 + 8 * g, A.S - 8);
          dv[i * (TN / 4) + jj] =
              load8<T>(static_cast<const T*>(A.dh) + (size_t)(r0 + r) * A.S + col);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm * TM * 16 + 16 * i + c;
#pragma unroll
      for (int jj = 0; jj < TN / 4; ++jj) {
        const int col = s0 + (wn * (TN / 4) + jj) * 32 + 8 * g;
        if (r >= nrows || col >= A.S) continue;
        if constexpr (MODE == kGatedBwd) {
          const size_t row = (size_t)(r0 + r);
          floatx8 dg, du;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float v, d;
            act_grad(A.act, acc[i][4 * jj + (q >> 2)][q & 3], v, d);
            const float dd = to_f32(dv[i * (TN / 4) + jj][q]);
            dg[q] = dd * acc[i][4 * jj + 2 + (q >> 2)][q & 3] * d;
            du[q] = dd * v;
          }
          TO* hi = static_cast<TO*>(A.out) + row * 2 * A.S + col;
          const typename Vec<TO>::x8 hg = convert8<TO, float>(dg), hu = convert8<TO, float>(du);
          store_gated<TO>(hi, hg, through);
          store_gated<TO>(hi + A.S, hu, through);
          if constexpr (ES == 2) {
            TO* lo = hi + (size_t)A.R * 2 * A.S;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              dg[q] -= to_f32(hg[q]);
              du[q] -= to_f32(hu[q]);
            }
            store_gated<TO>(lo, convert8<TO, float>(dg), through);
            store_gated<TO>(lo + A.S, convert8<TO, float>(du), through);
          }
          continue;
        }
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
        store_gated<TO>(h + row * A.S + col, oh, through);
        if (z) {
          store_gated<TO>(z + row * 2 * A.S + col, og, through);
          store_gated<TO>(z + row * 2 * A.S + A.S + col, ou, through);
        }
      }
    }
  } else {
    TO* out = static_cast<TO*>(A.out) + (size_t)split * A.R * A.S;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm * TM * 16 + (ES == 4 && L::ACOL ? TM * c + i : 16 * i + c);
      if (r >= nrows) continue;
      TO* row = out + (size_t)(r0 + r) * A.S;
      if constexpr (ES == 4) {
        // index 4 g + q of the TN tiles: TN consecutive columns
        typedef TO ON __attribute__((ext_vector_type(TN)));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = s0 + wn * TN * 16 + TN * (4 * g + q);
          if (col >= A.S) continue;
          ON o;
#pragma unroll
          for (int j = 0; j < TN; ++j) o[j] = from_f32<TO>(acc[i][j][q]);
          *reinterpret_cast<ON*>(row + col) = o;
        }
      } else {
        typedef typename Vec<TO>::x4 O4;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int col = s0 + wn * TN * 16 + 16 * j + 4 * g;
          if (col >= A.S) continue;
          O4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = from_f32<TO>(acc[i][j][q]);
          *reinterpret_cast<O4*>(row + col) = o;
        }
      }
    }
  }
}

// The gated projection of at most 64 tokens (decode batches), bound by
// streaming w_in from HBM once: a workgroup owns 16 columns of h, its waves
// split k, and the weights go straight into registers as matrix-core operands,
// in bursts of kBurst k steps of 16 rows of g and of u (each row's part of a
// burst is one run of 512 bytes), the next burst requested before the products
// of this one. The tokens' rows, read by every workgroup, come from L2. The
// waves' partial products are added in LDS in wave order.
// MT: tiles of 16 tokens; KW: waves per workgroup (more where few columns would
// leave CUs without a workgroup).
template <typename T, int MT, int KW>
__global__ __launch_bounds__(64 * KW) void gated_skinny_kernel(DenseArgs A) {
  typedef typename Vec<T>::x8 F;
  constexpr int kBurst = 16 / (int)sizeof(T);
  constexpr uint32_t ES = sizeof(T);
  __shared__ floatx4 part[KW][2][MT][64];
  const int lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s0 = blockIdx.x * 16;
  const int nsteps = (A.K + 31) / 32, per = (nsteps + KW - 1) / KW;
  const int k0 = wave * per * 32, k1 = min(A.K, k0 + per * 32);  // this wave's k
  const BufRes rW = make_rsrc(A.b, (uint64_t)2 * A.S * A.K * ES);
  const BufRes rX = make_rsrc(A.a, (uint64_t)A.R * A.K * ES);
  const uint32_t wg = s0 + c < A.S ? (uint32_t)(s0 + c) * A.K * ES : kOOB;
  const uint32_t wu = s0 + c < A.S ? (uint32_t)(A.S + s0 + c) * A.K * ES : kOOB;
  uint32_t xo[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    xo[i] = 16 * i + c < A.R ? (uint32_t)(16 * i + c) * A.K * ES : kOOB;
  struct Burst {
    F w[2][kBurst], x[MT][kBurst];
  };
  auto load = [&](Burst& b, int k) {
#pragma unroll
    for (int q = 0; q < kBurst; ++q) {
      const int kk = k + 32 * q + 8 * g;
      const bool ok = kk < k1;
      b.w[0][q] = load8_buf<T>(rW, ok && wg != kOOB ? wg + kk * ES : kOOB);
      b.w[1][q] = load8_buf<T>(rW, ok && wu != kOOB ? wu + kk * ES : kOOB);
    }
#pragma unroll
    for (int q = 0; q < kBurst; ++q) {
      const int kk = k + 32 * q + 8 * g;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        b.x[i][q] = load8_buf<T>(rX, kk < k1 && xo[i] != kOOB ? xo[i] + kk * ES : kOOB);
    }
  };
  floatx4 acc[2][MT];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[q][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto mul = [&](const Burst& b) {
#pragma unroll
    for (int q = 0; q < kBurst; ++q)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[0][i] = mma16(b.w[0][q], b.x[i][q], acc[0][i]);
        acc[1][i] = mma16(b.w[1][q], b.x[i][q], acc[1][i]);
      }
  };
  constexpr int KB = 32 * kBurst;
  Burst b0, b1;
  load(b0, k0);
  for (int k = k0; k < k1; k += 2 * KB) {
    load(b1, k + KB);  // (bursts past k1 read zeros)
    __builtin_amdgcn_sched_barrier(0);
    mul(b0);
    load(b0, k + 2 * KB);
    __builtin_amdgcn_sched_barrier(0);
    mul(b1);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][q][i][lane] = acc[q][i];
  __syncthreads();
  // lane (g, c) of tile i: columns s0 + 4 g .. + 3 of token 16 i + c
  for (int i = wave; i < MT; i += KW) {
    const int m = 16 * i + c, col = s0 + 4 * g;
    if (m >= A.R || col >= A.S) continue;
    floatx4 v = part[0][0][i][lane], u = part[0][1][i][lane];
#pragma unroll
    for (int w = 1; w < KW; ++w) {
      v = v + part[w][0][i][lane];
      u = u + part[w][1][i][lane];
    }
    typename Vec<T>::x4 og, ou, oh;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      og[q] = from_f32<T>(v[q]);
      ou[q] = from_f32<T>(u[q]);
      oh[q] = from_f32<T>(act_of(A.act, v[q]) * u[q]);
    }
    typedef typename Vec<T>::x4 V4;
    *reinterpret_cast<V4*>(static_cast<T*>(A.out) + (size_t)m * A.S + col) = oh;
    if (A.z) {
      T* z = static_cast<T*>(A.z) + (size_t)m * 2 * A.S + col;
      *reinterpret_cast<V4*>(z) = og;
      *reinterpret_cast<V4*>(z + A.S) = ou;
    }
  }
}

// out = the splits' partial products added in split order.
template <typename TO>
__global__ __launch_bounds__(256) void dense_sum_kernel(const float* __restrict__ part, int splits,
                                                        size_t n4, TO* __restrict__ out) {
  for (size_t q = (size_t)blockIdx.x * 256 + threadIdx.x; q < n4; q += (size_t)gridDim.x * 256) {
    floatx4 s = reinterpret_cast<const floatx4*>(part)[q];
    for (int p = 1; p < splits; ++p) s = s + reinterpret_cast<const floatx4*>(part)[p * n4 + q];
    typename Vec<TO>::x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = from_f32<TO>(s[j]);
    reinterpret_cast<typename Vec<TO>::x4*>(out)[q] = o;
  }
}

template <typename T, class C, Mode MODE, typename TO, bool SPLIT = false>
hipError_t go(const char* name, const DenseArgs& A, hipStream_t s) {
  constexpr int SN = is_gated(MODE) ? C::BN / 2 : C::BN;
  const int64_t units = (int64_t)((A.R + C::BM - 1) / C::BM) * ((A.S + SN - 1) / SN) *
                        (is_gated(MODE) ? 1 : A.splits);
  return launch(name, dense_kernel<T, C, MODE, TO, SPLIT>, dim3((unsigned)((units + 7) / 8 * 8)),
                dim3(C::NTH), 0, s, A);
}

template <typename T, Mode MODE>
hipError_t go_gated(const char* name, const DenseArgs& A, hipStream_t s) {
  const int tile = plan(sizeof(T) == 2, false, true, A.R, 2 * (int64_t)A.S, A.K, 1).tile;
  if constexpr (sizeof(T) == 2)
    if (tile == 256256) return go<T, Big, MODE, T>(name, A, s);
  if (tile == 128128) return go<T, Mid, MODE, T>(name, A, s);
  if constexpr (sizeof(T) == 4)
    if (tile == 32128) return go<T, TinyGated, MODE, T>(name, A, s);
  return go<T, Small, MODE, T>(name, A, s);
}

constexpr int kSkinnyTokens = 64;

template <typename T, int MT>
hipError_t go_skinny(const DenseArgs& A, hipStream_t s) {
  const int units = (A.S + 15) / 16;
  auto run = [&](auto kw) {
    constexpr int KW = decltype(kw)::value;
    return launch("gated_project", gated_skinny_kernel<T, MT, KW>, dim3((unsigned)units),
                  dim3(64 * KW), 0, s, A);
  };
  // (8 waves leave 256 registers each, which more tiles of tokens do not fit)
  if constexpr (MT == 1)
    if (units < 192) return run(std::integral_constant<int, 8>());
  return run(std::integral_constant<int, 4>());
}

template <typename T, Mode MODE, typename TO, bool SPLIT>
hipError_t go_tile(int tile, const char* name, const DenseArgs& A, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (tile == 256256) return go<T, Big, MODE, TO, SPLIT>(name, A, s);
    if (tile == 256192) return go<T, Wide, MODE, TO, SPLIT>(name, A, s);
  }
  if (tile == 128128) return go<T, Mid, MODE, TO, SPLIT>(name, A, s);
  if (tile == 64064) return go<T, Small64, MODE, TO, SPLIT>(name, A, s);
  return go<T, Tiny, MODE, TO, SPLIT>(name, A, s);
}

}  // namespace

hipError_t launch_gated_project(bool is_bf16, int M, int D, int F, int act, const void* x,
                                const void* w_in, void* z, void* h, hipStream_t s) {
  DenseArgs A{};
  A.a = x; A.b = w_in; A.out = h; A.z = z; A.R = M; A.S = F; A.K = D; A.act = act;
  if (M <= 16) return is_bf16 ? go_skinny<bf16, 1>(A, s) : go_skinny<float, 1>(A, s);
  if (M <= 32) return is_bf16 ? go_skinny<bf16, 2>(A, s) : go_skinny<float, 2>(A, s);
  if (M <= kSkinnyTokens) return is_bf16 ? go_skinny<bf16, 4>(A, s) : go_skinny<float, 4>(A, s);
  return is_bf16 ? go_gated<bf16, kGated>("gated_project", A, s)
                 : go_gated<float, kGated>("gated_project", A, s);
}

size_t gated_dz_bytes(bool is_bf16, int M, int F) {
  return (size_t)M * 2 * F * 4;  // fp32, or two bf16 halves
}

hipError_t launch_gated_dz(bool is_bf16, int M, int D, int F, int act, const void* x,
                           const void* w_in, const void* dh, void* dz, hipStream_t s) {
  DenseArgs A{};
  A.a = x; A.b = w_in; A.out = dz; A.dh = dh; A.R = M; A.S = F; A.K = D; A.act = act;
  return is_bf16 ? go_gated<bf16, kGatedBwd>("gated_dz", A, s)
                 : go_gated<float, kGatedBwd>("gated_dz", A, s);
}

size_t dense_ws_bytes(bool is_bf16, bool split, bool tn, int R, int S, int K) {
  const Runs r = runs_of(is_bf16, split, tn, R, S, K);
  return r.splits > 1 ? sizeof(float) * (size_t)r.splits * R * S : 0;
}

namespace {

// The sum of a product's k runs (in ws) to out.
template <typename TO>
hipError_t sum_runs(const DenseArgs& A, const void* ws, void* out, hipStream_t s) {
  const size_t n4 = (size_t)A.R * A.S / 4;
  const unsigned blocks = (unsigned)std::min<size_t>((n4 + 255) / 256, 4096);
  return launch("dense_sum", dense_sum_kernel<TO>, dim3(blocks), dim3(256), 0, s, (const float*)ws,
                A.splits, n4, (TO*)out);
}

}  // namespace

hipError_t launch_dense_nn(bool is_bf16, const char* name, int M, int K, int S, const void* a,
                           const void* a_lo, const void* b, void* out, void* ws, hipStream_t s) {
  DenseArgs A{};
  A.a = a; A.a_lo = a_lo; A.b = b; A.R = M; A.S = S; A.K = K;
  const Runs r = runs_of(is_bf16, a_lo != nullptr, false, M, S, K);
  A.splits = r.splits;
  A.ksplit = r.ksplit;
  A.out = r.splits > 1 ? ws : out;
  hipError_t e;
  if (!is_bf16) e = go_tile<float, kNN, float, false>(r.tile, name, A, s);
  else if (a_lo) e = go_tile<bf16, kNN, float, true>(r.tile, name, A, s);
  else if (r.splits > 1) e = go_tile<bf16, kNN, float, false>(r.tile, name, A, s);
  else e = go_tile<bf16, kNN, bf16, false>(r.tile, name, A, s);
  if (e != hipSuccess || r.splits == 1) return e;
  return is_bf16 && !a_lo ? sum_runs<bf16>(A, ws, out, s) : sum_runs<float>(A, ws, out, s);
}

hipError_t launch_dense_tn(bool is_bf16, const char* name, int M, int R, int S, const void* a,
                           const void* a_lo, const void* b, float* out, void* ws, hipStream_t s) {
  DenseArgs A{};
  A.a = a; A.a_lo = a_lo; A.b = b; A.R = R; A.S = S; A.K = M;
  const Runs r = runs_of(is_bf16, a_lo != nullptr, true, R, S, M);
  A.splits = r.splits;
  A.ksplit = r.ksplit;
  A.out = r.splits > 1 ? ws : (void*)out;
  hipError_t e;
  if (!is_bf16) e = go_tile<float, kTN, float, false>(r.tile, name, A, s);
  else if (a_lo) e = go_tile<bf16, kTN, float, true>(r.tile, name, A, s);
  else e = go_tile<bf16, kTN, float, false>(r.tile, name, A, s);
  if (e != hipSuccess || r.splits == 1) return e;
  return sum_runs<float>(A, ws, out, s);
}

}  // namespace swimba
