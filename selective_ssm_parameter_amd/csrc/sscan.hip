// Selective scan (swimba_ssm.h), forward, backward and one token:
//   delta = softplus(dt + bias),  a[n] = exp(delta A[n]),  h[n] = a[n] h[n] + delta x B[n],
//   u = sum_n C[n] h[n] + D x,  y = u silu(z);
//   v = dy silu(z),  e[n] = C[n] v + c[n],  c[n] <- a[n] e[n]   (walking back),
//   dx = delta sum e B + D v,  ddelta = sum e (A a h_prev + B x),  dA = sum_t e delta a h_prev,
//   dB[n] = sum_c e[c, n] delta x,  dC[n] = sum_c v h[c, n].
// Every channel has its own decays, so nothing here is a matrix product: bound by
// the vector units. The least is 6 issue slots of four clocks per token, channel and
// state forward (the exponential takes two) and 16 backward; the kernels below take
// some 8 and, with the sums over channels and what a token needs by itself, 28, and the
// segments' first passes another 5 each. Measured: 65536 x 2048 x 16 bf16 975 us (first
// pass 385 to 430; vector units issuing 98 % of the cycles), padded 8 x 2048 x 1536 x
// 16 forward and backward 434 to 470 us, 256 x 4096 x 16 one token 25 us (HBM).
//
// A wave walks the tokens of 16 channels x 16 states: lane (channel q = lane / 4,
// j = lane % 4) holds states 4 j .. 4 j + 3 of its channel, so that sums over
// states stay within four lanes (DPP) and what depends on the token and channel
// alone (softplus, gates, loads, stores) is done once: of each four tokens lane j
// of the four takes the j-th. B and C of 16 tokens go through LDS in fp32 (each
// wave its own copy, no barrier). A workgroup is up to 4 waves of channels side by
// side times the blocks of 16 states, whose sums are added in LDS in order.
// Sequences are cut into segments where there are too few channels to fill the
// card: a first pass finds the state that each segment alone leaves and the sum of
// its delta (the product of its decays is exp(A sum delta)), and the segments
// start from those of the earlier ones; the backward likewise from the later ones.
// The forward leaves the state entering every 16 tokens; the backward recomputes
// the states and decays of 16 tokens in registers from it, with one exponential
// each.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.hpp"
#include "lds_tiles.hpp"
#include "ssm.hpp"
#include "ssm_plan.hpp"

namespace swimba {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kTok = 16;     // tokens per block
constexpr int kQ = 4;        // states per lane
constexpr int kWaveCh = 16;  // channels per wave
constexpr int kStates = 16;  // states per wave
constexpr int kMaxWaves = 8;

__host__ __device__ inline int state_blocks(int N) { return (N + kStates - 1) / kStates; }
// Waves of channels side by side in a workgroup of at most 8 waves.
__host__ __device__ inline int channel_waves(int N) {
  const int nb = state_blocks(N);
  return nb <= 2 ? 4 : nb <= 4 ? 2 : 1;
}
__host__ __device__ inline int group_blocks(int Ch, int N, int G) {
  const int per = Ch / G, cols = kWaveCh * channel_waves(N);
  return (per + cols - 1) / cols;
}

// ---- lanes
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF, true));
}
// Lane q of each four, to all four.
template <int Q> __device__ __forceinline__ float quad(float v) { return dpp<Q * 0x55>(v); }
// The sum over the four lanes, in all of them.
__device__ __forceinline__ float quad_sum(float v) {
  v += dpp<0xB1>(v);         // lane ^ 1
  return v + dpp<0x4E>(v);   // lane ^ 2
}
// v[q] summed over the four lanes, the q-th sum to lane q.
__device__ __forceinline__ float quad_spread(const float (&v)[4], int j) {
  const bool b0 = j & 1, b1 = j & 2;
  const float r0 = (b0 ? v[1] : v[0]) + dpp<0xB1>(b0 ? v[0] : v[1]);
  const float r1 = (b0 ? v[3] : v[2]) + dpp<0xB1>(b0 ? v[2] : v[3]);
  return (b1 ? r1 : r0) + dpp<0x4E>(b1 ? r0 : r1);
}

// ---- elements
template <typename T>
__device__ __forceinline__ uint32_t load_bits(BufRes r, uint32_t off, uint32_t row) {
  if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, off, row, 0);
  else return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, row, 0);
}
template <typename T>
__device__ __forceinline__ float value(uint32_t bits) {
  return __uint_as_float(sizeof(T) == 4 ? bits : bits << 16);
}
template <typename T>
__device__ __forceinline__ void store_one(BufRes r, uint32_t off, uint32_t row, float v) {
  if constexpr (sizeof(T) == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, row, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, from_f32<T>(v)), r, off, row,
                                          0);
}
// The rows of a block of tokens as a buffer.
template <typename T>
__device__ __forceinline__ BufRes rows_buffer(const void* t, size_t row, int64_t ld, int rows,
                                              int cols) {
  return make_rsrc(static_cast<const T*>(t) + row * ld,
                   rows > 0 ? ((uint64_t)(rows - 1) * ld + cols) * sizeof(T) : 0);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sigm(float x) { return rcp_(1.f + exp2_(-x * kLog2e)); }

// softplus(v) = max(v, 0) + log(1 + t), t = exp(-|v|) in (0, 1], the logarithm as
// 2 atanh(s), s = t / (2 + t) <= 1/3 (log of a rounded 1 + t would lose a small
// step's relative precision). atanh(s) / s is a polynomial of degree 4 in s^2,
// fitted for this file by reweighted least squares on 0 <= s^2 <= 1/9: relative
// error 8e-9, 7e-8 evaluated in fp32. sig: sigmoid(v) (left out where not used).
__device__ __forceinline__ float softplus(float v, float& sig) {
  const float t = exp2_(-fabsf(v) * kLog2e);
  const float s = t * rcp_(2.f + t), q = s * s;
  float p = 0.14089155197143555f;
  p = __builtin_fmaf(p, q, 0.13980303704738617f);
  p = __builtin_fmaf(p, q, 0.20012454688549042f);
  p = __builtin_fmaf(p, q, 0.3333315849304199f);
  p = __builtin_fmaf(p, q, 1.f);
  sig = (v >= 0.f ? 1.f : t) * rcp_(1.f + t);
  return __builtin_fmaf(2.f * s, p, fmaxf(v, 0.f));  // (NaN through s)
}

// ---- places

// Where a wave works: its sequence and segment, and of each lane its channel and
// states. All but what depends on the lane is uniform in a wave.
struct Place {
  int b, seg, g, len;      // g: the group
  int c, n0;               // channel, first of the four states
  int sb, cw;              // the wave's block of states, its place among the channels' waves
  int j, q;                // lane % 4, lane / 4
  int blk0, blk1;          // blocks of the segment
  int off0, off1;          // blocks past the length, whose zeros it writes
  bool on;                 // the channel exists
  uint32_t cb;             // index of the workgroup's block of channels in its group
};
// segs: the segments that have workgroups, from `from` on. A sequence's blocks in
// use are shared by all of its segments, and so are those past its length (segments
// of equal length for all sequences leave the card to the long ones: a padded 8 x 2048
// x 1536 training step 472 instead of 453 us, with twelve workgroups a CU).
__device__ __forceinline__ Place place_of(const SScanArgs& A, int segs, int from = 0) {
  Place p;
  const int cw = channel_waves(A.N), gb = group_blocks(A.Ch, A.N, A.G), per = A.Ch / A.G;
  const unsigned cols = gb * A.G, id = blockIdx.x;
  const unsigned bs = id / cols, col = id - bs * cols;
  p.b = __builtin_amdgcn_readfirstlane(bs / segs);
  p.seg = __builtin_amdgcn_readfirstlane(bs - p.b * segs) + from;
  p.g = __builtin_amdgcn_readfirstlane(col / gb);
  p.cb = __builtin_amdgcn_readfirstlane(col - p.g * gb);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  p.sb = wave / cw;
  p.cw = wave - p.sb * cw;
  const int lane = lane_id();
  p.j = lane & 3;
  p.q = lane >> 2;
  const int in = (p.cb * cw + p.cw) * kWaveCh + p.q;
  p.on = in < per;
  p.c = p.g * per + min(in, per - 1);
  p.n0 = p.sb * kStates + p.j * kQ;
  p.len = A.T;
  if (A.lens) p.len = __builtin_amdgcn_readfirstlane(min(max(A.lens[p.b], 0), A.T));
  const int nblk = (A.T + kTok - 1) / kTok, live = (p.len + kTok - 1) / kTok;
  const int run = (live + A.segs - 1) / A.segs, off = (nblk - live + A.segs - 1) / A.segs;
  p.blk0 = min(live, p.seg * run);
  p.blk1 = min(live, p.blk0 + run);
  p.off0 = min(nblk, live + p.seg * off);
  p.off1 = min(nblk, p.off0 + off);
  return p;
}

// The four states' values of a [.., N] row (zeros past N, or where off).
__device__ __forceinline__ floatx4 load_states(const float* row, int n0, int N, bool on) {
  floatx4 v = {0.f, 0.f, 0.f, 0.f};
  if (!row || !on) return v;
  if (N % 4 == 0) {
    if (n0 < N) v = *reinterpret_cast<const floatx4*>(row + n0);
  } else {
#pragma unroll
    for (int k = 0; k < kQ; ++k)
      if (n0 + k < N) v[k] = row[n0 + k];
  }
  return v;
}
__device__ __forceinline__ void store_states(float* row, int n0, int N, floatx4 v) {
  if (N % 4 == 0) {
    if (n0 < N) *reinterpret_cast<floatx4*>(row + n0) = v;
  } else {
#pragma unroll
    for (int k = 0; k < kQ; ++k)
      if (n0 + k < N) row[n0 + k] = v[k];
  }
}

// One value per token and channel of a block: lane (q, j) holds tokens 4 i + j.
// The buffer ends with the block's rows in use, so that a row past them reads
// zeros (and a store there is dropped); lanes without a channel are out of range.
struct Four {
  uint32_t v[4];
};
__device__ __forceinline__ uint32_t four_offset(const Place& p, uint32_t pitch, uint32_t es) {
  return p.on ? p.j * pitch + p.c * es : kOOB;
}
template <typename T>
__device__ __forceinline__ Four load_four(const void* t, int64_t ld, const SScanArgs& A,
                                          const Place& p, int blk) {
  const int t0 = blk * kTok, rows = min(kTok, p.len - t0);
  const BufRes r = rows_buffer<T>(t, (size_t)p.b * A.T + t0, ld, rows, A.Ch);
  const uint32_t pitch = (uint32_t)ld * sizeof(T), off = four_offset(p, pitch, sizeof(T));
  Four f;
  if (rows == kTok) {  // no arithmetic per row
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = load_bits<T>(r, off, 4 * i * pitch);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = load_bits<T>(r, off + 4 * i * pitch, 0);
  }
  return f;
}
template <typename T>
__device__ __forceinline__ void store_four(void* t, int64_t ld, const SScanArgs& A,
                                           const Place& p, int blk, const float (&v)[4]) {
  const int t0 = blk * kTok, rows = min(kTok, A.T - t0);
  const BufRes r = rows_buffer<T>(t, (size_t)p.b * A.T + t0, ld, rows, A.Ch);
  const uint32_t pitch = (uint32_t)ld * sizeof(T), off = four_offset(p, pitch, sizeof(T));
  if (rows == kTok) {
#pragma unroll
    for (int i = 0; i < 4; ++i) store_one<T>(r, off, 4 * i * pitch, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) store_one<T>(r, off + 4 * i * pitch, 0, v[i]);
  }
}
// The values of a block that reaches past the length: zeros there.
__device__ __forceinline__ void clear_tail(const Place& p, int blk, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = blk * kTok + 4 * i + p.j < p.len ? v[i] : 0.f;
}

// B (or C) of a block of tokens: lane (q, j) loads states n0 .. n0 + 3 of token q,
// zeros past the length and past N.
template <typename T> struct Bits;
template <> struct Bits<float> { typedef int t __attribute__((ext_vector_type(4))); };
template <> struct Bits<bf16> { typedef int t __attribute__((ext_vector_type(2))); };
template <typename T>
__device__ __forceinline__ typename Bits<T>::t load_bc(const void* t, const SScanArgs& A,
                                                       const Place& p, int blk, bool vec) {
  const int t0 = blk * kTok, rows = min(kTok, p.len - t0);
  const BufRes r = rows_buffer<T>(t, (size_t)p.b * A.T + t0, A.ldbc, rows, A.G * A.N);
  constexpr uint32_t ES = sizeof(T);
  const uint32_t off = ((uint32_t)p.q * (uint32_t)A.ldbc + p.g * A.N + p.n0) * ES;
  const bool row = p.q < rows;
  typename Bits<T>::t v;
  if (vec) {
    const uint32_t o = row && p.n0 < A.N ? off : kOOB;
    if constexpr (ES == 4) v = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
    else v = __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, 0);
  } else {
    uint32_t e[kQ];
#pragma unroll
    for (int k = 0; k < kQ; ++k)
      e[k] = load_bits<T>(r, row && p.n0 + k < A.N ? off + k * ES : kOOB, 0);
    if constexpr (ES == 4) v = typename Bits<T>::t{(int)e[0], (int)e[1], (int)e[2], (int)e[3]};
    else v = typename Bits<T>::t{(int)(e[0] | e[1] << 16), (int)(e[2] | e[3] << 16)};
  }
  return v;
}
template <typename T>
__device__ __forceinline__ floatx4 widen(typename Bits<T>::t v) {
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(floatx4, v);
  else
    return floatx4{__uint_as_float((uint32_t)v[0] << 16), __uint_as_float((uint32_t)v[0] & 0xFFFF0000u),
                   __uint_as_float((uint32_t)v[1] << 16), __uint_as_float((uint32_t)v[1] & 0xFFFF0000u)};
}
// Whether four states of a row can be loaded at once.
template <typename T> __device__ __forceinline__ bool vec_bc(const SScanArgs& A) {
  return A.N % 4 == 0 && A.ldbc % 4 == 0;
}

// A wave's copy of B and C of 16 tokens.
struct BC {
  floatx4 b[kTok][4], c[kTok][4];
};

// The workspace of the segments' pass: [Bt][segs][Ch][16 blocks of states] states,
// then [Bt][segs][Ch] sums of delta.
struct SegBoard {
  float *state, *sum;
  int np;
  __device__ explicit SegBoard(const SScanArgs& A) {
    np = state_blocks(A.N) * kStates;
    state = static_cast<float*>(A.ws);
    sum = state + (size_t)A.Bt * A.segs * A.Ch * np;
  }
  __device__ size_t row(const SScanArgs& A, const Place& p, int seg) const {
    return ((size_t)p.b * A.segs + seg) * A.Ch + p.c;
  }
};

// f(constant 0 .. 3), and the other way.
template <class F> __device__ __forceinline__ void up4(F f) {
  f(std::integral_constant<int, 0>());
  f(std::integral_constant<int, 1>());
  f(std::integral_constant<int, 2>());
  f(std::integral_constant<int, 3>());
}
template <class F> __device__ __forceinline__ void down4(F f) {
  f(std::integral_constant<int, 3>());
  f(std::integral_constant<int, 2>());
  f(std::integral_constant<int, 1>());
  f(std::integral_constant<int, 0>());
}

// A times log2 e (decays are powers of 2), -inf as the largest finite number: a step of
// zero (a token past the length, a segment without tokens) then keeps the state as with
// any other decay, and any other step forgets it all the same. (NaN stays.)
__device__ __forceinline__ floatx4 rates(floatx4 a) {
  constexpr float kMost = 3.4028234e38f;
  a = a * kLog2e;
#pragma unroll
  for (int k = 0; k < kQ; ++k) a[k] = a[k] < -kMost ? -kMost : a[k];
  return a;
}

// A lane's constants: A (rates), dt_bias, D. Lanes
// without a channel hold zeros, so that all they compute from is zero.
struct Coef {
  floatx4 A2;
  float bias, D;
  __device__ Coef(const SScanArgs& A, const Place& p) {
    A2 = rates(load_states(A.A + (size_t)p.c * A.N, p.n0, A.N, p.on));
    bias = A.bias && p.on ? A.bias[p.c] : 0.f;
    D = A.D && p.on ? A.D[p.c] : 0.f;
  }
};

// v, carried through the segments from `from` up (or down) to `to`, without it: a
// batch of them loaded at once. Where A > 0 a segment's factor may pass float32's range
// while v, and v times it, do not: it is applied as two halves, each held below 2^127,
// so that a zero stays one (any other number is past the range after both of those).
__device__ __forceinline__ void join_segments(const SScanArgs& A, const Place& p, const Coef& co,
                                              int from, int to, floatx4& v) {
  constexpr int kBatch = 8;
  const SegBoard sb(A);
  const int step = to >= from ? 1 : -1, n = (to - from) * step;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    floatx4 e[kBatch];
    float d[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const size_t row = sb.row(A, p, from + step * min(i0 + i, n - 1));
      e[i] = *reinterpret_cast<const floatx4*>(sb.state + row * sb.np + p.n0);
      d[i] = sb.sum[row];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i >= n) break;
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        const float half = exp2_(fminf(0.5f * d[i] * co.A2[k], 127.f));
        v[k] = __builtin_fmaf(half, half * v[k], e[i][k]);
      }
    }
  }
}

// ---------------------------------------------------------------- forward

// Each segment's state from zero, and its sum of delta (of all but the last).
template <typename T>
__global__ __launch_bounds__(64 * kMaxWaves) void sscan_ends_kernel(SScanArgs A) {
  __shared__ floatx4 lds[kMaxWaves][kTok][4];
  const Place p = place_of(A, A.segs - 1);
  floatx4(&bt)[kTok][4] = lds[threadIdx.x >> 6];
  const bool vec = vec_bc<T>(A);
  const Coef co(A, p);
  floatx4 h = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  Four xr, dr;
  typename Bits<T>::t br;
  auto fetch = [&](int blk) {
    xr = load_four<T>(A.x, A.ldx, A, p, blk);
    dr = load_four<T>(A.dt, A.lddt, A, p, blk);
    br = load_bc<T>(A.B, A, p, blk, vec);
  };
  if (p.blk0 < p.blk1) fetch(p.blk0);
  for (int blk = p.blk0; blk < p.blk1; ++blk) {
    float delta[4], u[4], sig;
#pragma unroll
    for (int i = 0; i < 4; ++i) delta[i] = softplus(value<T>(dr.v[i]) + co.bias, sig);
    if ((blk + 1) * kTok > p.len) clear_tail(p, blk, delta);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = delta[i] * value<T>(xr.v[i]);
      sum += delta[i];
    }
    bt[p.q][p.j] = widen<T>(br);
    if (blk + 1 < p.blk1) fetch(blk + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      up4([&](auto Q) {
        const floatx4 Bv = bt[4 * i + Q()][p.j];
        const float d = quad<Q()>(delta[i]), ut = quad<Q()>(u[i]);
#pragma unroll
        for (int k = 0; k < kQ; ++k) h[k] = __builtin_fmaf(exp2_(d * co.A2[k]), h[k], ut * Bv[k]);
      });
  }
  sum = quad_sum(sum);
  if (!p.on) return;
  const SegBoard sb(A);
  const size_t row = sb.row(A, p, p.seg);
  *reinterpret_cast<floatx4*>(sb.state + row * sb.np + p.n0) = h;
  if (p.sb == 0 && p.j == 0) sb.sum[row] = sum;
}

// SPLIT: several blocks of states in the workgroup.
template <typename T, bool GATED, bool SPLIT>
__global__ __launch_bounds__(SPLIT ? 64 * kMaxWaves : 256) void sscan_kernel(SScanArgs A) {
  constexpr int WV = SPLIT ? kMaxWaves : 4;
  __shared__ BC lds[WV];
  __shared__ float part[SPLIT ? 2 : 1][SPLIT ? WV : 1][4][64];
  const Place p = place_of(A, A.segs);
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int nb = state_blocks(A.N), cw = channel_waves(A.N), np = nb * kStates;
  BC& bc = lds[wave];
  const bool vec = vec_bc<T>(A);
  const Coef co(A, p);
  const int nblk = (A.T + kTok - 1) / kTok;
  Four xr, dr, zr;
  typename Bits<T>::t br, cr;
  auto fetch = [&](int blk) {
    xr = load_four<T>(A.x, A.ldx, A, p, blk);
    dr = load_four<T>(A.dt, A.lddt, A, p, blk);
    if constexpr (GATED) zr = load_four<T>(A.z, A.ldz, A, p, blk);
    br = load_bc<T>(A.B, A, p, blk, vec);
    cr = load_bc<T>(A.C, A, p, blk, vec);
  };
  if (p.blk0 < p.blk1) fetch(p.blk0);
  // the state that enters the segment
  floatx4 h = load_states(A.h_init ? A.h_init + ((size_t)p.b * A.Ch + p.c) * A.N : nullptr, p.n0,
                          A.N, p.on);
  if (A.segs > 1) {
    join_segments(A, p, co, 0, p.seg, h);
  }
  for (int blk = p.blk0; blk < p.blk1; ++blk) {
    if (A.carry && p.on)
      *reinterpret_cast<floatx4*>(A.carry + (((size_t)p.b * nblk + blk) * A.Ch + p.c) * np +
                                  p.n0) = h;
    float x[4], delta[4], u[4], gate[4], out[4], sig;
#pragma unroll
    for (int i = 0; i < 4; ++i) delta[i] = softplus(value<T>(dr.v[i]) + co.bias, sig);
    const bool tail = (blk + 1) * kTok > p.len;
    if (tail) clear_tail(p, blk, delta);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = value<T>(xr.v[i]);
      u[i] = delta[i] * x[i];
      if constexpr (GATED) {
        const float z = value<T>(zr.v[i]);
        gate[i] = z * sigm(z);
      }
    }
    bc.b[p.q][p.j] = widen<T>(br);
    bc.c[p.q][p.j] = widen<T>(cr);
    if (blk + 1 < p.blk1) fetch(blk + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[4];
      up4([&](auto Q) {
        const floatx4 Bv = bc.b[4 * i + Q()][p.j], Cv = bc.c[4 * i + Q()][p.j];
        const float d = quad<Q()>(delta[i]), ut = quad<Q()>(u[i]);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
          h[k] = __builtin_fmaf(exp2_(d * co.A2[k]), h[k], ut * Bv[k]);
          s = __builtin_fmaf(Cv[k], h[k], s);
        }
        y[Q()] = s;
      });
      out[i] = quad_spread(y, p.j);
    }
    if constexpr (SPLIT) {
      const int half = blk & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) part[half][wave][i][lane] = out[i];
      stage_barrier();
      if (p.sb == 0)
        for (int s = 1; s < nb; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] += part[half][s * cw + p.cw][i][lane];
    }
    if (!SPLIT || p.sb == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        out[i] = __builtin_fmaf(co.D, x[i], out[i]);
        if constexpr (GATED) out[i] *= gate[i];
      }
      if (tail) clear_tail(p, blk, out);
      store_four<T>(A.y, A.Ch, A, p, blk, out);
    }
  }
  if (!SPLIT || p.sb == 0) {
    const float zeros[4] = {0.f, 0.f, 0.f, 0.f};
    for (int blk = p.off0; blk < p.off1; ++blk)
      store_four<T>(A.y, A.Ch, A, p, blk, zeros);
  }
  if (A.h_final && p.on && p.seg == A.segs - 1)
    store_states(A.h_final + ((size_t)p.b * A.Ch + p.c) * A.N, p.n0, A.N, h);
}

// ---------------------------------------------------------------- backward

// Each segment's gradient of the state that enters it, from zero behind it, and
// its sum of delta (of all but the first).
template <typename T, bool GATED>
__global__ __launch_bounds__(64 * kMaxWaves) void sscan_bwd_ends_kernel(SScanArgs A) {
  __shared__ floatx4 lds[kMaxWaves][kTok][4];
  const Place p = place_of(A, A.segs - 1, 1);
  floatx4(&ct)[kTok][4] = lds[threadIdx.x >> 6];
  const bool vec = vec_bc<T>(A);
  const Coef co(A, p);
  floatx4 c = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  Four dr, gr, zr;
  typename Bits<T>::t cr;
  auto fetch = [&](int blk) {
    dr = load_four<T>(A.dt, A.lddt, A, p, blk);
    gr = load_four<T>(A.dy, A.Ch, A, p, blk);
    if constexpr (GATED) zr = load_four<T>(A.z, A.ldz, A, p, blk);
    cr = load_bc<T>(A.C, A, p, blk, vec);
  };
  if (p.blk0 < p.blk1) fetch(p.blk1 - 1);
  for (int blk = p.blk1 - 1; blk >= p.blk0; --blk) {
    float delta[4], v[4], sig;
#pragma unroll
    for (int i = 0; i < 4; ++i) delta[i] = softplus(value<T>(dr.v[i]) + co.bias, sig);
    if ((blk + 1) * kTok > p.len) clear_tail(p, blk, delta);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = value<T>(gr.v[i]);
      if constexpr (GATED) {
        const float z = value<T>(zr.v[i]);
        v[i] *= z * sigm(z);
      }
      sum += delta[i];
    }
    ct[p.q][p.j] = widen<T>(cr);
    if (blk > p.blk0) fetch(blk - 1);
#pragma unroll
    for (int i = 3; i >= 0; --i)
      down4([&](auto Q) {
        const floatx4 Cv = ct[4 * i + Q()][p.j];
        const float d = quad<Q()>(delta[i]), vt = quad<Q()>(v[i]);
#pragma unroll
        for (int k = 0; k < kQ; ++k)
          c[k] = exp2_(d * co.A2[k]) * __builtin_fmaf(Cv[k], vt, c[k]);
      });
  }
  sum = quad_sum(sum);
  if (!p.on) return;
  const SegBoard sb(A);
  const size_t row = sb.row(A, p, p.seg);
  *reinterpret_cast<floatx4*>(sb.state + row * sb.np + p.n0) = c;
  if (p.sb == 0 && p.j == 0) sb.sum[row] = sum;
}

// The backward's workspace: the segments' board (where there are several), then
//   bc [G][blocks of channels][M][2][np]  partial dB and dC,
//   da [Bt segs][Ch][np]  and  dd [Bt segs][2][Ch]  partial dA, dD and ddt_bias.
struct BwdBoard {
  float *bc, *da, *dd;
  size_t bc_step;  // of a block of channels
  int np;
  __host__ __device__ explicit BwdBoard(const SScanArgs& A) {
    np = state_blocks(A.N) * kStates;
    const size_t rows = (size_t)A.Bt * A.segs;
    float* p = static_cast<float*>(A.ws);
    if (A.segs > 1) p += (rows * A.Ch * (np + 1) + 3) / 4 * 4;
    bc = p;
    bc_step = (size_t)A.Bt * A.T * 2 * np;
    da = bc + bc_step * A.G * group_blocks(A.Ch, A.N, A.G);
    dd = da + rows * A.Ch * np;
  }
  __host__ __device__ size_t floats(const SScanArgs& A) const {
    return dd - static_cast<float*>(A.ws) + (size_t)A.Bt * A.segs * 2 * A.Ch;
  }
};

// Values a and b of lanes l and l ^ 32 (or l ^ 16) exchanged and added: one register
// with a's sum in the lower and b's in the upper of the two.
__device__ __forceinline__ float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The same over lanes l ^ 8 and l ^ 4 (of rows of 16 lanes).
__device__ __forceinline__ float fold8(float a, float b, bool hi) {
  return (hi ? b : a) + dpp<0x128>(hi ? a : b);  // row_ror:8
}
__device__ __forceinline__ float fold4(float a, float b, bool hi) {
  const float lo = a + dpp<0x104>(a);   // row_shl:4, from lane + 4
  const float up = b + dpp<0x114>(b);   // row_shr:4, from lane - 4
  return hi ? up : lo;
}

template <typename T, bool GATED, bool SPLIT>
__global__ __launch_bounds__(SPLIT ? 64 * kMaxWaves : 256, SPLIT ? 1 : 2) void sscan_bwd_kernel(
    SScanArgs A) {
  constexpr int WV = SPLIT ? kMaxWaves : 4;
  __shared__ BC lds[WV];
  __shared__ floatx4 kept[WV][4][64];  // x, sigmoid, dy silu'(z), u: for the block's end
  __shared__ float2 dbc[2][WV][kTok][kStates];  // [token][kind, pair of states]
  __shared__ float part[SPLIT ? 2 : 1][SPLIT ? WV : 1][12][64];
  const Place p = place_of(A, A.segs);
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int nb = state_blocks(A.N), cw = channel_waves(A.N);
  BC& bc = lds[wave];
  const bool vec = vec_bc<T>(A);
  const Coef co(A, p);
  const int nblk = (A.T + kTok - 1) / kTok;
  const BwdBoard board(A);
  const int np = board.np;
  Four xr, dr, zr, gr;
  typename Bits<T>::t br, cr;
  floatx4 hr;
  auto fetch = [&](int blk) {
    xr = load_four<T>(A.x, A.ldx, A, p, blk);
    dr = load_four<T>(A.dt, A.lddt, A, p, blk);
    gr = load_four<T>(A.dy, A.Ch, A, p, blk);
    if constexpr (GATED) zr = load_four<T>(A.z, A.ldz, A, p, blk);
    br = load_bc<T>(A.B, A, p, blk, vec);
    cr = load_bc<T>(A.C, A, p, blk, vec);
    // (of a lane without a channel: another channel's, which meets only zeros)
    hr = *reinterpret_cast<const floatx4*>(
        A.carry_in + (((size_t)p.b * nblk + blk) * A.Ch + p.c) * np + p.n0);
  };
  if (p.blk0 < p.blk1) fetch(p.blk1 - 1);
  // the gradient of the state that leaves the segment
  floatx4 c = load_states(A.dh_final ? A.dh_final + ((size_t)p.b * A.Ch + p.c) * A.N : nullptr,
                          p.n0, A.N, p.on);
  if (A.segs > 1) {
    join_segments(A, p, co, A.segs - 1, p.seg, c);
    if (!p.on) c = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  floatx4 dA = {0.f, 0.f, 0.f, 0.f};
  float dD = 0.f, dbias = 0.f;
  for (int blk = p.blk1 - 1; blk >= p.blk0; --blk) {
    const int half = blk & 1;
    const bool tail = (blk + 1) * kTok > p.len;
    float delta[4], u[4], v[4];
    {
      float sig[4], g2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) delta[i] = softplus(value<T>(dr.v[i]) + co.bias, sig[i]);
      if (tail) clear_tail(p, blk, delta);
      floatx4 xs;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xs[i] = value<T>(xr.v[i]);
        u[i] = delta[i] * xs[i];
        v[i] = value<T>(gr.v[i]);
        if constexpr (GATED) {
          const float z = value<T>(zr.v[i]), sg = sigm(z);
          g2[i] = v[i] * (sg * __builtin_fmaf(z, 1.f - sg, 1.f));
          v[i] *= z * sg;
        }
        dD = __builtin_fmaf(v[i], xs[i], dD);
      }
      kept[wave][0][lane] = xs;
      kept[wave][1][lane] = floatx4{sig[0], sig[1], sig[2], sig[3]};
      if constexpr (GATED) kept[wave][2][lane] = floatx4{g2[0], g2[1], g2[2], g2[3]};
    }
    bc.b[p.q][p.j] = widen<T>(br);
    bc.c[p.q][p.j] = widen<T>(cr);
    floatx4 h[kTok + 1], a[kTok];
    h[0] = hr;
    // the block's states and u
    float eb[4], fa[4];
    floatx4 uy = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[4];
      up4([&](auto Q) {
        const int t = 4 * i + Q();
        const floatx4 Bv = bc.b[t][p.j];
        const float d = quad<Q()>(delta[i]), ut = quad<Q()>(u[i]);
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
          a[t][k] = exp2_(d * co.A2[k]);
          h[t + 1][k] = __builtin_fmaf(a[t][k], h[t][k], ut * Bv[k]);
        }
        if constexpr (GATED) {
          const floatx4 Cv = bc.c[t][p.j];
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < kQ; ++k) s = __builtin_fmaf(Cv[k], h[t + 1][k], s);
          y[Q()] = s;
        }
      });
      if constexpr (GATED) uy[i] = quad_spread(y, p.j);
      __builtin_amdgcn_sched_barrier(0);  // (reads of many tokens ahead would spill)
    }
    if constexpr (GATED) kept[wave][3][lane] = uy;
    // back through it
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      float yb[4], ya[4], w[2][8], r16[2][8];  // w: two tokens' dB and dC of this lane
      down4([&](auto Q) {
        const int t = 4 * i + Q();
        const floatx4 Bv = bc.b[t][p.j], Cv = bc.c[t][p.j];
        const float d = quad<Q()>(delta[i]), ut = quad<Q()>(u[i]), vt = quad<Q()>(v[i]);
        float sb = 0.f, sa = 0.f;
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
          const float e = __builtin_fmaf(Cv[k], vt, c[k]);
          c[k] = a[t][k] * e;
          const float flow = c[k] * h[t][k];
          sb = __builtin_fmaf(e, Bv[k], sb);
          sa = __builtin_fmaf(flow, co.A2[k], sa);
          dA[k] = __builtin_fmaf(flow, d, dA[k]);
          w[Q() & 1][k] = e * ut;
          w[Q() & 1][4 + k] = vt * h[t + 1][k];
        }
        yb[Q()] = sb;
        ya[Q()] = sa;
        // sums over the wave's channels: lane (bit 5: the later token of a pair, bit 4:
        // the pair, bit 3: dB or dC, bit 2: which pair of its four states, j) ends with
        // two of them
        if constexpr (Q() % 2 == 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) r16[Q() / 2][k] = fold32(w[0][k], w[1][k]);
        }
      });
      eb[i] = quad_spread(yb, p.j);
      fa[i] = quad_spread(ya, p.j);
      float r4[4], r2[2];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r4[k] = fold8(fold16(r16[0][k], r16[1][k]), fold16(r16[0][4 + k], r16[1][4 + k]), lane & 8);
#pragma unroll
      for (int k = 0; k < 2; ++k) r2[k] = fold4(r4[k], r4[2 + k], lane & 4);
      const int t = 4 * i + 2 * (lane >> 4 & 1) + (lane >> 5);
      dbc[half][wave][t][(lane >> 3 & 1) * 8 + 2 * p.j + (lane >> 2 & 1)] =
          make_float2(r2[0], r2[1]);
      // the next block's loads, once half of this one's states are done with
      if (i == 2 && blk > p.blk0) fetch(blk - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (GATED) part[half][wave][i][lane] = kept[wave][3][lane][i];
        part[half][wave][4 + i][lane] = eb[i];
        part[half][wave][8 + i][lane] = fa[i];
      }
    }
    stage_barrier();
    // partial dB and dC of the workgroup's channels: the waves of channels in order
    {
      const int rows = min(kTok, A.T - blk * kTok);
      float* out = board.bc + (size_t)(p.g * group_blocks(A.Ch, A.N, A.G) + p.cb) * board.bc_step +
                   ((size_t)p.b * A.T + blk * kTok) * 2 * np;
      for (int q = threadIdx.x; q < nb * kTok * kStates; q += blockDim.x) {
        const int s = q / (kTok * kStates), t = q / kStates % kTok, m = q % kStates;
        float2 r = dbc[half][s * cw][t][m];
        for (int w = 1; w < cw; ++w) {
          const float2 o = dbc[half][s * cw + w][t][m];
          r.x += o.x;
          r.y += o.y;
        }
        if (t < rows)
          *reinterpret_cast<float2*>(out + ((size_t)2 * t + m / 8) * np + s * kStates + 2 * (m % 8)) = r;
      }
    }
    if constexpr (GATED) uy = kept[wave][3][lane];
    if constexpr (SPLIT) {
      if (p.sb == 0)
        for (int s = 1; s < nb; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (GATED) uy[i] += part[half][s * cw + p.cw][i][lane];
            eb[i] += part[half][s * cw + p.cw][4 + i][lane];
            fa[i] += part[half][s * cw + p.cw][8 + i][lane];
          }
    }
    if (!SPLIT || p.sb == 0) {
      const floatx4 x = kept[wave][0][lane], sig = kept[wave][1][lane];
      float ox[4], od[4], oz[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ox[i] = __builtin_fmaf(delta[i], eb[i], co.D * v[i]);
        od[i] = __builtin_fmaf(x[i], eb[i], fa[i] * kLn2) * sig[i];
      }
      if (tail) {
        clear_tail(p, blk, ox);
        clear_tail(p, blk, od);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) dbias += od[i];
      store_four<T>(A.dx, A.lddx, A, p, blk, ox);
      store_four<T>(A.ddt, A.ldddt, A, p, blk, od);
      if constexpr (GATED) {
        const floatx4 g2 = kept[wave][2][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) oz[i] = g2[i] * __builtin_fmaf(co.D, x[i], uy[i]);
        if (tail) clear_tail(p, blk, oz);
        store_four<T>(A.dz, A.lddz, A, p, blk, oz);
      }
    }
  }
  if (!SPLIT || p.sb == 0) {
    const float zeros[4] = {0.f, 0.f, 0.f, 0.f};
    for (int blk = p.off0; blk < p.off1; ++blk) {
      store_four<T>(A.dx, A.lddx, A, p, blk, zeros);
      store_four<T>(A.ddt, A.ldddt, A, p, blk, zeros);
      if constexpr (GATED) store_four<T>(A.dz, A.lddz, A, p, blk, zeros);
    }
  }
  dD = quad_sum(dD);
  dbias = quad_sum(dbias);
  if (!p.on) return;
  const size_t row = (size_t)p.b * A.segs + p.seg;
  *reinterpret_cast<floatx4*>(board.da + (row * A.Ch + p.c) * np + p.n0) = dA;
  if (p.sb == 0 && p.j == 0) {
    board.dd[(row * 2 + 0) * A.Ch + p.c] = dD;
    board.dd[(row * 2 + 1) * A.Ch + p.c] = dbias;
  }
  if (A.dh_init && p.seg == 0)
    store_states(A.dh_init + ((size_t)p.b * A.Ch + p.c) * A.N, p.n0, A.N, c);
}

// The partial sums, added in order: dB and dC over the group's blocks of channels
// (a thread per token and state; zeros past a sequence's length), dA, dD and
// ddt_bias over sequences and segments (from workgroup `first` on).
template <typename T>
__global__ __launch_bounds__(256) void sscan_sum_kernel(SScanArgs A, unsigned first) {
  const BwdBoard bd(A);
  if (blockIdx.x < first) {
    const int gb = group_blocks(A.Ch, A.N, A.G);
    const size_t q = (size_t)blockIdx.x * 256 + threadIdx.x, cols = 2 * A.G * A.N;
    const size_t m = q / cols;
    if (m >= (size_t)A.Bt * A.T) return;
    const int r = (int)(q - m * cols), kind = r / (A.G * A.N), gn = r - kind * A.G * A.N;
    const int g = gn / A.N, n = gn - g * A.N;
    float v = 0.f;
    int len = A.T;
    const int b = (int)(m / A.T), t = (int)(m - (size_t)b * A.T);
    if (A.lens) len = A.lens[b];
    if (t < len) {
      const float* p = bd.bc + (size_t)g * gb * bd.bc_step + (m * 2 + kind) * bd.np + n;
#pragma unroll 8
      for (int s = 0; s < gb; ++s) v += p[s * bd.bc_step];
    }
    static_cast<T*>(kind ? A.dC : A.dB)[m * A.lddbc + gn] = from_f32<T>(v);
    return;
  }
  // 64 of them a workgroup, a quarter of the rows each wave
  __shared__ float sum[4][64];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const size_t q = (size_t)(blockIdx.x - first) * 64 + lane, na = (size_t)A.Ch * A.N;
  const int rows = A.Bt * A.segs, per = (rows + 3) / 4, r1 = min(rows, (wave + 1) * per);
  const float* p = nullptr;
  size_t pitch = 0;
  if (q < na) {
    const size_t c = q / A.N, n = q - c * A.N;
    p = bd.da + c * bd.np + n;
    pitch = (size_t)A.Ch * bd.np;
  } else if (q < na + 2 * (size_t)A.Ch) {
    p = bd.dd + (q - na);
    pitch = 2 * (size_t)A.Ch;
  }
  float v = 0.f;
  if (p) {
#pragma unroll 8
    for (int r = wave * per; r < r1; ++r) v += p[r * pitch];
  }
  sum[wave][lane] = v;
  __syncthreads();
  if (wave || !p) return;
  v = sum[0][lane] + sum[1][lane] + sum[2][lane] + sum[3][lane];
  if (q < na) {
    A.dA[q] = v;
  } else {
    const size_t i = q - na;
    float* out = i < (size_t)A.Ch ? A.dD : A.dbias;
    if (out) out[i < (size_t)A.Ch ? i : i - A.Ch] = v;
  }
}

// ---------------------------------------------------------------- one token

// Four lanes a channel, four states a lane at a time; R sequences a thread, whose
// states are requested together and which share A, D and dt_bias.
template <typename T, int R>
__global__ __launch_bounds__(256) void sscan_step_kernel(SScanArgs A) {
  const size_t q = ((size_t)blockIdx.x * 256 + threadIdx.x) >> 2;
  const int j = threadIdx.x & 3;
  const size_t bq = q / A.Ch;
  const int b0 = (int)bq * R;
  if (bq * R >= (size_t)A.Bt) return;  // (the four lanes together)
  const int c = (int)(q - bq * A.Ch), g = c / (A.Ch / A.G);
  const bool vec = vec_bc<T>(A);
  const float* Ap = A.A + (size_t)c * A.N;
  const float bias = A.bias ? A.bias[c] : 0.f, D = A.D ? A.D[c] : 0.f;
  // (past the last sequence: its values again, not stored)
  size_t b[R];
  float x[R], dt[R], z[R], s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    b[r] = min(b0 + r, A.Bt - 1);
    x[r] = to_f32(static_cast<const T*>(A.x)[b[r] * A.ldx + c]);
    dt[r] = to_f32(static_cast<const T*>(A.dt)[b[r] * A.lddt + c]);
    z[r] = A.z ? to_f32(static_cast<const T*>(A.z)[b[r] * A.ldz + c]) : 0.f;
    s[r] = 0.f;
  }
  for (int n0 = 4 * j; n0 < A.N; n0 += kStates) {
    floatx4 h[R];
    float Bv[R][4], Cv[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      h[r] = load_states(A.h_prev + (b[r] * A.Ch + c) * A.N, n0, A.N, true);
      const T* Bp = static_cast<const T*>(A.B) + b[r] * A.ldbc + (size_t)g * A.N;
      const T* Cp = static_cast<const T*>(A.C) + b[r] * A.ldbc + (size_t)g * A.N;
      if (vec) {
        typedef typename Vec<T>::x4 V4;
        const V4 bv = *reinterpret_cast<const V4*>(Bp + n0),
                 cv = *reinterpret_cast<const V4*>(Cp + n0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          Bv[r][k] = to_f32(bv[k]);
          Cv[r][k] = to_f32(cv[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          Bv[r][k] = n0 + k < A.N ? to_f32(Bp[n0 + k]) : 0.f;
          Cv[r][k] = n0 + k < A.N ? to_f32(Cp[n0 + k]) : 0.f;
        }
      }
    }
    const floatx4 Av = rates(load_states(Ap, n0, A.N, true));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float sig;
      const float delta = softplus(dt[r] + bias, sig), u = delta * x[r];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[r][k] = __builtin_fmaf(exp2_(delta * Av[k]), h[r][k], u * Bv[r][k]);
        s[r] = __builtin_fmaf(Cv[r][k], h[r][k], s[r]);
      }
      float* to = A.h + (b[r] * A.Ch + c) * A.N;
      if (b0 + r >= A.Bt) continue;
      // past the L2's reuse order (a hint) where four lanes store 64 aligned bytes or a wave's
      // channels are one run; us without and with it: 256 x 4096 x 4 22.2, 21.8, x 16 37.3,
      // 25.5, x 32 78.3, 68.3, x 64 151, 140, 64 x 4096 x 64 45.2, 27.7; but x 20 57.3, 63.6
      if (A.N % kStates == 0 || (A.N < kStates && A.N % 4 == 0))
        __builtin_nontemporal_store(h[r], reinterpret_cast<floatx4*>(to + n0));
      else
        store_states(to, n0, A.N, h[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s[r] = __builtin_fmaf(D, x[r], quad_sum(s[r]));
    if (A.z) s[r] *= z[r] * sigm(z[r]);
    if (j == 0 && b0 + r < A.Bt) static_cast<T*>(A.y)[b[r] * A.Ch + c] = from_f32<T>(s[r]);
  }
}

// ---------------------------------------------------------------- launch

// Segments per sequence, as many as give at most kWant workgroups, eight a CU: fewer
// leave CUs idle at the end, more join more segments and start more walks. Up to 6, 8,
// 12 and 16 a CU: 65536 x 2048 forward 1023, 984, 981, 996 us, 32 x 700 x 3000 forward
// 310, 307, 395, 395, a padded 8 x 2048 x 1536 training step 461, 441, 453, 461, an
// unpadded one 706, 711, 696, 718, a padded 64 x 512 x 1536 one 771, 771, 814, 817 (at
// least 12: 32 x 700 x 3000 423, the others as up to 12). And at most kSegRoot
// sqrt(blocks): where so few workgroups run that each one's time is that of its own
// instructions, a block takes some 2 to 3 us and the join some 0.15 us a segment, and
// the sum of both is least about there (a 2 x 777 x 402 fp32 training step: 59 us,
// 70 without this limit).
constexpr int64_t kWant = 8 * 256;
constexpr double kSegRoot = 4;
void segments(SScanArgs& A) {
  const int64_t wg = (int64_t)A.Bt * A.G * group_blocks(A.Ch, A.N, A.G);
  const int nblk = (A.T + kTok - 1) / kTok;
  const int64_t most = (int64_t)(kSegRoot * std::sqrt((double)nblk));
  int64_t s = std::max<int64_t>(1, std::min({kWant / wg, most, (int64_t)nblk}));
  const int64_t run = (nblk + s - 1) / s;
  A.segs = (int)((nblk + run - 1) / run);
}

unsigned workgroups(const SScanArgs& A, int segs) {
  return (unsigned)((int64_t)A.Bt * segs * A.G * group_blocks(A.Ch, A.N, A.G));
}
int threads_of(const SScanArgs& A) { return 64 * channel_waves(A.N) * state_blocks(A.N); }

SScanArgs sizes(int Bt, int T, int Ch, int N, int G) {
  SScanArgs A{};
  A.Bt = Bt; A.T = T; A.Ch = Ch; A.N = N; A.G = G;
  return A;
}

template <class F> hipError_t by_flag(bool f, F run) {
  return f ? run(std::true_type()) : run(std::false_type());
}

template <typename T>
hipError_t forward(SScanArgs A, hipStream_t s) {
  segments(A);
  if (A.segs > 1) {
    const hipError_t e = launch("selective_scan_ends", sscan_ends_kernel<T>,
                                dim3(workgroups(A, A.segs - 1)), dim3(threads_of(A)), 0, s, A);
    if (e != hipSuccess) return e;
  }
  return by_flag(A.z, [&](auto gated) {
    return by_flag(A.N > kStates, [&](auto split) {
      return launch("selective_scan", sscan_kernel<T, gated(), split()>,
                    dim3(workgroups(A, A.segs)), dim3(threads_of(A)), 0, s, A);
    });
  });
}

template <typename T>
hipError_t backward(SScanArgs A, hipStream_t s) {
  segments(A);
  hipError_t e;
  if (A.segs > 1) {
    e = by_flag(A.z, [&](auto gated) {
      return launch("selective_scan_bwd_ends", sscan_bwd_ends_kernel<T, gated()>,
                    dim3(workgroups(A, A.segs - 1)), dim3(threads_of(A)), 0, s, A);
    });
    if (e != hipSuccess) return e;
  }
  e = by_flag(A.z, [&](auto gated) {
    return by_flag(A.N > kStates, [&](auto split) {
      return launch("selective_scan_bwd", sscan_bwd_kernel<T, gated(), split()>,
                    dim3(workgroups(A, A.segs)), dim3(threads_of(A)), 0, s, A);
    });
  });
  if (e != hipSuccess) return e;
  const size_t nbc = (size_t)A.Bt * A.T * 2 * A.G * A.N;
  const size_t na = (size_t)A.Ch * (A.N + 2);
  const unsigned first = (unsigned)((nbc + 255) / 256);
  return launch("selective_scan_sum", sscan_sum_kernel<T>,
                dim3(first + (unsigned)((na + 63) / 64)), dim3(256), 0, s, A, first);
}

}  // namespace

size_t sscan_carry_bytes(int Bt, int T, int Ch, int N) {
  return sizeof(float) * (size_t)Bt * ((T + kTok - 1) / kTok) * Ch * state_blocks(N) * kStates;
}

size_t sscan_ws_bytes(int Bt, int T, int Ch, int N, int G) {
  SScanArgs A = sizes(Bt, T, Ch, N, G);
  segments(A);
  if (A.segs <= 1) return 0;
  return sizeof(float) * (size_t)Bt * A.segs * Ch * (state_blocks(N) * kStates + 1);
}

size_t sscan_bwd_ws_bytes(int Bt, int T, int Ch, int N, int G) {
  SScanArgs A = sizes(Bt, T, Ch, N, G);
  segments(A);
  return sizeof(float) * BwdBoard(A).floats(A);
}

int64_t sscan_threads(int64_t Bt, int64_t T, int64_t Ch, int64_t N, int64_t G) {
  const int64_t wg = Bt * G * group_blocks((int)Ch, (int)N, (int)G);
  const int64_t threads = 64 * (int64_t)channel_waves((int)N) * state_blocks((int)N);
  const int64_t scan = (wg + kWant) * threads;
  return std::max({scan, Bt * T * 2 * G * N + 4 * Ch * (N + 2) + 1024, Bt * Ch * 4});
}

hipError_t launch_sscan(bool is_bf16, const SScanArgs& a, hipStream_t s) {
  return is_bf16 ? forward<bf16>(a, s) : forward<float>(a, s);
}

hipError_t launch_sscan_backward(bool is_bf16, const SScanArgs& a, hipStream_t s) {
  return is_bf16 ? backward<bf16>(a, s) : backward<float>(a, s);
}

hipError_t launch_sscan_step(bool is_bf16, const SScanArgs& a, hipStream_t s) {
  auto run = [&](auto t, auto r) {
    const size_t rows = (a.Bt + r() - 1) / r();
    return launch("selective_step", sscan_step_kernel<decltype(t), r()>,
                  dim3((unsigned)((rows * a.Ch * 4 + 255) / 256)), dim3(256), 0, s, a);
  };
  const std::integral_constant<int, 2> two{};
  const std::integral_constant<int, 1> one{};
  if (step_sequences(a.Bt, a.Ch) == 2) return is_bf16 ? run(bf16(), two) : run(0.f, two);
  return is_bf16 ? run(bf16(), one) : run(0.f, one);
}

}  // namespace swimba
