// Gated linear recurrence over channels (swimba_layers.h), forward, backward
// and one token:
//   f = sigmoid(forget), g = 1 - f, h_t = f h_{t-1} + g x_t, y = h silu(gate);
//   e_t = dy silu(gate) + f_{t+1} e_{t+1},  dx = g e,  dforget = f g e (h_{t-1} - x),
//   dgate = dy h silu'(gate).
// A run of tokens maps the state that enters it to P h + S, with P the product
// of its f, and runs are composed: thread (16 tokens of a channel, walked in
// registers), wave (64 channels), workgroup (8 waves, a chunk of 128 tokens),
// sequence. Bound by HBM: each tensor is read once, by one kernel. A chunk's
// workgroup publishes its run, then waits for what precedes it: the runs of the
// earlier chunks of its group of 16, and the state that enters the group, which
// the last workgroup of the group before publishes; so a sequence is a chain of
// one hop per 2048 tokens, and the order of every sum is fixed. A published
// value is one 64-bit word that is stored and loaded whole, all ones until then
// (a fill before the kernel; a NaN is stored in its canonical form), so no
// ordering between words is needed. A workgroup's index gives its sequence and
// channels (its chain); its chunk is the next number of the chain's counter, so
// that it only ever waits for workgroups that took an earlier number of the
// same chain and hence already run: every wait ends. (One counter for all
// workgroups was no slower, but would need all of them in one order.)
//
// The steps keep their relative precision where f is near 1 (a memory of many
// tokens) and near 0 (a reset): with small = min(f, g) = t / (1 + t), t =
// exp(-|forget|), a step is h + g (x - h) while g is the smaller one and
// x - f (x - h) otherwise; the pair is kept as k = small with forget's sign.
// P is kept the same way: 1 - P (as G) next to P, and the one that is not
// close to 1 is used.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "layers.hpp"

namespace swimba {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTpt = 16;            // consecutive tokens per thread
constexpr int kWaves = 8;
constexpr int kTh = 64 * kWaves;
constexpr int kChunk = kTpt * kWaves;  // tokens per workgroup
constexpr int kGroup = 16;          // chunks per group
constexpr uint64_t kUnset = ~0ull;

// One channel of a row that starts `row` bytes into a buffer, at byte offset
// off: with off = kOOB a load reads zeros and a store is dropped.
template <typename T>
__device__ __forceinline__ uint32_t load_bits(BufRes r, uint32_t off, uint32_t row) {
  if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, off, row, 0);
  else return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, row, 0);
}
template <typename T>
__device__ __forceinline__ float value(uint32_t bits) {
  return __uint_as_float(sizeof(T) == 4 ? bits : bits << 16);
}
// NT: stored past the L2's reuse order (nothing here reads it again; the next
// kernel sees the values as those of any store), which took
// 43 -> 39 and 91 -> 77 us off a forward and backward of 8 x 2048 x 1536. Only
// where every row starts on a 128-byte line: partial lines are better gathered in
// L2 (3 x 1777 x 1001 fp32 backward: 43 us against 30).
template <typename T, bool NT>
__device__ __forceinline__ void store_one(BufRes r, uint32_t off, uint32_t row, float v) {
  constexpr int kAux = NT ? 2 : 0;
  if constexpr (sizeof(T) == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, row, kAux);
  else
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, from_f32<T>(v)), r, off, row,
                                          kAux);
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
// P as one number: G, or -P where that is the smaller one (as k for a token)
__device__ __forceinline__ float factor(const Run& r) { return r.G <= 0.5f ? r.G : -r.P; }
__device__ __forceinline__ float apply(const Run& r, float h) { return r.S + decay(factor(r), h); }
// a, then b
__device__ __forceinline__ Run join(const Run& a, const Run& b) {
  return Run{__builtin_fmaf(-a.G, b.G, a.G + b.G), a.P * b.P, apply(b, a.S)};
}
// One more token: S by the caller; G and P are the responses to a constant
// input 1 and to an initial state 1.
__device__ __forceinline__ void extend(Run& r, float k) {
  r.G = __builtin_fmaf(k, 1.f - r.G, neg(k) ? 1.f : r.G);
  r.P = decay(k, r.P);
}

// ---------------------------------------------------------------- chunks

struct Shared {
  float run[3][kWaves][64];    // each wave's run
  float2 prev[kGroup][64];     // the earlier runs of the group: factor, S
  float enter[64];             // the state that enters the group
  uint32_t ticket;
};

// A workgroup's chain (sequence and block of 64 channels) and chunk, and the
// tokens of this thread. The chain is the chunks up to the sequence's length
// (one at least), REV: from the last of them; the chunks past it take the
// numbers after the chain's and only write zeros. All but c and on are uniform
// in a wave, and said to be: buffers are built from them.
struct Place {
  int b, chunk, c, t0, len;  // c: channel; t0: first token within the sequence
  int step, nc, wave;        // position along the scan, chunks of the chain
  size_t cw;                 // row of the chunk among all sequences' chunks
  bool on, dead;             // dead: a chunk past the chain
};
template <bool REV>
__device__ __forceinline__ Place place_of(const GScanArgs& A, unsigned chain, int step) {
  Place p;
  const unsigned ncb = (A.C + 63) / 64;
  p.b = __builtin_amdgcn_readfirstlane(chain / ncb);
  p.len = A.T;
  if (A.lens) p.len = __builtin_amdgcn_readfirstlane(min(max(A.lens[p.b], 0), A.T));
  p.nc = max(1, (p.len + kChunk - 1) / kChunk);
  p.step = step;
  p.dead = step >= p.nc;
  p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  p.chunk = REV && !p.dead ? p.nc - 1 - p.step : p.step;
  p.cw = (size_t)p.b * ((A.T + kChunk - 1) / kChunk) + p.chunk;
  p.c = (chain - p.b * ncb) * 64 + (threadIdx.x & 63);
  p.t0 = p.chunk * kChunk + p.wave * kTpt;
  p.on = p.c < A.C;
  return p;
}

__device__ __forceinline__ uint64_t word(float lo, float hi) {
  return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float canonical(float v) {
  return v != v ? __uint_as_float(0x7FC00000u) : v;
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void post(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits for a word. It comes within microseconds unless another call works in
// the same workspace at the same time, which the interface rules out; rather
// than hang the device, the wait then ends with NaN. It is bounded by its own
// polls (a load past the caches each: some ten seconds in all), not by a clock,
// which would run on while the queue is off the device.
constexpr uint32_t kWaitPolls = 1u << 24;
__device__ __forceinline__ uint64_t wait_for(const uint64_t* p) {
  uint64_t v = peek(p);
  for (uint32_t n = 0; v == kUnset && n < kWaitPolls; ++n) {
    __builtin_amdgcn_s_sleep(1);
    v = peek(p);
  }
  return v;
}

// The workspace: a counter per chain, 128 bytes apart; a word per chunk and
// channel (the chunk's run: S, factor); a word per group and channel (the state
// entering it). All of it starts as all ones.
constexpr size_t kCounterStep = 128;
size_t __host__ __device__ inline counter_bytes(int Bt, int C) {
  return kCounterStep * (size_t)Bt * ((C + 63) / 64);
}
struct Board {
  uint64_t *runs, *enter;
  int nc, ng;  // chunks and groups per sequence
  __device__ explicit Board(const GScanArgs& A) {
    nc = (A.T + kChunk - 1) / kChunk;
    ng = (nc + kGroup - 1) / kGroup;
    runs = reinterpret_cast<uint64_t*>(static_cast<char*>(A.ws) + counter_bytes(A.Bt, A.C));
    enter = runs + (size_t)A.Bt * nc * A.C;
  }
};

// The workgroup's place: its chain from its index, its chunk from the chain's
// counter.
template <bool REV, bool CHAIN>
__device__ __forceinline__ Place take_place(const GScanArgs& A, Shared& sh) {
  if constexpr (CHAIN) {
    const unsigned chains = (unsigned)A.Bt * ((A.C + 63) / 64);
    const unsigned chain = blockIdx.x % chains;
    if (threadIdx.x == 0)
      sh.ticket = atomicAdd(reinterpret_cast<uint32_t*>(static_cast<char*>(A.ws) +
                                                        kCounterStep * chain), 1u) + 1u;
    __syncthreads();
    return place_of<REV>(A, chain, __builtin_amdgcn_readfirstlane(sh.ticket));
  } else {
    return place_of<REV>(A, blockIdx.x, 0);
  }
}

// The state that enters this thread's tokens, the one that enters the chunk,
// and in the wave at the end of the chunk the one that leaves it.
struct States {
  float mine, in, out;
};

// What the waves before this one (in the order of the scan) do to the chunk's
// state. Every thread of the workgroup calls it.
template <bool REV>
__device__ __forceinline__ Run waves_before(const Place& p, Shared& sh, const Run& own) {
  const int lane = threadIdx.x & 63, ord = REV ? kWaves - 1 - p.wave : p.wave;
  sh.run[0][ord][lane] = own.G;
  sh.run[1][ord][lane] = own.P;
  sh.run[2][ord][lane] = own.S;
  __syncthreads();
  Run r = identity();
  for (int w = 0; w < ord; ++w)
    r = join(r, Run{sh.run[0][w][lane], sh.run[1][w][lane], sh.run[2][w][lane]});
  return r;
}

// The state that enters the sequence (start, or null for zeros) where
// enter_states takes it: of a chain, in the last wave of the first group's
// chunks. Loaded before the chunk's tokens, so that waiting for it does not wait
// for them.
template <bool REV, bool CHAIN>
__device__ __forceinline__ float first_state(const GScanArgs& A, const Place& p,
                                             const float* start) {
  const bool last = p.wave == (REV ? 0 : kWaves - 1);
  if (!start || !p.on || (CHAIN && !(last && p.step < kGroup))) return 0.f;
  return start[(size_t)p.b * A.C + p.c];
}

// From each thread's run to its states. CHAIN: sequences have more than one chunk.
template <bool REV, bool CHAIN>
__device__ __forceinline__ States enter_states(const GScanArgs& A, const Place& p, Shared& sh,
                                               const Run& own, float first) {
  const int lane = threadIdx.x & 63, ord = REV ? kWaves - 1 - p.wave : p.wave;
  const bool last = ord == kWaves - 1;
  // The state that leaves the sequence may be written over the one that enters
  // it: by a wave of this workgroup after the barrier below, or by a workgroup
  // that waited for the run that this one posts. The (empty) use makes the load
  // of `first` complete before both.
  asm volatile("" : "+v"(first) : : "memory");
  const Run before = waves_before<REV>(p, sh, own);
  const Run total = join(before, own);  // of the chunk, in the last wave
  States st;
  st.in = first;
  if constexpr (CHAIN) {
    const Board bd(A);
    const int g = p.step / kGroup, i = p.step % kGroup;
    const uint64_t* runs = bd.runs + ((size_t)p.b * bd.nc + g * kGroup) * A.C + p.c;
    uint64_t* enter = bd.enter + ((size_t)p.b * bd.ng + g) * A.C + p.c;
    if (p.on) {
      if (last && i + 1 < kGroup && p.step + 1 < p.nc)
        post(const_cast<uint64_t*>(runs) + (size_t)i * A.C,
             word(canonical(total.S), canonical(factor(total))));
      // wave w collects the runs of chunks w and w + 8 of the group, the last
      // wave also the entering state
      for (int q = ord; q < i; q += kWaves) {
        const uint64_t v = wait_for(runs + (size_t)q * A.C);
        sh.prev[q][lane] = make_float2(__uint_as_float((uint32_t)(v >> 32)),
                                       __uint_as_float((uint32_t)v));
      }
      if (last) sh.enter[lane] = g == 0 ? first : __uint_as_float((uint32_t)wait_for(enter));
    }
    __syncthreads();
    if (p.on) {
      st.in = sh.enter[lane];
      for (int q = 0; q < i; ++q) {
        const float2 r = sh.prev[q][lane];
        st.in = r.y + decay(r.x, st.in);
      }
      if (last && i + 1 == kGroup && p.step + 1 < p.nc)
        post(enter + A.C, word(apply(total, st.in), 0.f));
    }
  }
  st.mine = apply(before, st.in);
  st.out = apply(total, st.in);
  return st;
}

// The chunk's rows of a tensor as a buffer.
template <typename T>
__device__ __forceinline__ BufRes chunk_buffer(const void* t, size_t row, int64_t ld, int rows,
                                               int C) {
  return make_rsrc(static_cast<const T*>(t) + row * ld,
                   rows > 0 ? ((uint64_t)(rows - 1) * ld + C) * sizeof(T) : 0);
}

// ---------------------------------------------------------------- forward

// FULL: all of the chunk's tokens are in use (no selects on the token).
template <typename T, bool CHAIN, bool GATED, bool NT, bool FULL>
__device__ __forceinline__ void gscan_chunk(const GScanArgs& A, const Place& p, Shared& sh) {
  constexpr uint32_t ES = sizeof(T);
  const int t1 = p.chunk * kChunk;
  const int rows = FULL ? kChunk : min(kChunk, A.T - t1);  // the chunk's rows
  const size_t row = (size_t)p.b * A.T + t1;
  const int w0 = p.t0 - t1;                          // this thread's first row
  const int live = FULL ? kTpt : min(max(p.len - p.t0, 0), kTpt);  // its tokens in use
  const BufRes rx = chunk_buffer<T>(A.x, row, A.ld, rows, A.C);
  const BufRes rf = chunk_buffer<T>(A.f, row, A.ld, rows, A.C);
  const BufRes ro = chunk_buffer<T>(GATED ? A.o : A.x, row, A.ld, rows, A.C);
  const BufRes ry = chunk_buffer<T>(A.y, row, A.C, rows, A.C);
  const uint32_t pitch = (uint32_t)A.ld * ES, ypitch = A.C * ES;
  const uint32_t col = p.on ? p.c * ES : kOOB;
  if (!FULL && p.dead) {
#pragma unroll
    for (int i = 0; i < kTpt; ++i)
      store_one<T, NT>(ry, w0 + i < rows ? col : kOOB, (w0 + i) * ypitch, 0.f);
    return;
  }
  const float first = first_state<false, CHAIN>(A, p, A.h_init);
  uint32_t xr[kTpt], fr[kTpt], gr[kTpt];
#pragma unroll
  for (int i = 0; i < kTpt; ++i) {
    const uint32_t off = i < live ? col : kOOB, r = (w0 + i) * pitch;
    fr[i] = load_bits<T>(rf, off, r);
    xr[i] = load_bits<T>(rx, off, r);
    if constexpr (GATED) gr[i] = load_bits<T>(ro, off, r);
  }
  float k[kTpt];
  Run own = identity();
#pragma unroll
  for (int i = 0; i < kTpt; ++i) {
    // past the length: f = 1 (the logit and x read as 0)
    k[i] = gate_of(value<T>(fr[i]));
    if constexpr (!FULL) k[i] *= i < live ? 1.f : 0.f;
    extend(own, k[i]);
    own.S = step(k[i], value<T>(xr[i]), own.S);
  }
  const States st = enter_states<false, CHAIN>(A, p, sh, own, first);
  if (p.on && A.carry && p.wave == 0) A.carry[p.cw * A.C + p.c] = st.in;
  if (p.on && A.h_final && p.step == p.nc - 1 && p.wave == kWaves - 1)
    A.h_final[(size_t)p.b * A.C + p.c] = st.out;
  float h = st.mine;
#pragma unroll
  for (int i = 0; i < kTpt; ++i) {
    h = step(k[i], value<T>(xr[i]), h);
    float v = h;
    if constexpr (GATED) {
      const float ov = value<T>(gr[i]);
      v *= ov * sigm(ov);
    }
    store_one<T, NT>(ry, w0 + i < rows ? col : kOOB, (w0 + i) * ypitch, i < live ? v : 0.f);
  }
}

template <typename T, bool CHAIN, bool GATED, bool NT>
__global__ __launch_bounds__(kTh) void gscan_kernel(GScanArgs A) {
  __shared__ Shared sh;
  const Place p = take_place<false, CHAIN>(A, sh);
  if ((p.chunk + 1) * (int64_t)kChunk <= p.len) gscan_chunk<T, CHAIN, GATED, NT, true>(A, p, sh);
  else gscan_chunk<T, CHAIN, GATED, NT, false>(A, p, sh);
}

// ---------------------------------------------------------------- backward

// Walking back, c = f_t e_t is the gradient that leaves token t for the state
// before it: c <- f (u + c), u = dy silu(gate). The states come from the
// forward's carry and the runs of the chunk's waves.
// (A second copy of the code for chunks in full use, as in the forward, made it
// slower: 84 against 71 us for a padded batch of 8 x 2048 x 1536.)
template <typename T, bool CHAIN, bool GATED, bool NT>
__global__ __launch_bounds__(kTh, 4) void gscan_bwd_kernel(GScanArgs A) {
  constexpr uint32_t ES = sizeof(T);
  __shared__ Shared sh;
  const Place p = take_place<true, CHAIN>(A, sh);
  const int t1 = p.chunk * kChunk, rows = min(kChunk, A.T - t1);
  const size_t row = (size_t)p.b * A.T + t1;
  const int w0 = p.t0 - t1;
  const int live = min(max(p.len - p.t0, 0), kTpt);
  const BufRes rx = chunk_buffer<T>(A.x, row, A.ld, rows, A.C);
  const BufRes rf = chunk_buffer<T>(A.f, row, A.ld, rows, A.C);
  const BufRes ro = chunk_buffer<T>(GATED ? A.o : A.x, row, A.ld, rows, A.C);
  const BufRes rd = chunk_buffer<T>(A.dy, row, A.C, rows, A.C);
  const BufRes sx = chunk_buffer<T>(A.dx, row, A.ldd, rows, A.C);
  const BufRes sf = chunk_buffer<T>(A.df, row, A.ldd, rows, A.C);
  const BufRes so = chunk_buffer<T>(GATED ? A.d_o : A.dx, row, A.ldd, rows, A.C);
  const uint32_t pitch = (uint32_t)A.ld * ES, dpitch = (uint32_t)A.ldd * ES;
  const uint32_t col = p.on ? p.c * ES : kOOB;
  if (p.dead) {
#pragma unroll
    for (int i = 0; i < kTpt; ++i) {
      const uint32_t off = w0 + i < rows ? col : kOOB, r = (w0 + i) * dpitch;
      store_one<T, NT>(sx, off, r, 0.f);
      store_one<T, NT>(sf, off, r, 0.f);
      if constexpr (GATED) store_one<T, NT>(so, off, r, 0.f);
    }
    return;
  }
  const float first = first_state<true, CHAIN>(A, p, A.dh_final);
  uint32_t xr[kTpt], fr[kTpt], gr[kTpt], dr[kTpt];
#pragma unroll
  for (int i = 0; i < kTpt; ++i) {
    const uint32_t off = i < live ? col : kOOB, r = (w0 + i) * pitch;
    fr[i] = load_bits<T>(rf, off, r);
    dr[i] = load_bits<T>(rd, off, (w0 + i) * A.C * ES);
    if constexpr (GATED) gr[i] = load_bits<T>(ro, off, r);
    xr[i] = load_bits<T>(rx, off, r);
  }
  float k[kTpt], e[kTpt];
  Run fw = identity();
#pragma unroll
  for (int i = 0; i < kTpt; ++i) {
    k[i] = gate_of(value<T>(fr[i]));
    k[i] *= i < live ? 1.f : 0.f;  // past the length: f = 1
    e[i] = value<T>(dr[i]);
    if constexpr (GATED) {
      const float ov = value<T>(gr[i]);
      e[i] *= ov * sigm(ov);
    }
    extend(fw, k[i]);
    fw.S = step(k[i], value<T>(xr[i]), fw.S);
  }
  Run bw = fw;
  bw.S = 0.f;
#pragma unroll
  for (int i = kTpt - 1; i >= 0; --i) bw.S = decay(k[i], e[i] + bw.S);
  const Run fbefore = waves_before<false>(p, sh, fw);
  float h = p.on ? apply(fbefore, A.carry_in[p.cw * A.C + p.c]) : 0.f;
  __syncthreads();  // the runs in LDS are no longer read
  const States st = enter_states<true, CHAIN>(A, p, sh, bw, first);
  if (p.on && A.dh_init && p.step == p.nc - 1 && p.wave == 0)
    A.dh_init[(size_t)p.b * A.C + p.c] = st.out;
  // e_t from the last token back
  float c = st.mine;
#pragma unroll
  for (int i = kTpt - 1; i >= 0; --i) {
    e[i] += c;
    c = decay(k[i], e[i]);
  }
#pragma unroll
  for (int i = 0; i < kTpt; ++i) {
    const float kk = k[i], a = fabsf(kk), xv = value<T>(xr[i]);
    const uint32_t off = w0 + i < rows ? col : kOOB, r = (w0 + i) * dpitch;
    const bool in = i < live;
    store_one<T, NT>(sx, off, r, in ? inject(kk, e[i]) : 0.f);
    store_one<T, NT>(sf, off, r, in ? __builtin_fmaf(-a, a, a) * e[i] * (h - xv) : 0.f);
    h = step(kk, xv, h);
    if constexpr (GATED) {
      const float ov = value<T>(gr[i]), sg = sigm(ov);
      const float vo = value<T>(dr[i]) * h * (sg * __builtin_fmaf(ov, 1.f - sg, 1.f));
      store_one<T, NT>(so, off, r, in ? vo : 0.f);
    }
  }
}

// The workspace before a chained kernel: nothing published.
__global__ __launch_bounds__(256) void gscan_unset_kernel(uint4* ws, size_t n) {
  for (size_t q = (size_t)blockIdx.x * 256 + threadIdx.x; q < n; q += (size_t)gridDim.x * 256)
    ws[q] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// ---------------------------------------------------------------- one token

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

// One channel per lane for both types: pairs of bf16 channels (4-byte accesses)
// needed 121 and 234 registers against 84 and 129 and were 3 % and 15 % slower
// (65536 x 2048 forward, padded 8 x 2048 x 1536 training step).
// BWD: the backward's kernel.
template <typename T, bool BWD>
hipError_t go(const GScanArgs& A, hipStream_t s) {
  const bool chain = gscan_chunks(A.T) > 1;
  if (chain) {
    const size_t n = gscan_ws_bytes(A.Bt, A.T, A.C) / 16;
    const unsigned blocks = (unsigned)std::min<size_t>((n + 255) / 256, 2048);
    const hipError_t e = launch("gated_scan_unset", gscan_unset_kernel, dim3(blocks), dim3(256), 0,
                                s, (uint4*)A.ws, n);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)gscan_blocks(A.Bt, A.T, A.C));
  // output rows that start on 128-byte lines
  auto lines = [](const void* t, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(t) | (uintptr_t)(ld * sizeof(T))) % 128 == 0;
  };
  const bool nt = BWD ? lines(A.dx, A.ldd) && lines(A.df, A.ldd) && (!A.o || lines(A.d_o, A.ldd))
                      : lines(A.y, A.C);
  auto run = [&](auto chained, auto gated, auto through) {
    constexpr bool CH = decltype(chained)::value, GA = decltype(gated)::value,
                   NT = decltype(through)::value;
    if constexpr (BWD)
      return launch("gated_scan_bwd", gscan_bwd_kernel<T, CH, GA, NT>, grid, dim3(kTh), 0, s, A);
    else
      return launch("gated_scan", gscan_kernel<T, CH, GA, NT>, grid, dim3(kTh), 0, s, A);
  };
  const std::true_type yes{};
  const std::false_type no{};
  auto run_nt = [&](auto chained, auto gated) {
    return nt ? run(chained, gated, yes) : run(chained, gated, no);
  };
  if (chain) return A.o ? run_nt(yes, yes) : run_nt(yes, no);
  return A.o ? run_nt(no, yes) : run_nt(no, no);
}

}  // namespace

int gscan_chunks(int T) { return (T + kChunk - 1) / kChunk; }

int64_t gscan_blocks(int64_t Bt, int64_t T, int64_t C) {
  return Bt * ((T + kChunk - 1) / kChunk) * ((C + 63) / 64);
}

size_t gscan_ws_bytes(int Bt, int T, int C) {
  const size_t nc = gscan_chunks(T), ng = (nc + kGroup - 1) / kGroup;
  if (nc <= 1) return 0;
  return (counter_bytes(Bt, C) + sizeof(uint64_t) * (size_t)Bt * (nc + ng) * C + 15) / 16 * 16;
}

hipError_t launch_gscan(bool is_bf16, const GScanArgs& a, hipStream_t s) {
  return is_bf16 ? go<bf16, false>(a, s) : go<float, false>(a, s);
}

hipError_t launch_gscan_backward(bool is_bf16, const GScanArgs& a, hipStream_t s) {
  return is_bf16 ? go<bf16, true>(a, s) : go<float, true>(a, s);
}

hipError_t launch_gscan_step(bool is_bf16, const void* x, const void* f, const void* o, int64_t ld,
                             const float* h_prev, float* h, void* y, int Bt, int C,
                             hipStream_t s) {
  auto go = [&](auto tag, auto vec) {
    typedef decltype(tag) T;
    constexpr int VEC = decltype(vec)::value;
    const dim3 grid((unsigned)(((size_t)Bt * (C / VEC) + 255) / 256));
    return launch("gated_step", gscan_step_kernel<T, VEC>, grid, dim3(256), 0, s, (const T*)x,
                  (const T*)f, (const T*)o, ld, h_prev, h, (T*)y, Bt, C);
  };
  const std::integral_constant<int, 4> four{};
  const std::integral_constant<int, 1> one{};
  const bool by4 = C % 4 == 0 && ld % 4 == 0;
  if (is_bf16) return by4 ? go(bf16(), four) : go(bf16(), one);
  return by4 ? go(0.f, four) : go(0.f, one);
}

}  // namespace swimba
