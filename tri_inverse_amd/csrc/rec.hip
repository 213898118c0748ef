// rec.hip -- the gated linear recurrence of every channel: whole sequences forwards and backwards,
// and single tokens.
//
// Per sequence and channel, s = sigmoid, tokens in order:
//   log a_t = -w s(A_t) | log s(A_t) | A_t          u_t = b_t s(I_t) X_t,  b = sqrt(1 - a^2) | 1 - a | 1
//   h_t = a_t h_{t-1} + u_t
// Backwards, with D_t the whole gradient of h_t and e_t = a_t D_t that of h_{t-1}:
//   D_t = dH_t + e_{t+1}   (e past the end: the gradient of the last state)
//   dX = D b s(I),  dI = D b X s(I) (1 - s(I)),  dg = e_t h_{t-1} + D s(I) X b'(g),
//   dA = -w s'(A) dg | (1 - s(A)) dg | dg,  dw = -sum s(A) dg,  dh_0 = e_1
//
// h is affine in its start: over a run of tokens h = P h_start + h_run, P the product of the run's
// decays.  A workgroup takes a tile of 8 runs and 128 channels, two to a lane, so that a row of a
// wave is 256 contiguous bytes (bf16), each wave a run of tokens in registers.  The ends of the runs
// join in LDS.  The tiles of a row and 128 channels form a chain, and the data is read once: a
// workgroup publishes its tile's end (P, h), waits for those before it, and forms its outputs from the
// registers it still holds.  Ends join by eights: a tile reads the ends of the tiles before it in its
// eight, of the eights before its own in their eight, and the state before those 64 tiles.  So a chain
// has one step in a row for 64 tiles, and the order of the sums does not depend on the workgroups'
// progress: the same call gives the same bits.
//
// Waiting: a word of a chain carries its value and, by not being NOT_YET, that it is there, in one
// 64-bit store, so no fence is needed.  A workgroup takes its tile from its chain's counter,
// in the order of the workgroups' starts: whatever it waits for has been taken by a workgroup that is
// already running, which itself waits only for earlier ones, so every wait ends.  A wait is bounded
// all the same: past the bound it takes NaN for the state.
//
// Decays, states and sums are fp32; 1 - a is formed without cancelling (a series near 0), each output is
// rounded once.
//
// Measured (a copy of 1 GiB reaches 5.05 TB/s): 4 sequences of 8192 tokens, 2048 channels, bf16, 537 MB, 130
// us, 4.1 TB/s.  With the stores through the caches it took 138, of which the chain 4, the gates' arithmetic 13,
// both together 23.  One sequence of 65536 tokens, 1024 channels, 403 MB, 120 us, without the chain 91: of 8
// chains alone a tile waits for the slowest of 64 that run beside it.  Training step of 4 x 4096 tokens,
// 2048 channels, 738 MB, 208 us: the kernels 69 forwards and 139 backwards in a profile (100 without chain and gates).
// Tiles: 64 tokens forwards take 150 us for the first, 32 tokens 211 (each tile has its share of the
// chain); 128 backwards spill, 260 us for the training step.  Workgroups that walk on along their chain
// took 140 and, for the second, 142; three workgroups a CU, with half of u in LDS, 139 and 136.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

constexpr int RUNS = 8;       // waves of a workgroup, a run of tokens each
constexpr int CH = 2 * WAVE;  // channels of a workgroup
constexpr int FWD_TILE = 128, BWD_TILE = 64;  // tokens of a tile: as many as leave room for two workgroups a CU
static_assert(GDN_REC_TILE % (FWD_TILE / RUNS) == 0 && BWD_TILE % GDN_REC_TILE == 0, "states at the starts of runs and tiles");

typedef float f32x2 __attribute__((ext_vector_type(2)));

// a value of which the compiler knows nothing from here on
template <class V>
__device__ __forceinline__ void hide(V& v) {
  asm volatile("" : "+v"(v));
}

// outputs go past what the caches hold (the non-temporal bit): prefill 137.7 -> 132 us, training step 218 -> 211; also where
// rows end inside lines: training steps of 4 x 4096 tokens of 520 and 776 channels 90 -> 84 and 117 -> 111, forwards alone
// 2 % less to 2 % more
constexpr int PAST = 2;

// two neighbouring channels as they lie in memory, and as fp32
template <class E>
struct Pair;
template <>
struct Pair<__bf16> {
  typedef uint32_t raw;
  static __device__ __forceinline__ raw load(__amdgpu_buffer_rsrc_t p, uint32_t lane, uint32_t row) {
    return __builtin_amdgcn_raw_buffer_load_b32(p, lane, row, 0);
  }
  static __device__ __forceinline__ void store(raw v, __amdgpu_buffer_rsrc_t p, uint32_t lane, uint32_t row) {
    __builtin_amdgcn_raw_buffer_store_b32(v, p, lane, row, PAST);
  }
  static __device__ __forceinline__ f32x2 open(raw v) {
    return f32x2{__builtin_bit_cast(float, v << 16), __builtin_bit_cast(float, v & 0xffff0000u)};
  }
  static __device__ __forceinline__ raw close(f32x2 v) {
    typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
    bf16x2 r;
    r[0] = (__bf16)v[0];
    r[1] = (__bf16)v[1];
    return __builtin_bit_cast(uint32_t, r);
  }
};
template <>
struct Pair<float> {
  typedef f32x2 raw;
  static __device__ __forceinline__ raw load(__amdgpu_buffer_rsrc_t p, uint32_t lane, uint32_t row) {
    return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(p, lane, row, 0));
  }
  static __device__ __forceinline__ void store(raw v, __amdgpu_buffer_rsrc_t p, uint32_t lane, uint32_t row) {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), p, lane, row, PAST);
  }
  static __device__ __forceinline__ f32x2 open(raw v) { return v; }
  static __device__ __forceinline__ raw close(f32x2 v) { return v; }
};

__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// exponentials are of 2, which the hardware forms: log-decays are held in units of log 2
constexpr float LOG2E = 1.44269504f, LN2 = 0.693147181f;
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
// e^-z of a gate z in E.  The rounding of -z log2 e, below 2^-23 |z| of e^-z, counts in fp32 from |z| = 8 on: there a factor
// 1 + x makes it good, to 2^-22 at any z.  The lower bound keeps the factor where the remainder of an infinite z is NaN; a
// NaN z is NaN in e.  Of a bf16 z its own rounding, 2^-9 |z|, leaves more (and the correction takes 3 % of the time: prefill
// 133 -> 137 us, training step 213 -> 218; in fp32 a packed call of 11171 tokens of 1544 channels 76 -> 77).
template <class E>
__device__ __forceinline__ float exp_minus(float z) {
  constexpr float LOW = 1.92596299e-8f;  // of log2 e behind LOG2E
  const float x = -LOG2E * z, e = exp2_of(x);
  if constexpr (sizeof(E) == 2) return e;
  return e * fmaxf(fmaf(LN2, fmaf(-LOW, z, fmaf(-LOG2E, z, -x)), 1.f), 0.5f);
}
template <class E>
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + exp_minus<E>(z)); }
// sigmoid and what it leaves of 1, which a difference would cancel; 2^-126 and not 0 for far z < 0, NaN of NaN
template <class E>
__device__ __forceinline__ void sigmoid_rest(float z, float& s, float& rest) {
  const float e = __builtin_elementwise_minimum(exp_minus<E>(z), 0x1p126f);
  s = rcp(1.f + e);
  rest = e * s;
}

// 1 - 2^(n gl), n = 1 or 2, given as `direct` from a: below 1/4 in n g the series (its first term left out is
// below 2^-24 of it), above it the difference, right to 2^-21
template <int N>
__device__ __forceinline__ float rest_of(float gl, float direct) {
  constexpr float x = N * LN2, x2 = x * x, x3 = x2 * x;
  float r = -x3 * x3 / 720.f;
  r = fmaf(r, gl, -x3 * x2 / 120.f);
  r = fmaf(r, gl, -x2 * x2 / 24.f);
  r = fmaf(r, gl, -x3 / 6.f);
  r = fmaf(r, gl, -x2 / 2.f);
  r = fmaf(r, gl, -x);
  return fabsf(gl) < 0.25f * LOG2E / N ? r * gl : direct;
}

// the decay of a token and the factor b of its input.  wl = -w log2 e.
template <class E, int DECAY, int NORM>
struct Gate {
  float a, b;
  __device__ __forceinline__ Gate(float A, float wl) {
    float q = 1.f;  // 1 - a, or 1 - a^2
    if constexpr (DECAY == GDN_DECAY_SIGMOID) {
      const float e = exp_minus<E>(A);
      a = rcp(1.f + e);
      const float rest = A < 0.f ? 1.f - a : e * a;  // e may be infinite
      q = NORM == GDN_REC_NORM_SQRT ? rest * (1.f + a) : rest;
    } else {
      const float gl = DECAY == GDN_DECAY_POWER ? wl * sigmoid<E>(A) : LOG2E * A;
      a = exp2_of(gl);
      if constexpr (NORM == GDN_REC_NORM_SQRT) q = rest_of<2>(gl, fmaf(-a, a, 1.f));
      if constexpr (NORM == GDN_REC_NORM_LINEAR) q = rest_of<1>(gl, 1.f - a);
    }
    b = NORM == GDN_REC_NORM_SQRT ? __builtin_amdgcn_sqrtf(q) : NORM == GDN_REC_NORM_LINEAR ? q : 1.f;
  }
};
// b'(g) of a and b
template <int NORM>
__device__ __forceinline__ float slope(float a, float b) {
  if constexpr (NORM == GDN_REC_NORM_NONE) return 0.f;
  if constexpr (NORM == GDN_REC_NORM_LINEAR) return -a;
  return b == 0.f ? 0.f : -a * a * rcp(b);  // where a = 1 the gradient of b = 0 counts as 0
}
// what turns dg into dA (first) and into dw (r)
template <class E, int DECAY>
struct GateGrad {
  float to_A = 1.f, r = 0.f;
  __device__ __forceinline__ GateGrad(float A, float wl) {
    float rest;
    if constexpr (DECAY == GDN_DECAY_SIGMOID) sigmoid_rest<E>(A, r, to_A);
    if constexpr (DECAY == GDN_DECAY_POWER) {
      sigmoid_rest<E>(A, r, rest);
      to_A = LN2 * (wl * r) * rest;
    }
  }
};

// ---- sequences in a run of tokens ---------------------------------------------------------

// bit j of the masks: token t0 + j belongs to a sequence, is its first, its last one.  In lane j: the
// sequence of token t0 + j, its first token and the one behind its last.  Offsets are clamped to the
// tokens, sequences to the given ones, so offsets that break their rule lead to no access outside.
template <int RUN>
struct Run {
  uint32_t in, first, last;
  int seq, from, to;
  // all tokens in one sequence that neither starts nor ends here
  __device__ __forceinline__ bool plain() const { return in == (uint32_t)((1ull << RUN) - 1) && (first | last) == 0; }
  __device__ __forceinline__ int seq_of(int j) const { return __builtin_amdgcn_readlane(seq, j); }
};

__device__ __forceinline__ int offset_at(const RecLaunch& a, int i) {
  const int o = a.offsets[i];
  return o < 0 ? 0 : o > (int)a.T ? (int)a.T : o;
}

template <int RUN>
__device__ __forceinline__ Run<RUN> find_run(const RecLaunch& a, int64_t t0, int b) {
  Run<RUN> r;
  if (!a.offsets) {
    const int64_t left = a.T - t0;
    const int n = left < 0 ? 0 : left > RUN ? RUN : (int)left;
    r.in = (uint32_t)((1ull << n) - 1);
    r.first = t0 == 0 && n > 0 ? 1u : 0u;
    r.last = left >= 1 && left <= RUN ? 1u << (n - 1) : 0u;
    r.seq = b;
    r.from = 0;
    r.to = (int)a.T;
    return r;
  }
  const int64_t t = t0 + lane_id();
  int lo = -1, hi = a.n_seq;  // lo: the last sequence that starts at t or before
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (offset_at(a, mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  const bool some = lo >= 0;
  r.seq = some ? lo : 0;
  r.from = some ? offset_at(a, lo) : 0;
  r.to = some ? offset_at(a, lo + 1) : 0;
  const bool in = some && t < r.to && t < a.T && lane_id() < RUN;
  r.in = (uint32_t)__builtin_amdgcn_ballot_w64(in);
  r.first = (uint32_t)__builtin_amdgcn_ballot_w64(in && t == r.from);
  r.last = (uint32_t)__builtin_amdgcn_ballot_w64(in && t + 1 == r.to);
  return r;
}

// ---- a workgroup's place, its rows -----------------------------------------------------------

// the workgroup's chain (a row b and 128 channels) and its tile, in the chain's order: forwards the tiles in
// order, backwards from the last one on
struct Where {
  int wave, b, c;  // c: the lane's first channel; D or more: none
  int order;
  int tile, t0;    // the tile in its row; the run's first token
};

template <int RUN, bool BWD>
__device__ __forceinline__ Where find_place(const RecLaunch& a) {
  __shared__ uint32_t ticket;
  Where at;
  at.wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const uint32_t blocks = (uint32_t)((a.D + CH - 1) / CH), chains = gridDim.x / (uint32_t)a.tiles;
  const uint32_t chain = blockIdx.x % chains;
  at.order = 0;
  if (a.tiles > 1) {
    if (threadIdx.x == 0) ticket = __hip_atomic_fetch_add(a.tickets + chain, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    at.order = __builtin_amdgcn_readfirstlane((int)(ticket + 1u));  // the counter starts at NOT_YET
  }
  at.b = (int)(chain / blocks);
  at.c = (int)(chain - (uint32_t)at.b * blocks) * CH + 2 * lane_id();
  at.tile = BWD ? (int)a.tiles - 1 - at.order : at.order;
  at.t0 = at.tile * RUN * RUNS + at.wave * RUN;
  return at;
}

// the rows of a run of a tensor, addressed by a uniform offset of its row and a lane's offset in it, 32 bits
// each (a run's rows span less than 2^31 bytes: strides are below REC_MAX_STRIDE)
template <class E>
struct Rows {
  __amdgpu_buffer_rsrc_t p;
  uint32_t step;
  __device__ __forceinline__ Rows(const RecLaunch& a, const Where& at, const void* t, int64_t stride) {
    const int64_t row = (int64_t)at.b * a.T + (at.t0 < (int)a.T ? at.t0 : (int)a.T - 1);
    step = (uint32_t)stride * (uint32_t)sizeof(E);
    p = __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(reinterpret_cast<const E*>(t) + row * stride), 0, -1, 0x27000);
  }
  // row j; past the last token the last row, past the last channel the first ones
  __device__ __forceinline__ typename Pair<E>::raw load(const RecLaunch& a, const Where& at, int j) const {
    const int left = (int)a.T - 1 - at.t0, last = left > 0 ? left : 0;
    return Pair<E>::load(p, (at.c < a.D ? (uint32_t)at.c : 0u) * (uint32_t)sizeof(E), (uint32_t)(j < last ? j : last) * step);
  }
  // row j, of a token that exists
  __device__ __forceinline__ void store(const RecLaunch& a, const Where& at, int j, f32x2 v) const {
    if (at.c < a.D) Pair<E>::store(Pair<E>::close(v), p, (uint32_t)at.c * (uint32_t)sizeof(E), (uint32_t)j * step);
  }
};

__device__ __forceinline__ f32x2 state_in(const RecLaunch& a, const float* S, int64_t row, int c) {
  f32x2 h{0.f, 0.f};
  if (S && c < a.D) h = *reinterpret_cast<const f32x2*>(S + row * a.D + c);
  return h;
}
__device__ __forceinline__ void state_out(const RecLaunch& a, float* S, int64_t row, int c, f32x2 h) {
  if (S && c < a.D) *reinterpret_cast<f32x2*>(S + row * a.D + c) = h;
}

__device__ __forceinline__ f32x2 fma2(f32x2 x, f32x2 y, f32x2 z) {
  return f32x2{fmaf(x[0], y[0], z[0]), fmaf(x[1], y[1], z[1])};
}
__device__ __forceinline__ f32x2 mul2(f32x2 x, f32x2 y) { return f32x2{x[0] * y[0], x[1] * y[1]}; }

// -w log2 e
__device__ __forceinline__ f32x2 channel_w(const RecLaunch& a, int c) {
  f32x2 w{0.f, 0.f};
  if (a.w && c < a.D) w = *reinterpret_cast<const f32x2*>(a.w + c);
  return f32x2{-LOG2E * w[0], -LOG2E * w[1]};
}

// Sequences without tokens return their states as they were given.  They are dealt out over the waves of all tiles, each
// lane of a wave looks at one; the states of the empty ones go four at a time, so that their loads do not wait for each
// other's stores.  Forwards and backwards: 1024 sequences of none to two tokens, 2048 channels, 66 us, 200000 of which 64
// have a token, 136 channels, 13 ms (by one wave, one after the other, 94 us and 159 ms).
__device__ __forceinline__ void empty_sequences(const RecLaunch& a, const Where& at, const float* from, float* to) {
  if (!a.offsets || !to) return;
  const int64_t waves = a.tiles * RUNS;
  for (int64_t s0 = (int64_t)at.tile * RUNS + at.wave; s0 < a.n_seq; s0 += waves * WAVE) {
    const int64_t s = s0 + lane_id() * waves;
    uint64_t empty = __builtin_amdgcn_ballot_w64(s < a.n_seq && offset_at(a, (int)s) >= offset_at(a, (int)s + 1));
    while (empty) {
      constexpr int N = 4;
      int64_t row[N];
      f32x2 h[N];
      int n = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (!empty) break;
        row[k] = s0 + __builtin_ctzll(empty) * waves;
        h[k] = state_in(a, from, row[k], at.c);
        empty &= empty - 1;
        ++n;
      }
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < n) state_out(a, to, row[k], at.c, h[k]);
    }
  }
}

// ---- chains -------------------------------------------------------------------------------

constexpr uint32_t NOT_YET = ~0u;  // what the workspace is filled with; the bits of one NaN, never published
constexpr int EIGHT = 8;
constexpr int WAIT_ROUNDS = 1 << 22;  // some seconds

// (P, h) of two channels
__device__ __forceinline__ uint32_t there(float h) {
  const uint32_t u = __builtin_bit_cast(uint32_t, h);
  return u == NOT_YET ? 0x7fc00000u : u;
}
__device__ __forceinline__ void publish(uint64_t* p, f32x2 P, f32x2 h) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float Pk = P[k], hk = h[k];
    __hip_atomic_store(p + k, (uint64_t)there(hk) << 32 | __builtin_bit_cast(uint32_t, Pk), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
  }
}
// a lane's words of one entry, looked at until they are there.  Every lane of the wave calls look and wait;
// lanes that are off (p NULL) wait for nothing.
struct Words {
  const uint64_t* p = nullptr;
  uint64_t v[2] = {0, 0};
  __device__ __forceinline__ void look(const uint64_t* at) {
    p = at;
    look();
  }
  __device__ __forceinline__ void look() {
    if (p)
#pragma unroll
      for (int k = 0; k < 2; ++k) v[k] = __hip_atomic_load(p + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ bool ready() const {
    return (uint32_t)(v[0] >> 32) != NOT_YET && (uint32_t)(v[1] >> 32) != NOT_YET;
  }
  // while the words are not there one lane looks at its own: 64 lanes of all waiting waves would take as
  // much of the memory's rate as the rows do
  __device__ __forceinline__ void wait(f32x2& P, f32x2& h) {
    for (int i = 0; i < WAIT_ROUNDS && !wave_all(ready()); ++i) {
      __builtin_amdgcn_s_sleep(2);
      if (lane_id() == 0) look();
      if (wave_all(lane_id() != 0 || ready())) look();
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t lo = (uint32_t)v[k], hi = (uint32_t)(v[k] >> 32);
      P[k] = __builtin_bit_cast(float, lo);
      h[k] = __builtin_bit_cast(float, hi);  // past the bound NOT_YET, a NaN
    }
  }
};

// ends of runs, of tiles and of eights, two channels a lane
template <int N>
struct Ends {
  f32x2 P[N][WAVE], h[N][WAVE];
  __device__ __forceinline__ void put(int i, f32x2 p, f32x2 x) {
    P[i][lane_id()] = p;
    h[i][lane_id()] = x;
  }
  // h behind entry i that starts from x; fresh: a sequence starts in it, so nothing comes from before
  __device__ __forceinline__ f32x2 behind(int i, f32x2 x, bool fresh) const {
    const f32x2 y = h[i][lane_id()];
    return fresh ? y : fma2(P[i][lane_id()], x, y);
  }
};

// the runs of a tile in the chain's order, and what comes from before the tile
struct Link {
  Ends<RUNS> run;
  int fresh[RUNS];  // a sequence starts (backwards: ends) in the run
  int from;         // the first tile in the chain's order that the tile's start comes from; its own: none
  Ends<EIGHT - 1> tiles, eights;
  f32x2 before[WAVE];

  // the state before run n of the tile that starts from x
  __device__ __forceinline__ f32x2 before_run(int n, f32x2 x) const {
    for (int k = 0; k < n; ++k) x = run.behind(k, x, fresh[k] != 0);
    return x;
  }
};

// A tile's place in its chain.  All waves make one, behind the barrier that follows the runs' ends (wave: the
// wave's run in the chain's order): the tile's end is published, and the words that the tile's start
// comes from are asked for, all at once.  start() waits for them; what stands between hides their way.
struct Joint {
  const RecLaunch& a;
  Link& l;
  int wave, q, from, tiles, tile0, tile1, eight0, eight1;
  bool on, fresh;
  int c;
  int64_t row, row8, row64;  // the row's words: tile by tile, eight by eight, 64 by 64
  f32x2 P{1.f, 1.f}, h{0.f, 0.f};
  Words near, far;

  __device__ __forceinline__ uint64_t* tile_words(int k) const { return a.chain_tiles + (row + k) * a.D + c; }
  __device__ __forceinline__ uint64_t* eight_words(int k) const { return a.chain_eights + (row8 + k) * a.D + c; }
  __device__ __forceinline__ uint64_t* state_words(int k) const { return a.chain_states + (row64 + k) * a.D + c; }
  // the slots of the tiles before this one in its eight, and of the eights before its own; the last wave
  // takes the state before the 64
  __device__ __forceinline__ bool one() const { return wave < EIGHT - 1 && tile0 + wave >= tile1 && tile0 + wave < q; }
  __device__ __forceinline__ bool two() const {
    return from < tile0 && wave < EIGHT - 1 && eight0 + wave >= eight1 && eight0 + wave < q / EIGHT;
  }
  __device__ __forceinline__ bool three() const { return wave == EIGHT - 1 && from < eight0 * EIGHT; }

  __device__ __forceinline__ Joint(const RecLaunch& args, const Where& at, int run, Link& link)
      : a(args), l(link), wave(run), q(at.order), from(link.from), tiles((int)args.tiles), on(at.c < args.D), fresh(false), c(at.c) {
    static_assert(RUNS == EIGHT, "a wave for every slot");
    tile0 = q / EIGHT * EIGHT;
    eight0 = q / (EIGHT * EIGHT) * EIGHT;
    tile1 = from > tile0 ? from : tile0;
    eight1 = from / EIGHT > eight0 ? from / EIGHT : eight0;
    row = (int64_t)at.b * tiles;
    row8 = (int64_t)at.b * (tiles / EIGHT);
    row64 = (int64_t)at.b * (tiles / (EIGHT * EIGHT));
    if (tiles == 1) return;
    if (wave == 0) {
      for (int k = 0; k < RUNS; ++k) {
        h = l.run.behind(k, h, l.fresh[k] != 0);
        P = mul2(P, l.run.P[k][lane_id()]);
        fresh = fresh || l.fresh[k] != 0;
      }
      if (on && q + 1 < tiles) publish(tile_words(q), P, h);
    }
    near.look(one() && on ? tile_words(tile0 + wave) : nullptr);
    far.look(on && two() ? eight_words(eight0 + wave) : on && three() ? state_words(eight0 / EIGHT - 1) : nullptr);
  }

  __device__ __forceinline__ f32x2 start() {
    f32x2 x{0.f, 0.f};
    if (tiles == 1) return x;
    const bool closes = q % EIGHT == EIGHT - 1 && q + 1 < tiles;  // the tile ends its eight, for others to use
    if (from < q) {
      f32x2 Pk, hk;
      near.wait(Pk, hk);
      if (one()) l.tiles.put(wave, Pk, hk);
      // the eight's end does not wait for what comes before the eight
      if (closes) {
        __syncthreads();
        if (wave == 0) {
          f32x2 y{0.f, 0.f}, Py{1.f, 1.f};  // Py is read only where no sequence starts in the eight
          for (int k = tile1; k < q; ++k) {
            y = l.tiles.behind(k - tile0, y, k == from);
            Py = mul2(Py, l.tiles.P[k - tile0][lane_id()]);
          }
          if (on) publish(eight_words(q / EIGHT), mul2(Py, P), fresh ? h : fma2(P, y, h));
        }
      }
      far.wait(Pk, hk);
      if (two()) l.eights.put(wave, Pk, hk);
      if (three()) l.before[lane_id()] = hk;
      __syncthreads();
      if (from < eight0 * EIGHT) x = l.before[lane_id()];
      if (from < tile0)
        for (int k = eight1; k < q / EIGHT; ++k) x = l.eights.behind(k - eight0, x, k == from / EIGHT);
      for (int k = tile1; k < q; ++k) x = l.tiles.behind(k - tile0, x, k == from);
    } else if (closes && wave == 0 && on) {
      publish(eight_words(q / EIGHT), P, h);  // nothing comes from before: h alone is read
    }
    // the state behind 64 tiles
    if (wave == 0 && q % (EIGHT * EIGHT) == EIGHT * EIGHT - 1 && q + 1 < tiles && on)
      publish(state_words(eight0 / EIGHT), P, fresh || from == q ? h : fma2(P, x, h));
    return x;
  }
};

// the rows of a run, two channels a lane: A, X, I and backwards dH
template <class E, int RUN, bool GATE, bool BWD>
struct Raw {
  typename Pair<E>::raw A[RUN], X[RUN], I[GATE ? RUN : 1], G[BWD ? RUN : 1];
};
template <class E, int RUN, bool GATE, bool BWD>
__device__ __forceinline__ void load_rows(const RecLaunch& a, const Where& at, Raw<E, RUN, GATE, BWD>& r) {
  const Rows<E> A(a, at, a.A, a.a_stride), X(a, at, a.X, a.x_stride), I(a, at, GATE ? a.I : a.X, GATE ? a.i_stride : a.x_stride),
      G(a, at, BWD ? a.dH : a.X, BWD ? a.D : a.x_stride);
#pragma unroll
  for (int j = 0; j < RUN; ++j) r.A[j] = A.load(a, at, j);
  if constexpr (BWD)
#pragma unroll
    for (int j = 0; j < RUN; ++j) r.G[j] = G.load(a, at, j);
#pragma unroll
  for (int j = 0; j < RUN; ++j) r.X[j] = X.load(a, at, j);
  if constexpr (GATE)
#pragma unroll
    for (int j = 0; j < RUN; ++j) r.I[j] = I.load(a, at, j);
}

// a and b of a token
template <class E, int DECAY, int NORM>
__device__ __forceinline__ void open_gate(typename Pair<E>::raw A, f32x2 w, f32x2& dec, f32x2& b) {
  const f32x2 Av = Pair<E>::open(A);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Gate<E, DECAY, NORM> g(Av[k], w[k]);
    dec[k] = g.a;
    b[k] = g.b;
  }
}
// u = b s(I) X of a token
template <class E, bool GATE>
__device__ __forceinline__ f32x2 input_of(typename Pair<E>::raw X, typename Pair<E>::raw I, f32x2 b) {
  f32x2 u = mul2(b, Pair<E>::open(X));
  if constexpr (GATE) {
    const f32x2 i = Pair<E>::open(I);
    u = mul2(u, f32x2{sigmoid<E>(i[0]), sigmoid<E>(i[1])});
  }
  return u;
}

// the run's end (P, h) from P = 1 and h
template <bool PLAIN, int RUN>
__device__ __forceinline__ void walk(const RecLaunch& a, const Where& at, const Run<RUN>& r, const f32x2 (&dec)[RUN],
                                     const f32x2 (&u)[RUN], f32x2& P, f32x2& h) {
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    if (!PLAIN) {
      if (!(r.in >> j & 1)) continue;
      if (r.first >> j & 1) h = state_in(a, a.h0, r.seq_of(j), at.c);
    }
    h = fma2(dec[j], h, u[j]);
    P = mul2(P, dec[j]);
  }
}

}  // namespace

// H, the last states and the states at the tiles' starts (each where wanted)
template <class E, int DECAY, int NORM, bool GATE>
__global__ __launch_bounds__(RUNS* WAVE) __attribute__((amdgpu_waves_per_eu(4, 4))) void rec_fwd_kernel(RecLaunch a) {
  constexpr int RUN = FWD_TILE / RUNS;
  __shared__ Link l;
  const Where at = find_place<RUN, false>(a);
  Raw<E, RUN, GATE, false> raw;
  load_rows(a, at, raw);
  const Run<RUN> r = find_run<RUN>(a, at.t0, at.b);
  f32x2 dec[RUN], u[RUN];
  const f32x2 w = channel_w(a, at.c);
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    f32x2 b;
    open_gate<E, DECAY, NORM>(raw.A[j], w, dec[j], b);
    u[j] = input_of<E, GATE>(raw.X[j], raw.I[GATE ? j : 0], b);
  }
  f32x2 P{1.f, 1.f}, h{0.f, 0.f};
  if (r.plain())
    walk<true>(a, at, r, dec, u, P, h);
  else
    walk<false>(a, at, r, dec, u, P, h);
  l.run.put(at.wave, P, h);
  const bool goes_on = (r.in & 1) && !(r.first & 1);  // the run's first token continues a sequence
  if (lane_id() == 0) {
    l.fresh[at.wave] = r.first != 0;
    if (at.wave == 0) l.from = goes_on ? r.from / (RUN * RUNS) : at.order;
  }
  __syncthreads();
  h = l.before_run(at.wave, Joint(a, at, at.wave, l).start());
  if (at.t0 % GDN_REC_TILE == 0 && at.t0 < a.T)
    state_out(a, a.states, (int64_t)at.b * a.n_states + at.t0 / GDN_REC_TILE, at.c, goes_on ? h : f32x2{0.f, 0.f});
  if (!a.H) return;  // the states alone
  const Rows<E> H(a, at, a.H, a.D);
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    if (!(r.in >> j & 1)) continue;
    if (r.first >> j & 1) h = state_in(a, a.h0, r.seq_of(j), at.c);
    h = fma2(dec[j], h, u[j]);
    H.store(a, at, j, h);
    if (r.last >> j & 1) state_out(a, a.h_out, r.seq_of(j), at.c, h);
  }
  empty_sequences(a, at, a.h0, a.h_out);
}

// all gradients, from the states at the tiles' starts; the chain runs backwards
template <class E, int DECAY, int NORM, bool GATE>
__global__ __launch_bounds__(RUNS* WAVE) __attribute__((amdgpu_waves_per_eu(4, 4))) void rec_bwd_kernel(RecLaunch a) {
  constexpr int RUN = BWD_TILE / RUNS;
  __shared__ Link l;
  __shared__ f32x2 fwd[RUNS][WAVE];  // the runs' ends forwards
  __shared__ int starts[RUNS];
  const Where at = find_place<RUN, true>(a);
  const int run = RUNS - 1 - at.wave;  // in the chain's order
  Raw<E, RUN, GATE, true> raw;
  load_rows(a, at, raw);
  f32x2 h{0.f, 0.f};
  if (a.tiles > 1) h = state_in(a, a.states, (int64_t)at.b * a.n_states + at.tile * (BWD_TILE / GDN_REC_TILE), at.c);
  const Run<RUN> r = find_run<RUN>(a, at.t0, at.b);
  const f32x2 w = channel_w(a, at.c);
  f32x2 dec[RUN], b[RUN], u[RUN];
#pragma unroll
  for (int j = 0; j < RUN; ++j) open_gate<E, DECAY, NORM>(raw.A[j], w, dec[j], b[j]);
  f32x2 P{1.f, 1.f}, e{0.f, 0.f};
#pragma unroll
  for (int j = RUN - 1; j >= 0; --j) {
    if (!(r.in >> j & 1)) continue;
    if (r.last >> j & 1) e = state_in(a, a.dh, r.seq_of(j), at.c);
    const f32x2 d = Pair<E>::open(raw.G[j]);
    e = f32x2{dec[j][0] * (d[0] + e[0]), dec[j][1] * (d[1] + e[1])};
    P = mul2(P, dec[j]);
  }
  l.run.put(run, P, e);
  if (lane_id() == 0) {
    starts[at.wave] = r.first != 0;
    l.fresh[run] = r.last != 0;
  }
  if (run == 0) {
    // the tile's last token goes on into the next tile
    const bool goes_on = (r.in >> (RUN - 1) & 1) && !(r.last >> (RUN - 1) & 1);
    const int to = __builtin_amdgcn_readlane(r.to, RUN - 1);
    if (lane_id() == 0) l.from = goes_on ? (int)a.tiles - 1 - (to - 1) / (RUN * RUNS) : at.order;
  }
  __syncthreads();
  Joint joint(a, at, run, l);
  // the states, while the words are on their way
#pragma unroll
  for (int j = 0; j < RUN; ++j) u[j] = input_of<E, GATE>(raw.X[j], raw.I[GATE ? j : 0], b[j]);
  f32x2 x{0.f, 0.f};
  walk<false>(a, at, r, dec, u, P, x);
  fwd[at.wave][lane_id()] = x;
  __syncthreads();
  // the runs' products are those of the chain's way
  for (int k = 0; k < at.wave; ++k) {
    const f32x2 y = fwd[k][lane_id()];
    h = starts[k] != 0 ? y : fma2(l.run.P[RUNS - 1 - k][lane_id()], h, y);
  }
  // u gives way to the states before the tokens
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    if (!(r.in >> j & 1)) continue;
    if (r.first >> j & 1) h = state_in(a, a.h0, r.seq_of(j), at.c);
    const f32x2 before = h;
    h = fma2(dec[j], h, u[j]);
    u[j] = before;
  }
  // the rows are opened anew below: kept open from above they would take twice the registers
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    hide(raw.A[j]);
    hide(raw.X[j]);
    hide(raw.G[j]);
    if constexpr (GATE) hide(raw.I[j]);
  }
  e = l.before_run(run, joint.start());
  const Rows<E> X(a, at, a.dX, a.D), A(a, at, a.dA, a.D), I(a, at, GATE ? a.dI : a.dX, a.D);
  f32x2 dw{0.f, 0.f};
#pragma unroll
  for (int j = RUN - 1; j >= 0; --j) {
    f32x2 dX{0.f, 0.f}, dA{0.f, 0.f}, dI{0.f, 0.f};
    if (r.in >> j & 1) {
      if (r.last >> j & 1) e = state_in(a, a.dh, r.seq_of(j), at.c);
      const f32x2 d = Pair<E>::open(raw.G[j]), Av = Pair<E>::open(raw.A[j]), x = Pair<E>::open(raw.X[j]);
      const f32x2 iv = Pair<E>::open(raw.I[GATE ? j : 0]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const GateGrad<E, DECAY> g(Av[k], w[k]);
        const float D = d[k] + e[k];
        e[k] = dec[j][k] * D;
        float s = 1.f, rest = 0.f;
        if constexpr (GATE) sigmoid_rest<E>(iv[k], s, rest);
        const float dz = D * b[j][k], z = s * x[k];
        dX[k] = dz * s;
        dI[k] = dz * z * rest;
        const float dg = fmaf(e[k], u[j][k], D * z * slope<NORM>(dec[j][k], b[j][k]));
        dA[k] = dg * g.to_A;
        dw[k] = fmaf(-g.r, dg, dw[k]);
      }
      if (r.first >> j & 1) state_out(a, a.dh0, r.seq_of(j), at.c, e);
    }
    if (at.t0 + j < a.T) {  // rows of no sequence: zeros
      X.store(a, at, j, dX);
      A.store(a, at, j, dA);
      if constexpr (GATE) I.store(a, at, j, dI);
    }
  }
  empty_sequences(a, at, a.dh, a.dh0);
  if (DECAY != GDN_DECAY_POWER || !a.dw) return;
  __syncthreads();
  fwd[at.wave][lane_id()] = dw;
  __syncthreads();
  if (at.wave != 0 || at.c >= a.D) return;
  dw = f32x2{0.f, 0.f};
  for (int k = 0; k < RUNS; ++k) dw += fwd[k][lane_id()];
  *reinterpret_cast<f32x2*>(a.part + ((int64_t)at.b * a.tiles + at.tile) * a.D + at.c) = dw;
}

// token by token, the state in registers for the whole call: a wave for each 128 channels of a
// sequence.  h_out may be h0: a lane reads and writes its own channels alone.
template <class E, int DECAY, int NORM, bool GATE>
__global__ __launch_bounds__(256) void rec_step_kernel(RecLaunch a) {
  const uint32_t blocks = (uint32_t)((a.D + CH - 1) / CH);
  const uint32_t i = blockIdx.x * 4 + threadIdx.x / WAVE, b = i / blocks;
  const int c = (int)(i - b * blocks) * CH + 2 * lane_id();
  if (b >= (uint32_t)a.n_seq || c >= a.D) return;
  f32x2 h = state_in(a, a.h0, (int)b, c);
  const f32x2 w = channel_w(a, c);
  typedef typename Pair<E>::raw raw;
  for (int64_t t = 0; t < a.T; ++t) {
    const int64_t row = (int64_t)b * a.T + t;
    const f32x2 Av = Pair<E>::open(*reinterpret_cast<const raw*>(reinterpret_cast<const E*>(a.A) + row * a.a_stride + c));
    const f32x2 x = Pair<E>::open(*reinterpret_cast<const raw*>(reinterpret_cast<const E*>(a.X) + row * a.x_stride + c));
    f32x2 iv{0.f, 0.f};
    if constexpr (GATE) iv = Pair<E>::open(*reinterpret_cast<const raw*>(reinterpret_cast<const E*>(a.I) + row * a.i_stride + c));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Gate<E, DECAY, NORM> g(Av[k], w[k]);
      h[k] = fmaf(g.a, h[k], g.b * (GATE ? sigmoid<E>(iv[k]) : 1.f) * x[k]);
    }
    *reinterpret_cast<raw*>(reinterpret_cast<E*>(a.H) + row * a.D + c) = Pair<E>::close(h);
  }
  state_out(a, a.h_out, (int)b, c, h);
}

// without tokens, the states as they were given, or zeros
__global__ __launch_bounds__(256) void rec_copy_kernel(const float* from, float* to, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    to[i] = from ? from[i] : 0.f;
}

// NOT_YET in every word of the chains
__global__ __launch_bounds__(256) void rec_clear_kernel(u32x4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = u32x4{NOT_YET, NOT_YET, NOT_YET, NOT_YET};
}

// ---- host side ----------------------------------------------------------------------------

namespace {

template <class F>
int by_kind(const RecLaunch& p, F&& f) {
  auto gate = [&](auto e, auto decay, auto norm) {
    return p.I ? f(e, decay, norm, std::true_type{}) : f(e, decay, norm, std::false_type{});
  };
  auto norm = [&](auto e, auto decay) {
    switch (p.norm) {
      case GDN_REC_NORM_SQRT: return gate(e, decay, std::integral_constant<int, GDN_REC_NORM_SQRT>{});
      case GDN_REC_NORM_LINEAR: return gate(e, decay, std::integral_constant<int, GDN_REC_NORM_LINEAR>{});
      default: return gate(e, decay, std::integral_constant<int, GDN_REC_NORM_NONE>{});
    }
  };
  auto decay = [&](auto e) {
    switch (p.decay) {
      case GDN_DECAY_POWER: return norm(e, std::integral_constant<int, GDN_DECAY_POWER>{});
      case GDN_DECAY_SIGMOID: return norm(e, std::integral_constant<int, GDN_DECAY_SIGMOID>{});
      default: return norm(e, std::integral_constant<int, GDN_DECAY_LOG>{});
    }
  };
  return p.bf16 ? decay((__bf16*)nullptr) : decay((float*)nullptr);
}

int64_t channel_blocks(const RecLaunch& p) { return (p.D + CH - 1) / CH; }
int64_t rows_of(const RecLaunch& p) { return p.offsets ? 1 : p.n_seq; }
size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// the workspace in order: a chain's words (the ends of the tiles and of their eights, the states behind 64
// tiles, the counters), backwards those of a pass for the states and the states themselves, dw's parts
struct Parts {
  int64_t n;
  size_t tiles, eights, states, tickets, chain;  // offsets in a chain's words, and their size
  size_t fwd_chain, starts, part, bytes;         // backwards
  Parts(const RecLaunch& p, bool bwd) {
    const int tile = bwd ? BWD_TILE : FWD_TILE;
    const int64_t rows = rows_of(p), v = rows * p.D;
    n = (p.T + tile - 1) / tile;
    tiles = 0;
    eights = tiles + up16((size_t)(n * v) * 8);
    states = eights + up16((size_t)(n / EIGHT * v) * 8);
    tickets = states + up16((size_t)(n / EIGHT / EIGHT * v) * 8);
    chain = n > 1 ? tickets + up16((size_t)(rows * channel_blocks(p)) * 4) : 0;
    bytes = chain;
    if (!bwd) return;
    fwd_chain = bytes;
    starts = fwd_chain + Parts(p, false).chain;
    part = starts + (n > 1 ? up16((size_t)(rows * p.n_states * p.D) * 4) : 0);
    bytes = part + (p.decay == GDN_DECAY_POWER ? up16((size_t)(n * v) * 4) : 0);
  }
};

// the call with its chain's words at ws, filled
RecLaunch chained(const RecLaunch& p, bool bwd, char* ws, hipStream_t s) {
  RecLaunch q = p;
  const Parts at(p, bwd);
  q.tiles = at.n;
  if (q.tiles > 1) {
    q.chain_tiles = reinterpret_cast<uint64_t*>(ws + at.tiles);
    q.chain_eights = reinterpret_cast<uint64_t*>(ws + at.eights);
    q.chain_states = reinterpret_cast<uint64_t*>(ws + at.states);
    q.tickets = reinterpret_cast<uint32_t*>(ws + at.tickets);
    const int64_t n = (int64_t)(at.chain / 16), g = (n + 255) / 256;
    hipLaunchKernelGGL(rec_clear_kernel, dim3((unsigned)(g < 2048 ? g : 2048)), dim3(256), 0, s,
                       reinterpret_cast<u32x4*>(ws), n);
  }
  return q;
}

void copy_states(const float* from, float* to, int64_t n, hipStream_t s) {
  if (!to || n == 0) return;
  const int64_t g = (n + 255) / 256;
  hipLaunchKernelGGL(rec_copy_kernel, dim3((unsigned)(g < 1024 ? g : 1024)), dim3(256), 0, s, from, to, n);
}

dim3 grid_of(const RecLaunch& q) { return dim3((unsigned)(q.tiles * rows_of(q) * channel_blocks(q))); }

}  // namespace

size_t rec_workspace(const RecLaunch& p, bool bwd) { return p.T == 0 || rows_of(p) == 0 ? 0 : Parts(p, bwd).bytes; }

bool rec_grid_ok(const RecLaunch& p) {
  // a launch has fewer than 2^32 threads
  constexpr int least = FWD_TILE < BWD_TILE ? FWD_TILE : BWD_TILE;
  const int64_t tiles = (p.T + least - 1) / least, rows = rows_of(p) > 0 ? rows_of(p) : 1;
  return tiles <= (((int64_t)1 << 32) - 1) / (RUNS * WAVE) / channel_blocks(p) / rows;
}
bool rec_step_grid_ok(const RecLaunch& p) { return p.n_seq <= (((int64_t)1 << 32) - 256) / WAVE / channel_blocks(p); }

int launch_rec_fwd(const RecLaunch& p, void* workspace, hipStream_t s) {
  if (p.T == 0) {
    copy_states(p.h0, p.h_out, (int64_t)p.n_seq * p.D, s);
    return 0;
  }
  if (p.n_seq == 0) {  // rows of no sequence: zeros before every token
    copy_states(nullptr, p.states, p.n_states * p.D, s);
    return 0;
  }
  const RecLaunch q = chained(p, false, reinterpret_cast<char*>(workspace), s);
  return by_kind(p, [&](auto e, auto decay, auto norm, auto gate) {
    typedef std::remove_pointer_t<decltype(e)> E;
    hipLaunchKernelGGL((rec_fwd_kernel<E, decay.value, norm.value, gate.value>), grid_of(q), dim3(RUNS * WAVE), 0, s, q);
    return 0;
  });
}

int launch_rec_bwd(const RecLaunch& p, void* workspace, hipStream_t s) {
  if (p.T == 0 || rows_of(p) == 0) {
    copy_states(p.dh, p.dh0, (int64_t)p.n_seq * p.D, s);
    copy_states(nullptr, p.dw, p.D, s);
    return 0;
  }
  char* ws = reinterpret_cast<char*>(workspace);
  const Parts at(p, true);
  RecLaunch q = chained(p, true, ws, s);
  q.part = reinterpret_cast<float*>(ws + at.part);
  const bool form = q.tiles > 1 && !p.states;
  RecLaunch f{};
  if (form) {
    q.states = reinterpret_cast<float*>(ws + at.starts);
    f = chained(p, false, ws + at.fwd_chain, s);
    f.H = nullptr;
    f.h_out = nullptr;
    f.states = q.states;
  }
  return by_kind(p, [&](auto e, auto decay, auto norm, auto gate) {
    typedef std::remove_pointer_t<decltype(e)> E;
    if (form) hipLaunchKernelGGL((rec_fwd_kernel<E, decay.value, norm.value, gate.value>), grid_of(f), dim3(RUNS * WAVE), 0, s, f);
    hipLaunchKernelGGL((rec_bwd_kernel<E, decay.value, norm.value, gate.value>), grid_of(q), dim3(RUNS * WAVE), 0, s, q);
    if (q.dw) launch_column_sum(q.part, q.tiles * rows_of(q), q.D, 1, q.dw, nullptr, s);
    return 0;
  });
}

int launch_rec_step(const RecLaunch& p, hipStream_t s) {
  const int64_t waves = (int64_t)p.n_seq * channel_blocks(p);
  const dim3 grid((unsigned)((waves + 3) / 4)), block(256);
  return by_kind(p, [&](auto e, auto decay, auto norm, auto gate) {
    hipLaunchKernelGGL((rec_step_kernel<std::remove_pointer_t<decltype(e)>, decay.value, norm.value, gate.value>), grid, block, 0, s, p);
    return 0;
  });
}

}  // namespace gdn
