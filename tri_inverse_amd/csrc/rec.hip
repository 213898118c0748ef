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
// decays.  A workgroup takes a tile of 64 tokens and 128 channels, two to a lane, so that a row
// of a wave is 256 contiguous bytes (bf16), each wave a run of 8 tokens in registers.  The ends of the runs
// join in LDS; the ends of the tiles in a second launch; a third forms the outputs from every
// tile's start.  Decays, states and sums are fp32; 1 - a is formed without cancelling (expm1),
// each output is rounded once.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

constexpr int RUN = 8;      // tokens of a wave
constexpr int RUNS = 8;     // waves of a workgroup
constexpr int TILE = REC_TILE;
constexpr int CH = 2 * WAVE;  // channels of a workgroup
static_assert(RUN * RUNS == TILE, "");

typedef float f32x2 __attribute__((ext_vector_type(2)));

// two neighbouring channels as they lie in memory, and as fp32
template <class E>
struct Pair;
template <>
struct Pair<__bf16> {
  typedef uint32_t raw;
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
  static __device__ __forceinline__ f32x2 open(raw v) { return v; }
  static __device__ __forceinline__ raw close(f32x2 v) { return v; }
};

__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// sigmoid and what it leaves of 1, neither by a difference that cancels
__device__ __forceinline__ void sigmoid2(float z, float& s, float& rest) {
  const float e = __expf(-z);
  s = rcp(1.f + e);
  rest = z < 0.f ? 1.f - s : e * s;
}
__device__ __forceinline__ float sigmoid1(float z) { return rcp(1.f + __expf(-z)); }

// e^g - 1, a = e^g known: near 0 the series, whose first term left out is below 2^-24 of it
__device__ __forceinline__ float expm1_of(float g, float a) {
  float p = 1.f / 720.f;
  p = fmaf(p, g, 1.f / 120.f);
  p = fmaf(p, g, 1.f / 24.f);
  p = fmaf(p, g, 1.f / 6.f);
  p = fmaf(p, g, 0.5f);
  p = fmaf(p, g, 1.f);
  return fabsf(g) < 0.25f ? p * g : a - 1.f;
}

// the decay of a token, the factor b of its input; backwards also b'(g) and what turns dg into dA
// (to_A) and dw (r)
template <int DECAY, int NORM>
struct Gate {
  float a, b, db, to_A, r;
  __device__ __forceinline__ Gate(float A, float w) {
    float m = 0.f;  // a - 1
    db = 0.f;
    r = 0.f;
    if constexpr (DECAY == GDN_DECAY_SIGMOID) {
      sigmoid2(A, a, to_A);
      m = -to_A;
    } else {
      float g = A;
      to_A = 1.f;
      if constexpr (DECAY == GDN_DECAY_POWER) {
        float rest;
        sigmoid2(A, r, rest);
        g = -w * r;
        to_A = g * rest;
      }
      a = __expf(g);
      if constexpr (NORM != GDN_REC_NORM_NONE) m = expm1_of(g, a);
    }
    if constexpr (NORM == GDN_REC_NORM_SQRT) {
      const float q = -m * (2.f + m);  // 1 - a^2
      // a = 1: b = 0, whose own gradient counts as 0
      const float rs = q == 0.f ? 0.f : __builtin_amdgcn_rsqf(q);
      b = q * rs;
      db = -a * a * rs;
    } else {
      b = NORM == GDN_REC_NORM_LINEAR ? -m : 1.f;
      if constexpr (NORM == GDN_REC_NORM_LINEAR) db = -a;
    }
  }
};

// ---- sequences in a run of tokens ---------------------------------------------------------

// bit j of the masks: token t0 + j belongs to a sequence, is its first, its last one.  seq: in lane j
// the sequence of token t0 + j.  Offsets are clamped to the tokens, sequences to the given ones, so
// offsets that break their rule lead to no access outside.
struct Run {
  uint32_t in, first, last;
  int seq;
  // all tokens in one sequence that neither starts nor ends here
  __device__ __forceinline__ bool plain() const { return in == (1u << RUN) - 1 && (first | last) == 0; }
  __device__ __forceinline__ int seq_of(int j) const { return __builtin_amdgcn_readlane(seq, j); }
};

__device__ __forceinline__ int64_t offset_at(const RecLaunch& a, int i) {
  const int64_t o = a.offsets[i];
  return o < 0 ? 0 : o > a.T ? a.T : o;
}

__device__ __forceinline__ Run find_run(const RecLaunch& a, int64_t t0, int b) {
  Run r;
  if (!a.offsets) {
    const int64_t left = a.T - t0;
    const int n = left < 0 ? 0 : left > RUN ? RUN : (int)left;
    r.in = (1u << n) - 1;
    r.first = t0 == 0 && n > 0 ? 1u : 0u;
    r.last = left >= 1 && left <= RUN ? 1u << (n - 1) : 0u;
    r.seq = b;
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
  const int64_t s = some ? offset_at(a, lo) : 0, e = some ? offset_at(a, lo + 1) : 0;
  const bool in = some && t < e && t < a.T && lane_id() < RUN;
  r.in = (uint32_t)__builtin_amdgcn_ballot_w64(in);
  r.first = (uint32_t)__builtin_amdgcn_ballot_w64(in && t == s);
  r.last = (uint32_t)__builtin_amdgcn_ballot_w64(in && t + 1 == e);
  return r;
}

// what joining needs to know of a tile
enum { TILE_STARTS = 1, TILE_CONTINUES = 2, TILE_ENDS = 4, TILE_GOES_ON = 8 };

struct Where {
  int wave, cb, b;
  int64_t tile, t0;  // the tile in its row; the run's first token
  int c;             // the lane's first channel; D or more: none
  __device__ __forceinline__ Where(const RecLaunch& a) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const uint32_t blocks = (uint32_t)((a.D + CH - 1) / CH);
    const uint32_t i = blockIdx.x / blocks;
    cb = (int)(blockIdx.x - i * blocks);
    b = (int)(i / (uint32_t)a.tiles);
    tile = i - (uint32_t)b * (uint32_t)a.tiles;
    t0 = tile * TILE + (int64_t)wave * RUN;
    c = cb * CH + 2 * lane_id();
  }
};

// the run's rows of a tensor, two channels a lane: rows past the last token and lanes past the last
// channel load what lies inside instead
template <class E>
__device__ __forceinline__ void load_run(const RecLaunch& a, const Where& at, const void* p, int64_t stride,
                                         typename Pair<E>::raw (&v)[RUN]) {
  const E* base = reinterpret_cast<const E*>(p) + (int64_t)at.b * a.T * stride;
  const int c = at.c < a.D ? at.c : 0;
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    const int64_t t = at.t0 + j < a.T ? at.t0 + j : a.T - 1;
    v[j] = *reinterpret_cast<const typename Pair<E>::raw*>(base + t * stride + c);
  }
}

template <class E>
__device__ __forceinline__ void store_row(const RecLaunch& a, const Where& at, void* p, int j, f32x2 v) {
  if (at.c < a.D)
    *reinterpret_cast<typename Pair<E>::raw*>(reinterpret_cast<E*>(p) + ((int64_t)at.b * a.T + at.t0 + j) * a.D + at.c) =
        Pair<E>::close(v);
}

__device__ __forceinline__ f32x2 state_in(const RecLaunch& a, const float* S, int seq, int c) {
  f32x2 h{0.f, 0.f};
  if (S && c < a.D) h = *reinterpret_cast<const f32x2*>(S + (int64_t)seq * a.D + c);
  return h;
}
__device__ __forceinline__ void state_out(const RecLaunch& a, float* S, int seq, int c, f32x2 h) {
  if (S && c < a.D) *reinterpret_cast<f32x2*>(S + (int64_t)seq * a.D + c) = h;
}

__device__ __forceinline__ f32x2 fma2(f32x2 x, f32x2 y, f32x2 z) {
  return f32x2{fmaf(x[0], y[0], z[0]), fmaf(x[1], y[1], z[1])};
}

__device__ __forceinline__ f32x2 channel_w(const RecLaunch& a, int c) {
  f32x2 w{0.f, 0.f};
  if (a.w && c < a.D) w = *reinterpret_cast<const f32x2*>(a.w + c);
  return w;
}

// a and u of every token of the run
template <class E, int DECAY, int NORM>
__device__ __forceinline__ void open_run(const RecLaunch& a, const Where& at, f32x2 (&dec)[RUN], f32x2 (&u)[RUN]) {
  typename Pair<E>::raw A[RUN], X[RUN], I[RUN];
  load_run<E>(a, at, a.A, a.a_stride, A);
  load_run<E>(a, at, a.X, a.x_stride, X);
  if (a.I) load_run<E>(a, at, a.I, a.i_stride, I);
  const f32x2 w = channel_w(a, at.c);
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    const f32x2 Av = Pair<E>::open(A[j]), x = Pair<E>::open(X[j]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Gate<DECAY, NORM> g(Av[k], w[k]);
      dec[j][k] = g.a;
      u[j][k] = g.b * x[k];
    }
    if (a.I) {
      const f32x2 i = Pair<E>::open(I[j]);
#pragma unroll
      for (int k = 0; k < 2; ++k) u[j][k] *= sigmoid1(i[k]);
    }
  }
}

// the end of a run that starts from h: P and h on entry (1, start), reset where a sequence starts
template <bool PLAIN, class Fn>
__device__ __forceinline__ void walk(const RecLaunch& a, const Where& at, const Run& r, const f32x2 (&dec)[RUN],
                                     const f32x2 (&u)[RUN], f32x2& P, f32x2& h, Fn&& each) {
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    if (!PLAIN) {
      if (!(r.in >> j & 1)) continue;
      if (r.first >> j & 1) {
        h = state_in(a, a.h0, r.seq_of(j), at.c);
        P = f32x2{0.f, 0.f};
      }
    }
    each(j, h);
    h = fma2(dec[j], h, u[j]);
    P = f32x2{P[0] * dec[j][0], P[1] * dec[j][1]};
  }
}

// runs and tiles join by (P, h): a run in which a sequence starts takes nothing from before
__device__ __forceinline__ f32x2 join(f32x2 P, f32x2 h, f32x2 start, bool starts) {
  return starts ? h : fma2(P, start, h);
}

struct RunEnds {
  f32x2 P[RUNS][WAVE], h[RUNS][WAVE];
  int starts[RUNS];
};

// the state before run n of the tile that starts from h
__device__ __forceinline__ f32x2 before_run(const RunEnds& e, int n, f32x2 h) {
  for (int k = 0; k < n; ++k) h = join(e.P[k][lane_id()], e.h[k][lane_id()], h, e.starts[k] != 0);
  return h;
}

// sequences without tokens return their states as they were given; dealt out over the tiles
__device__ __forceinline__ void empty_sequences(const RecLaunch& a, const Where& at, const float* from, float* to) {
  if (!a.offsets || !to || at.wave != 0) return;
  for (int64_t s = at.tile; s < a.n_seq; s += a.tiles)
    if (offset_at(a, (int)s) >= offset_at(a, (int)s + 1)) state_out(a, to, (int)s, at.c, state_in(a, from, (int)s, at.c));
}

}  // namespace

// the ends (P, h) of every tile, and its flags
template <class E, int DECAY, int NORM>
__global__ __launch_bounds__(RUNS* WAVE) void rec_ends_kernel(RecLaunch a) {
  __shared__ RunEnds ends;
  __shared__ uint32_t masks[RUNS][3];
  const Where at(a);
  f32x2 dec[RUN], u[RUN];
  const Run r = find_run(a, at.t0, at.b);
  open_run<E, DECAY, NORM>(a, at, dec, u);
  f32x2 P{1.f, 1.f}, h{0.f, 0.f};
  auto nothing = [](int, f32x2) {};
  if (r.plain())
    walk<true>(a, at, r, dec, u, P, h, nothing);
  else
    walk<false>(a, at, r, dec, u, P, h, nothing);
  ends.P[at.wave][lane_id()] = P;
  ends.h[at.wave][lane_id()] = h;
  ends.starts[at.wave] = r.first != 0;
  if (lane_id() == 0) {
    masks[at.wave][0] = r.in;
    masks[at.wave][1] = r.first;
    masks[at.wave][2] = r.last;
  }
  __syncthreads();
  if (at.wave != 0) return;
  P = f32x2{1.f, 1.f};
  h = f32x2{0.f, 0.f};
  uint32_t first = 0, last = 0;
  for (int k = 0; k < RUNS; ++k) {
    h = join(ends.P[k][lane_id()], ends.h[k][lane_id()], h, ends.starts[k] != 0);
    const f32x2 Pk = ends.P[k][lane_id()];
    P = f32x2{P[0] * Pk[0], P[1] * Pk[1]};
    first |= masks[k][1];
    last |= masks[k][2];
  }
  const int64_t i = (int64_t)at.b * a.tiles + at.tile;
  if (at.c < a.D) {
    *reinterpret_cast<f32x2*>(a.tile_P + i * a.D + at.c) = P;
    *reinterpret_cast<f32x2*>(a.tile_h + i * a.D + at.c) = h;
  }
  if (at.cb == 0 && lane_id() == 0)
    a.tile_flags[i] = (first ? TILE_STARTS : 0) | (last ? TILE_ENDS : 0) |
                      ((masks[0][0] & 1) && !(masks[0][1] & 1) ? TILE_CONTINUES : 0) |
                      ((masks[RUNS - 1][0] >> (RUN - 1)) && !(masks[RUNS - 1][2] >> (RUN - 1)) ? TILE_GOES_ON : 0);
}

// the ends (P, e) of every tile backwards
template <class E, int DECAY, int NORM>
__global__ __launch_bounds__(RUNS* WAVE) void rec_ends_bwd_kernel(RecLaunch a) {
  __shared__ RunEnds ends;
  const Where at(a);
  const Run r = find_run(a, at.t0, at.b);
  typename Pair<E>::raw A[RUN], G[RUN];
  load_run<E>(a, at, a.A, a.a_stride, A);
  load_run<E>(a, at, a.dH, a.D, G);
  const f32x2 w = channel_w(a, at.c);
  f32x2 P{1.f, 1.f}, e{0.f, 0.f};
#pragma unroll
  for (int j = RUN - 1; j >= 0; --j) {
    if (!(r.in >> j & 1)) continue;
    if (r.last >> j & 1) {
      e = state_in(a, a.dh, r.seq_of(j), at.c);
      P = f32x2{0.f, 0.f};
    }
    const f32x2 Av = Pair<E>::open(A[j]), d = Pair<E>::open(G[j]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Gate<DECAY, GDN_REC_NORM_NONE> g(Av[k], w[k]);
      e[k] = g.a * (d[k] + e[k]);
      P[k] *= g.a;
    }
  }
  ends.P[at.wave][lane_id()] = P;
  ends.h[at.wave][lane_id()] = e;
  ends.starts[at.wave] = r.last != 0;
  __syncthreads();
  if (at.wave != 0) return;
  P = f32x2{1.f, 1.f};
  e = f32x2{0.f, 0.f};
  for (int k = RUNS - 1; k >= 0; --k) {
    const f32x2 Pk = ends.P[k][lane_id()];
    e = join(Pk, ends.h[k][lane_id()], e, ends.starts[k] != 0);
    P = f32x2{P[0] * Pk[0], P[1] * Pk[1]};
  }
  const int64_t i = (int64_t)at.b * a.tiles + at.tile;
  if (at.c < a.D) {
    *reinterpret_cast<f32x2*>(a.tile_P + i * a.D + at.c) = P;
    *reinterpret_cast<f32x2*>(a.tile_h + i * a.D + at.c) = e;
  }
}

// every tile's start from the tiles' ends, in order (backwards: from the last tile on); a wave for each
// 128 channels of a row
__global__ __launch_bounds__(WAVE) void rec_join_kernel(RecLaunch a, int backwards, float* starts) {
  const int blocks = (a.D + CH - 1) / CH, b = blockIdx.x / blocks, c = (blockIdx.x - b * blocks) * CH + 2 * lane_id();
  const bool on = c < a.D;
  const int stops = backwards ? TILE_ENDS : TILE_STARTS, takes = backwards ? TILE_GOES_ON : TILE_CONTINUES;
  f32x2 h{0.f, 0.f};
  for (int64_t k = 0; k < a.tiles; ++k) {
    const int64_t i = (int64_t)b * a.tiles + (backwards ? a.tiles - 1 - k : k), o = i * a.D + c;
    const int flags = a.tile_flags[i];
    if (!(flags & takes)) h = f32x2{0.f, 0.f};
    if (on) {
      *reinterpret_cast<f32x2*>(starts + o) = h;
      h = join(*reinterpret_cast<const f32x2*>(a.tile_P + o), *reinterpret_cast<const f32x2*>(a.tile_h + o), h,
               (flags & stops) != 0);
    }
  }
}

// H from every tile's start, and the last states
template <class E, int DECAY, int NORM>
__global__ __launch_bounds__(RUNS* WAVE) void rec_out_kernel(RecLaunch a) {
  __shared__ RunEnds ends;
  const Where at(a);
  f32x2 dec[RUN], u[RUN];
  const Run r = find_run(a, at.t0, at.b);
  open_run<E, DECAY, NORM>(a, at, dec, u);
  f32x2 P{1.f, 1.f}, h{0.f, 0.f};
  auto nothing = [](int, f32x2) {};
  if (r.plain())
    walk<true>(a, at, r, dec, u, P, h, nothing);
  else
    walk<false>(a, at, r, dec, u, P, h, nothing);
  ends.P[at.wave][lane_id()] = P;
  ends.h[at.wave][lane_id()] = h;
  ends.starts[at.wave] = r.first != 0;
  __syncthreads();
  const int64_t i = (int64_t)at.b * a.tiles + at.tile;
  h = before_run(ends, at.wave, a.tiles > 1 ? state_in(a, a.states, (int)i, at.c) : f32x2{0.f, 0.f});
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    if (!(r.in >> j & 1)) continue;
    if (r.first >> j & 1) h = state_in(a, a.h0, r.seq_of(j), at.c);
    h = fma2(dec[j], h, u[j]);
    store_row<E>(a, at, a.H, j, h);
    if (r.last >> j & 1) state_out(a, a.h_out, r.seq_of(j), at.c, h);
  }
  if (a.tiles == 1 && at.wave == 0) state_out(a, a.states, (int)i, at.c, f32x2{0.f, 0.f});
  empty_sequences(a, at, a.h0, a.h_out);
}

// all gradients from every tile's start, forwards and backwards
template <class E, int DECAY, int NORM>
__global__ __launch_bounds__(RUNS* WAVE) void rec_bwd_kernel(RecLaunch a) {
  __shared__ RunEnds fwd, bwd;
  const Where at(a);
  const Run r = find_run(a, at.t0, at.b);
  typename Pair<E>::raw A[RUN], X[RUN], I[RUN], G[RUN];
  load_run<E>(a, at, a.A, a.a_stride, A);
  load_run<E>(a, at, a.X, a.x_stride, X);
  if (a.I) load_run<E>(a, at, a.I, a.i_stride, I);
  load_run<E>(a, at, a.dH, a.D, G);
  const f32x2 w = channel_w(a, at.c);
  f32x2 dec[RUN], u[RUN];
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    const f32x2 Av = Pair<E>::open(A[j]), x = Pair<E>::open(X[j]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Gate<DECAY, NORM> g(Av[k], w[k]);
      dec[j][k] = g.a;
      u[j][k] = g.b * x[k];
    }
    if (a.I) {
      const f32x2 i = Pair<E>::open(I[j]);
#pragma unroll
      for (int k = 0; k < 2; ++k) u[j][k] *= sigmoid1(i[k]);
    }
  }
  f32x2 P{1.f, 1.f}, h{0.f, 0.f}, e{0.f, 0.f};
  walk<false>(a, at, r, dec, u, P, h, [](int, f32x2) {});
  fwd.P[at.wave][lane_id()] = P;
  fwd.h[at.wave][lane_id()] = h;
  fwd.starts[at.wave] = r.first != 0;
  P = f32x2{1.f, 1.f};
#pragma unroll
  for (int j = RUN - 1; j >= 0; --j) {
    if (!(r.in >> j & 1)) continue;
    if (r.last >> j & 1) e = state_in(a, a.dh, r.seq_of(j), at.c);
    const f32x2 d = Pair<E>::open(G[j]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      e[k] = dec[j][k] * (d[k] + e[k]);
      P[k] *= dec[j][k];
    }
  }
  bwd.P[at.wave][lane_id()] = P;
  bwd.h[at.wave][lane_id()] = e;
  bwd.starts[at.wave] = r.last != 0;
  __syncthreads();
  const int64_t i = (int64_t)at.b * a.tiles + at.tile;
  h = before_run(fwd, at.wave, a.tiles > 1 ? state_in(a, a.states, (int)i, at.c) : f32x2{0.f, 0.f});
  e = a.tiles > 1 ? state_in(a, a.tile_e, (int)i, at.c) : f32x2{0.f, 0.f};
  for (int k = RUNS - 1; k > at.wave; --k)
    e = join(bwd.P[k][lane_id()], bwd.h[k][lane_id()], e, bwd.starts[k] != 0);
  f32x2 before[RUN];
  walk<false>(a, at, r, dec, u, P, h, [&](int j, f32x2 x) { before[j] = x; });
  f32x2 dw{0.f, 0.f};
#pragma unroll
  for (int j = RUN - 1; j >= 0; --j) {
    f32x2 dX{0.f, 0.f}, dA{0.f, 0.f}, dI{0.f, 0.f};
    if (r.in >> j & 1) {
      if (r.last >> j & 1) e = state_in(a, a.dh, r.seq_of(j), at.c);
      const f32x2 d = Pair<E>::open(G[j]), Av = Pair<E>::open(A[j]), x = Pair<E>::open(X[j]);
      const f32x2 iv = a.I ? Pair<E>::open(I[j]) : f32x2{0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Gate<DECAY, NORM> g(Av[k], w[k]);
        const float D = d[k] + e[k];
        e[k] = g.a * D;
        float s = 1.f, rest = 0.f;
        if (a.I) sigmoid2(iv[k], s, rest);
        const float dz = D * g.b, z = s * x[k];
        dX[k] = dz * s;
        dI[k] = dz * z * rest;
        const float dg = fmaf(e[k], before[j][k], D * z * g.db);
        dA[k] = dg * g.to_A;
        dw[k] = fmaf(-g.r, dg, dw[k]);
      }
      if (r.first >> j & 1) state_out(a, a.dh0, r.seq_of(j), at.c, e);
    }
    if (at.t0 + j < a.T) {  // rows of no sequence: zeros
      store_row<E>(a, at, a.dX, j, dX);
      store_row<E>(a, at, a.dA, j, dA);
      if (a.I) store_row<E>(a, at, a.dI, j, dI);
    }
  }
  empty_sequences(a, at, a.dh, a.dh0);
  if (DECAY != GDN_DECAY_POWER || !a.dw) return;
  __syncthreads();
  fwd.P[at.wave][lane_id()] = dw;
  __syncthreads();
  if (at.wave != 0 || at.c >= a.D) return;
  dw = f32x2{0.f, 0.f};
  for (int k = 0; k < RUNS; ++k) dw += fwd.P[k][lane_id()];
  *reinterpret_cast<f32x2*>(a.part + i * a.D + at.c) = dw;
}

// token by token, the state in registers for the whole call: a wave for each 128 channels of a
// sequence.  h_out may be h0: a lane reads and writes its own channels alone.
template <class E, int DECAY, int NORM>
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
    if (a.I) iv = Pair<E>::open(*reinterpret_cast<const raw*>(reinterpret_cast<const E*>(a.I) + row * a.i_stride + c));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Gate<DECAY, NORM> g(Av[k], w[k]);
      h[k] = fmaf(g.a, h[k], g.b * (a.I ? sigmoid1(iv[k]) : 1.f) * x[k]);
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

// ---- host side ----------------------------------------------------------------------------

namespace {

template <class F>
int by_kind(const RecLaunch& p, F&& f) {
  auto norm = [&](auto e, auto decay) {
    switch (p.norm) {
      case GDN_REC_NORM_SQRT: return f(e, decay, std::integral_constant<int, GDN_REC_NORM_SQRT>{});
      case GDN_REC_NORM_LINEAR: return f(e, decay, std::integral_constant<int, GDN_REC_NORM_LINEAR>{});
      default: return f(e, decay, std::integral_constant<int, GDN_REC_NORM_NONE>{});
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

// the workspace in order: the tiles' ends, their flags, their starts (backwards both ways), dw's parts
struct Parts {
  size_t P, h, flags, states, e, part, bytes;
  Parts(const RecLaunch& p, bool bwd) {
    const size_t n = (size_t)(rows_of(p) * p.tiles), v = up16(n * p.D * 4);
    size_t at = 0;
    auto take = [&](size_t s) {
      const size_t here = at;
      at += s;
      return here;
    };
    const bool many = p.tiles > 1;
    P = take(many ? v : 0);
    h = take(many ? v : 0);
    flags = take(many ? up16(n * 4) : 0);
    states = take(many ? v : 0);
    e = take(many && bwd ? v : 0);
    part = take(bwd && p.decay == GDN_DECAY_POWER ? v : 0);
    bytes = at;
  }
};

RecLaunch placed(const RecLaunch& p, void* workspace, bool bwd) {
  RecLaunch q = p;
  const Parts at(p, bwd);
  char* ws = reinterpret_cast<char*>(workspace);
  q.tile_P = reinterpret_cast<float*>(ws + at.P);
  q.tile_h = reinterpret_cast<float*>(ws + at.h);
  q.tile_flags = reinterpret_cast<int*>(ws + at.flags);
  if (!q.states && p.tiles > 1) q.states = reinterpret_cast<float*>(ws + at.states);
  q.tile_e = reinterpret_cast<float*>(ws + at.e);
  q.part = reinterpret_cast<float*>(ws + at.part);
  return q;
}

void copy_states(const float* from, float* to, int64_t n, hipStream_t s) {
  if (!to || n == 0) return;
  const int64_t g = (n + 255) / 256;
  hipLaunchKernelGGL(rec_copy_kernel, dim3((unsigned)(g < 1024 ? g : 1024)), dim3(256), 0, s, from, to, n);
}

template <class E, int DECAY, int NORM>
void find_states(const RecLaunch& q, dim3 grid, hipStream_t s) {
  const dim3 block(RUNS * WAVE);
  hipLaunchKernelGGL((rec_ends_kernel<E, DECAY, NORM>), grid, block, 0, s, q);
  hipLaunchKernelGGL(rec_join_kernel, dim3((unsigned)(channel_blocks(q) * rows_of(q))), dim3(WAVE), 0, s, q, 0,
                     q.states);
}

}  // namespace

size_t rec_workspace(const RecLaunch& p, bool bwd) { return p.T == 0 ? 0 : Parts(p, bwd).bytes; }

bool rec_grid_ok(const RecLaunch& p) {
  // a launch has fewer than 2^32 threads
  return p.tiles <= (((int64_t)1 << 32) - 1) / (RUNS * WAVE) / channel_blocks(p) / (rows_of(p) > 0 ? rows_of(p) : 1);
}
bool rec_step_grid_ok(const RecLaunch& p) { return p.n_seq <= (((int64_t)1 << 32) - 256) / WAVE / channel_blocks(p); }

int launch_rec_fwd(const RecLaunch& p, void* workspace, hipStream_t s) {
  if (p.T == 0) {
    copy_states(p.h0, p.h_out, (int64_t)p.n_seq * p.D, s);
    return 0;
  }
  const RecLaunch q = placed(p, workspace, false);
  const dim3 grid((unsigned)(q.tiles * rows_of(q) * channel_blocks(q))), block(RUNS * WAVE);
  return by_kind(p, [&](auto e, auto decay, auto norm) {
    typedef std::remove_pointer_t<decltype(e)> E;
    if (q.tiles > 1) find_states<E, decay.value, norm.value>(q, grid, s);
    hipLaunchKernelGGL((rec_out_kernel<E, decay.value, norm.value>), grid, block, 0, s, q);
    return 0;
  });
}

int launch_rec_bwd(const RecLaunch& p, void* workspace, hipStream_t s) {
  if (p.T == 0 || rows_of(p) == 0) {
    copy_states(p.dh, p.dh0, (int64_t)p.n_seq * p.D, s);
    copy_states(nullptr, p.dw, p.D, s);
    return 0;
  }
  const RecLaunch q = placed(p, workspace, true);
  const dim3 grid((unsigned)(q.tiles * rows_of(q) * channel_blocks(q))), block(RUNS * WAVE);
  return by_kind(p, [&](auto e, auto decay, auto norm) {
    typedef std::remove_pointer_t<decltype(e)> E;
    if (q.tiles > 1) {
      find_states<E, decay.value, norm.value>(q, grid, s);
      hipLaunchKernelGGL((rec_ends_bwd_kernel<E, decay.value, norm.value>), grid, block, 0, s, q);
      hipLaunchKernelGGL(rec_join_kernel, dim3((unsigned)(channel_blocks(q) * rows_of(q))), dim3(WAVE), 0, s, q,
                         1, q.tile_e);
    }
    hipLaunchKernelGGL((rec_bwd_kernel<E, decay.value, norm.value>), grid, block, 0, s, q);
    if (q.dw) launch_column_sum(q.part, q.tiles * rows_of(q), q.D, 1, q.dw, nullptr, s);
    return 0;
  });
}

int launch_rec_step(const RecLaunch& p, hipStream_t s) {
  const int64_t waves = (int64_t)p.n_seq * channel_blocks(p);
  const dim3 grid((unsigned)((waves + 3) / 4)), block(256);
  return by_kind(p, [&](auto e, auto decay, auto norm) {
    hipLaunchKernelGGL((rec_step_kernel<std::remove_pointer_t<decltype(e)>, decay.value, norm.value>), grid, block, 0, s, p);
    return 0;
  });
}

}  // namespace gdn
