// qk.hip -- the norm of queries and keys for each head, with the position rotation in the same pass,
// from the projection's rows [B][T][heads][d] to the head-major [B][H][T][d] of the mixers.
//
//   y = R(p) (n * w),  n = x * rstd,  rstd = (inv sum x^2 + eps)^-1/2,  inv = 1/d (RMS) or 1 (unit rows)
// Backwards, with dn = R(-p) dy and u = dn * w:
//   dw = sum_rows dn * n,   dx = rstd (u - n inv sum(u n))
// R(p) turns pair i by p f_i: the turns p f_i / 2 pi are formed in fp64 with their remainders and only what they
// leave of a quarter is rounded to fp32, so an angle is right to 2^-24 of a quarter turn at any position.
//
// Bound by bytes: each row is read once into registers and its result written, and a lane keeps its
// angles' cosines and sines for all heads of its token that its workgroup takes; the next heads' rows are
// on their way while it forms the last ones' results.  A lane's pairs are its own, so no value crosses
// lanes but for the row's sum.  Lanes of a wave take neighbouring tokens: what they write of a head is
// contiguous.  Gradients of the weights as in norm.hip: partial rows by workgroup, added in order.
//
// Measured (a copy of 1 GiB reaches 5.05 TB/s): 4 x 8192 tokens, 16 and 16 heads of 128, bf16, all turned, 537
// MB, 100 us, 5.4 TB/s (115 with every head's loads behind the last one's results; 145 with 16-byte
// accesses and the pairs' other halves loaded too, 116 with them exchanged between lanes).  Backwards, 4
// x 4096 tokens, 403 MB, 91 us, 4.4 TB/s, of which the kernel 87, 4.6 TB/s, the column sum 4.6.  64 tokens of 32 and 16 heads, 64 of 128
// values turned: 3.5 us, latency.
#include <algorithm>

#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

// cosine and sine of the angle pos freq.  1 / 2 pi in two parts and the remainders of the products keep what rounding
// takes from far turns (without them 4.8 x 2^-24 of a quarter turn at 2^31); to the nearest quarter in fp64, the rest (at
// most an eighth) by the series, whose first terms left out are below 2^-28
__device__ __forceinline__ void cos_sin(double pos, double freq, float& c, float& s) {
#pragma clang fp contract(off)  // the remainders are those of the products as rounded
  constexpr double INV = 0x1.45f306dc9c883p-3, INV_REST = -0x1.6b01ec5417056p-57;
  const double angle = pos * freq;
  double turns = angle * INV;
  const double rest = fma(fma(pos, freq, -angle), INV, fma(angle, INV_REST, fma(angle, INV, -turns)));
  turns = (turns - rint(turns)) + rest;
  turns -= rint(turns);  // past 2^52 turns the rest is more than one
  const double quarter = rint(4.0 * turns);
  const float x = (float)(fma(-0.25, quarter, turns) * 6.283185307179586);
  const float x2 = x * x;
  float p = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  p = fmaf(x2, p, 1.f / 120.f);
  p = fmaf(x2, p, -1.f / 6.f);
  const float sn = fmaf(x * x2, p, x);
  float q = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
  q = fmaf(x2, q, -1.f / 720.f);
  q = fmaf(x2, q, 1.f / 24.f);
  const float cs = fmaf(x2 * x2, q, fmaf(x2, -0.5f, 1.f));
  const int k = (int)quarter & 3;
  c = k & 1 ? sn : cs;
  s = k & 1 ? cs : sn;
  if (k == 1 || k == 2) c = -c;
  if (k >= 2) s = -s;
}

// a lane's place in a row, two runs of 4 values.  HALVES: its pairs are (run 0, run 1) value by value, the runs
// half the rotated part apart, half the rest for the lanes behind it.  Otherwise pairs are neighbours in
// a run: 8 neighbouring bf16 values, or fp32 runs half the row apart, so that lanes' runs lie next to each other.
template <class E, bool HALVES>
struct Place {
  static constexpr bool WIDE = sizeof(E) == 2 && !HALVES;
  int at[2];
  bool on;
  __device__ __forceinline__ Place(const QkLaunch& a, int lane) {
    on = 8 * lane < a.d;
    if (!on) lane = 0;  // loads what lies inside
    if constexpr (WIDE) {
      at[0] = 8 * lane;
      at[1] = 8 * lane + 4;
    } else {
      const bool in = !HALVES || 8 * lane < a.rot;
      const int first = in ? 0 : a.rot, width = !HALVES ? a.d : in ? a.rot : a.d - a.rot;
      at[0] = first + 4 * (lane - first / 8);
      at[1] = at[0] + width / 2;
    }
  }
};

// cosines and sines of a lane's four pairs
struct Turn {
  float c[4], s[4];
  // SPARE: one pair after the other, which takes fewer registers from the rows on their way
  template <bool HALVES, bool SPARE, class P>
  __device__ __forceinline__ void find(const QkLaunch& a, const P& p, uint32_t token, uint32_t tokens, uint32_t t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = HALVES ? p.at[0] + i : p.at[i / 2] + 2 * (i % 2);  // the pair's first value
      c[i] = 1.f;
      s[i] = 0.f;
      if (v < a.rot) {
        const int pair = HALVES ? v : v / 2;
        const double pos = a.positions ? (double)a.positions[(int64_t)a.axis[pair] * tokens + token] : (double)t;
        cos_sin(pos, a.freqs[pair], c[i], s[i]);
      }
      if constexpr (SPARE) __builtin_amdgcn_sched_barrier(0);
    }
  }
  template <bool HALVES, bool BACK>
  __device__ __forceinline__ void turn(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = HALVES ? i : 2 * i, n = HALVES ? 4 + i : 2 * i + 1;
      const float sn = BACK ? -s[i] : s[i], u = x[m], v = x[n];
      x[m] = u * c[i] - v * sn;
      x[n] = v * c[i] + u * sn;
    }
  }
};

// a lane's values of a row as they lie in memory
template <class E>
struct Row;
template <>
struct Row<__bf16> {
  u32x2 run[2];
  template <bool WIDE>
  __device__ __forceinline__ void load(const __bf16* p, const int (&at)[2]) {
    if constexpr (WIDE) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p + at[0]);
      run[0] = u32x2{v[0], v[1]};
      run[1] = u32x2{v[2], v[3]};
    } else {
      run[0] = *reinterpret_cast<const u32x2*>(p + at[0]);
      run[1] = *reinterpret_cast<const u32x2*>(p + at[1]);
    }
  }
  __device__ __forceinline__ void open(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x2 w = run[i];
      const f32x4 v = unpack4(__builtin_bit_cast(bf16x4, w));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
    }
  }
};
template <>
struct Row<float> {
  f32x4 run[2];
  template <bool WIDE>
  __device__ __forceinline__ void load(const float* p, const int (&at)[2]) {
    run[0] = *reinterpret_cast<const f32x4*>(p + at[0]);
    run[1] = *reinterpret_cast<const f32x4*>(p + at[1]);
  }
  __device__ __forceinline__ void open(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = run[i][e];
  }
};
// NT: stores of whole lines, past what the caches hold
template <bool NT, class E, class P>
__device__ __forceinline__ void store_row(E* p, const P& at, const float (&x)[8]) {
  const f32x4 lo{x[0], x[1], x[2], x[3]}, hi{x[4], x[5], x[6], x[7]};
  if constexpr (P::WIDE) {
    store16<NT>(reinterpret_cast<u32x4*>(p + at.at[0]), __builtin_bit_cast(u32x4, pack8(lo, hi)));
  } else if constexpr (sizeof(E) == 2) {
    store16<NT>(reinterpret_cast<u32x2*>(p + at.at[0]), __builtin_bit_cast(u32x2, pack4(lo)));
    store16<NT>(reinterpret_cast<u32x2*>(p + at.at[1]), __builtin_bit_cast(u32x2, pack4(hi)));
  } else {
    store16<NT>(reinterpret_cast<f32x4*>(p + at.at[0]), lo);
    store16<NT>(reinterpret_cast<f32x4*>(p + at.at[1]), hi);
  }
}
__device__ __forceinline__ void load_weights(const float* w, const int (&at)[2], float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = w ? w[at[e / 4] + e % 4] : 1.f;
}

// 1 / n(x) of a row; 1 without a norm
template <int LPR>
__device__ __forceinline__ float row_rstd(const QkLaunch& a, const float (&x)[8], bool on) {
  if (a.norm == GDN_QK_NONE) return 1.f;
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  ss = group_sum<LPR>(on ? ss : 0.f);
  return 1.f / sqrtf((a.norm == GDN_QK_RMS ? ss / (float)a.d : ss) + a.eps);
}

}  // namespace

// a row's token and place; a token past the last one stands for the last one, whose row it loads
struct Token {
  uint32_t token, b, t;
  bool on;
  __device__ __forceinline__ Token(const QkLaunch& a, uint32_t at, uint32_t tokens) {
    on = at < tokens;
    token = on ? at : tokens - 1;
    b = token / (uint32_t)a.T;
    t = token - b * (uint32_t)a.T;
  }
};

// workgroup: 256 / LPR tokens, `per` heads of queries and keys from blockIdx.y * per on
template <int LPR, class E, bool HALVES, bool NT>
__global__ __launch_bounds__(256) void qk_kernel(QkLaunch a, int per) {
  typedef Place<E, HALVES> P;
  constexpr int U = sizeof(E) == 2 ? 4 : 2;  // heads at a time
  const P at(a, threadIdx.x % LPR);
  const uint32_t tokens = (uint32_t)(a.B * a.T);
  const Token k(a, blockIdx.x * (256 / LPR) + threadIdx.x / LPR, tokens);
  const int first = blockIdx.y * per, last = min(first + per, a.Hq + a.Hk);
  Turn angle;
  bool found = false;
  auto heads = [&](int h0, int h1, int H, const void* in, int64_t stride, const float* weights, void* out) {
    if (h0 >= h1) return;
    const E* src = reinterpret_cast<const E*>(in) + (int64_t)k.token * stride;
    E* dst = reinterpret_cast<E*>(out) + ((int64_t)k.b * H * a.T + k.t) * a.d;
    Row<E> row[U];
    auto load = [&](int h) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        row[u].template load<P::WIDE>(src + (int64_t)min(h + u, h1 - 1) * a.d, at.at);
    };
    load(h0);
    float w[8];
    load_weights(weights, at.at, w);
    if (!found) angle.template find<HALVES, false>(a, at, k.token, tokens, k.t);
    found = true;
    for (int h = h0; h < h1; h += U) {
      Row<E> now[U];
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = row[u];
      if (h + U < h1) load(h + U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= h1) break;
        float x[8];
        now[u].open(x);
        const float rstd = row_rstd<LPR>(a, x, at.on);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= rstd * w[e];
        angle.template turn<HALVES, false>(x);
        if (k.on && at.on) store_row<NT>(dst + (int64_t)(h + u) * a.T * a.d, at, x);
      }
    }
  };
  heads(first, min(last, a.Hq), a.Hq, a.Q_in, a.q_stride, a.wq, a.Q);
  heads(max(first - a.Hq, 0), last - a.Hq, a.Hk, a.K_in, a.k_stride, a.wk, a.K);
}

// workgroups walk pieces of work: groups of tokens, and runs of `per` heads
template <int LPR, class E, bool HALVES, bool NT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4, 4))) void qk_bwd_kernel(QkLaunch a, int per, uint32_t runs, uint32_t pieces, float* part) {
  typedef Place<E, HALVES> P;
  constexpr int U = 1;
  __shared__ float sums[256 / LPR][8 * LPR];
  const P at(a, threadIdx.x % LPR);
  const uint32_t tokens = (uint32_t)(a.B * a.T);
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
  for (uint32_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
    const uint32_t group = piece / runs;
    const Token k(a, group * (256 / LPR) + threadIdx.x / LPR, tokens);
    const int first = (int)(piece - group * runs) * per, last = min(first + per, a.Hq + a.Hk);
    Turn angle;
    bool found = false;
    auto heads = [&](auto which, int h0, int h1, int H, const void* in, int64_t stride, const float* weights,
                     const void* dy, void* dx) {
      constexpr int W = which.value;
      if (h0 >= h1) return;
      const E* src = reinterpret_cast<const E*>(in) + (int64_t)k.token * stride;
      const E* grad = reinterpret_cast<const E*>(dy) + ((int64_t)k.b * H * a.T + k.t) * a.d;
      E* dst = reinterpret_cast<E*>(dx) + (int64_t)k.token * H * a.d;
      Row<E> rx[U], rg[U];
      auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t i = min(h + u, h1 - 1);
          rx[u].template load<P::WIDE>(src + i * a.d, at.at);
          rg[u].template load<P::WIDE>(grad + i * a.T * a.d, at.at);
        }
      };
      load(h0);
      float w[8];
      load_weights(weights, at.at, w);
      if (!found) angle.template find<HALVES, true>(a, at, k.token, tokens, k.t);
      found = true;
      for (int h = h0; h < h1; h += U) {
        Row<E> nx[U], ng[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          nx[u] = rx[u];
          ng[u] = rg[u];
        }
        if (h + U < h1) load(h + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h + u >= h1) break;
          float x[8], g[8];
          nx[u].open(x);
          ng[u].open(g);
          // a token past the last one adds nothing to dw
          const float size = row_rstd<LPR>(a, x, at.on), rstd = k.on ? size : 0.f;
          angle.template turn<HALVES, true>(g);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] *= rstd;
            dw[W][e] = fmaf(g[e], x[e], dw[W][e]);
            g[e] *= w[e];
            dot = fmaf(g[e], x[e], dot);
          }
          dot = a.norm == GDN_QK_NONE ? 0.f : group_sum<LPR>(at.on ? dot : 0.f);
          if (a.norm == GDN_QK_RMS) dot /= (float)a.d;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = rstd * (g[e] - x[e] * dot);
          if (k.on && at.on) store_row<NT>(dst + (int64_t)(h + u) * a.d, at, x);
        }
      }
    };
    heads(std::integral_constant<int, 0>{}, first, min(last, a.Hq), a.Hq, a.Q_in, a.q_stride, a.wq, a.dQ, a.Q);
    heads(std::integral_constant<int, 1>{}, max(first - a.Hq, 0), last - a.Hq, a.Hk, a.K_in, a.k_stride, a.wk, a.dK, a.K);
  }
  if (!part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at.on) sums[threadIdx.x / LPR][at.at[e / 4] + e % 4] = dw[which][e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += 256) {
      double s = 0.0;
      for (int k = 0; k < 256 / LPR; ++k) s += (double)sums[k][i];
      part[((int64_t)blockIdx.x * 2 + which) * a.d + i] = (float)s;
    }
  }
}

// ---- host side ----------------------------------------------------------------------------

namespace {

int row_lanes(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// Whether stores cover whole lines of 128 bytes; they then go past what the caches hold.  Of parts of
// lines that costs more than it gives (4 x 8192 tokens of 32 heads of 128 bf16 values, 8 of them
// turned: 129 us instead of 110; all turned: 100 instead of 105).  Rows of neighbouring bf16 values count from a
// line's length on, wherever they start (4 x 8191 tokens of 32 heads of 96: 80 us instead of 84; 64 heads of 32, half a
// line: 58 instead of 50).
bool whole_lines(const QkLaunch& p) {
  const int size = p.bf16 ? 2 : 4;
  if (!p.halves) return p.bf16 ? p.d >= 64 : p.d / 2 * size % 128 == 0;
  return p.rot / 2 * size % 128 == 0 && (p.d - p.rot) / 2 * size % 128 == 0;
}

template <class F>
int by_kind(const QkLaunch& p, F&& f) {
  auto lines = [&](auto lpr, auto e, auto halves) {
    return whole_lines(p) ? f(lpr, e, halves, std::true_type{}) : f(lpr, e, halves, std::false_type{});
  };
  auto pairs = [&](auto lpr, auto e) {
    return p.halves ? lines(lpr, e, std::true_type{}) : lines(lpr, e, std::false_type{});
  };
  auto type = [&](auto lpr) { return p.bf16 ? pairs(lpr, (__bf16*)nullptr) : pairs(lpr, (float*)nullptr); };
  switch (row_lanes(p.d)) {
    case 4: return type(std::integral_constant<int, 4>{});
    case 8: return type(std::integral_constant<int, 8>{});
    case 16: return type(std::integral_constant<int, 16>{});
    default: return type(std::integral_constant<int, 32>{});
  }
}

int64_t token_groups(const QkLaunch& p) {
  const int per = 256 / row_lanes(p.d);
  return ((int64_t)p.B * p.T + per - 1) / per;
}
// heads of a workgroup: all of a token's where the tokens alone make four workgroups for each CU,
// fewer where they do not (the angles are then formed by more than one)
int heads_per_group(const QkLaunch& p) {
  const int64_t heads = p.Hq + p.Hk, groups = token_groups(p), runs = (1024 + groups - 1) / groups;
  return (int)((heads + (runs < heads ? runs : heads) - 1) / (runs < heads ? runs : heads));
}
int head_runs(const QkLaunch& p) {
  const int per = heads_per_group(p);
  return (p.Hq + p.Hk + per - 1) / per;
}
// Backwards a lane adds at most 64 rows to each of its sums for a weight, in 32 bits; the sums go on in 64.  So a piece of
// work has at most 64 heads, and there are more workgroups than 1024 where those would walk over more rows (16 x 8192
// tokens of 16 and 16 heads of 128: 2048 workgroups, 642 us; 1024 of them, 128 rows to a sum, 635).
constexpr int MOST_ROWS = 64;
struct BwdWork {
  int per, runs;
  int64_t pieces, groups;
  BwdWork(const QkLaunch& p) {
    per = std::min(heads_per_group(p), MOST_ROWS);
    runs = (p.Hq + p.Hk + per - 1) / per;
    pieces = token_groups(p) * runs;
    const int rows = std::min(per, std::max(p.Hq, p.Hk)), walk = MOST_ROWS / rows;  // of a piece; pieces in a row
    groups = std::max(std::min<int64_t>(pieces, 1024), (pieces + walk - 1) / walk);
  }
};

}  // namespace

size_t qk_bwd_workspace(const QkLaunch& p) { return (size_t)BwdWork(p).groups * 2 * p.d * 4; }

int launch_qk(const QkLaunch& p, hipStream_t s) {
  return by_kind(p, [&](auto lpr, auto e, auto halves, auto nt) {
    const dim3 grid((unsigned)token_groups(p), (unsigned)head_runs(p)), block(256);
    hipLaunchKernelGGL((qk_kernel<lpr.value, std::remove_pointer_t<decltype(e)>, halves.value, nt.value>), grid, block, 0, s, p,
                       heads_per_group(p));
    return 0;
  });
}

int launch_qk_bwd(const QkLaunch& p, void* workspace, hipStream_t s) {
  float* part = p.dwq || p.dwk ? reinterpret_cast<float*>(workspace) : nullptr;
  const bool rows = (int64_t)p.B * p.T > 0 && p.Hq + p.Hk > 0;
  int64_t n = 0;
  if (rows)
    by_kind(p, [&](auto lpr, auto e, auto halves, auto nt) {
      const BwdWork w(p);
      n = w.groups;
      const dim3 grid((unsigned)n), block(256);
      typedef std::remove_pointer_t<decltype(e)> E;
      // stores past the caches pay for fp32 (2 x 4096 tokens of 32 heads of 128: 84 us, through them 89), not for
      // bf16 (4 x 4096 tokens: 94.4, through them 90.9)
      constexpr bool past = nt.value && sizeof(E) == 4;
      hipLaunchKernelGGL((qk_bwd_kernel<lpr.value, E, halves.value, past>), grid, block, 0, s,
                         p, w.per, (uint32_t)w.runs, (uint32_t)w.pieces, part);
      return 0;
    });
  if (p.dwq || p.dwk) launch_column_sum(part, n, p.d, 2, p.dwq, p.dwk, s);  // no rows: zeros
  return 0;
}

}  // namespace gdn
