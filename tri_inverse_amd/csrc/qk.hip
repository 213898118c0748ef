// qk.hip -- the norm of queries and keys for each head, with the position rotation in the same pass,
// from the projection's rows [B][T][heads][d] to the head-major [B][H][T][d] of the mixers.
//
//   y = R(p) (n * w),  n = x * rstd,  rstd = (inv sum x^2 + eps)^-1/2,  inv = 1/d (RMS) or 1 (unit rows)
// Backwards, with dn = R(-p) dy and u = dn * w:
//   dw = sum_rows dn * n,   dx = rstd (u - n inv sum(u n))
// R(p) turns pair i by p f_i: the turns p f_i / 2 pi are formed in fp64 and only what they leave of
// a quarter is rounded to fp32, so an angle is right to 2^-24 of a quarter turn at any position.
//
// Bound by bytes: each row is read once into registers and its result written.  A lane holds four
// pairs of a row whole (two runs of 4 values, r/2 apart or next to each other), so that no value
// crosses lanes but for the row's sum, and keeps its angles' cosines and sines for all heads of
// its token that its workgroup takes.  Lanes of a wave take neighbouring tokens: what they write of a head is
// contiguous.  Gradients of the weights as in norm.hip: partial rows by workgroup, added in order.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

__device__ __forceinline__ void load4(const __bf16* p, float* x) {
  const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = (float)v[e];
}
__device__ __forceinline__ void load4(const float* p, float* x) {
  const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = v[e];
}
__device__ __forceinline__ void store4(__bf16* p, const float* x) {
  *reinterpret_cast<bf16x4*>(p) = pack4(f32x4{x[0], x[1], x[2], x[3]});
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
}

// sum over aligned groups of LPR lanes, in every lane of the group
template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
  x += dpp_f<0xB1>(x);  // quad_perm 1,0,3,2
  x += dpp_f<0x4E>(x);  // quad_perm 2,3,0,1
  if constexpr (LPR >= 8) x += dpp_f<0x141>(x);  // row_half_mirror
  if constexpr (LPR >= 16) x += dpp_f<0x140>(x);  // row_mirror
  if constexpr (LPR >= 32) {
    float a, b;
    self_swap_f<16>(x, a, b);
    x = a + b;
  }
  return x;
}

// cosine and sine of `turns` whole turns: to the nearest quarter in fp64, the rest (at most an eighth)
// by the series, whose first terms left out are below 2^-28
__device__ __forceinline__ void cos_sin(double turns, float& c, float& s) {
  turns -= rint(turns);
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

// a lane's place in a row: two runs of 4 values, and whether they are its pairs
struct Place {
  int at0, at1, pair;
  bool on, turns;
};
template <bool HALVES>
__device__ __forceinline__ Place place(const QkLaunch& a, int lane) {
  Place p;
  p.on = 8 * lane < a.d;
  p.turns = 8 * lane < a.rot;
  p.pair = 4 * lane;
  p.at0 = HALVES && p.turns ? 4 * lane : 8 * lane;
  p.at1 = HALVES && p.turns ? a.rot / 2 + 4 * lane : 8 * lane + 4;
  return p;
}

struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn turn_of(const QkLaunch& a, const Place& p, uint32_t token, uint32_t tokens, uint32_t t) {
  Turn r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.c[i] = 1.f;
    r.s[i] = 0.f;
  }
  if (p.on && p.turns)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double pos =
          a.positions ? (double)a.positions[(int64_t)a.axis[p.pair + i] * tokens + token] : (double)t;
      cos_sin(pos * (a.freqs[p.pair + i] * 0.15915494309189535), r.c[i], r.s[i]);
    }
  return r;
}
// pairs in a lane: (x[i], x[4 + i]), or (x[2 i], x[2 i + 1])
template <bool HALVES>
__device__ __forceinline__ void turn(float (&x)[8], const Turn& r, float sign) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = HALVES ? i : 2 * i, q = HALVES ? 4 + i : 2 * i + 1;
    const float s = sign * r.s[i], u = x[p], v = x[q];
    x[p] = u * r.c[i] - v * s;
    x[q] = v * r.c[i] + u * s;
  }
}

template <class E>
__device__ __forceinline__ void load_row(const E* p, const Place& at, bool on, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
  if (on) {
    load4(p + at.at0, x);
    load4(p + at.at1, x + 4);
  }
}
template <class E>
__device__ __forceinline__ void store_row(E* p, const Place& at, bool on, const float (&x)[8]) {
  if (on) {
    store4(p + at.at0, x);
    store4(p + at.at1, x + 4);
  }
}
__device__ __forceinline__ void load_weights(const float* w, const Place& at, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 1.f;
  if (w && at.on) {
    load4(w + at.at0, x);
    load4(w + at.at1, x + 4);
  }
}

// 1 / n(x) of a row; 1 without a norm
template <int LPR>
__device__ __forceinline__ float row_rstd(const QkLaunch& a, const float (&x)[8]) {
  if (a.norm == GDN_QK_NONE) return 1.f;
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  ss = lanes_sum<LPR>(ss);
  return 1.f / sqrtf((a.norm == GDN_QK_RMS ? ss / (float)a.d : ss) + a.eps);
}

}  // namespace

// workgroup: 256 / LPR tokens, `per` heads of queries and keys from blockIdx.y * per on
template <int LPR, class E, bool HALVES>
__global__ __launch_bounds__(256) void qk_kernel(QkLaunch a, int per) {
  const Place at = place<HALVES>(a, threadIdx.x % LPR);
  const uint32_t tokens = (uint32_t)(a.B * a.T);
  const uint32_t token = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const bool on = token < tokens && at.on;
  const uint32_t b = token / (uint32_t)a.T, t = token - b * (uint32_t)a.T;
  Turn r{};
  if (token < tokens) r = turn_of(a, at, token, tokens, t);
  const int first = blockIdx.y * per, last = min(first + per, a.Hq + a.Hk);
  auto heads = [&](int h0, int h1, int H, const void* in, int64_t stride, const float* weights, void* out) {
    if (h0 >= h1) return;
    float w[8];
    load_weights(weights, at, w);
    const E* src = reinterpret_cast<const E*>(in) + (int64_t)token * stride;
    E* dst = reinterpret_cast<E*>(out) + ((int64_t)b * H * a.T + t) * a.d;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      float x[8];
      load_row(src + (int64_t)h * a.d, at, on, x);
      const float rstd = row_rstd<LPR>(a, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= rstd * w[e];
      turn<HALVES>(x, r, 1.f);
      store_row(dst + (int64_t)h * a.T * a.d, at, on, x);
    }
  };
  heads(first, min(last, a.Hq), a.Hq, a.Q_in, a.q_stride, a.wq, a.Q);
  heads(max(first - a.Hq, 0), last - a.Hq, a.Hk, a.K_in, a.k_stride, a.wk, a.K);
}

// workgroups walk pieces of work: groups of tokens, and runs of `per` heads
template <int LPR, class E, bool HALVES>
__global__ __launch_bounds__(256) void qk_bwd_kernel(QkLaunch a, int per, uint32_t runs, uint32_t pieces, float* part) {
  __shared__ float sums[256 / LPR][8 * LPR];
  const Place at = place<HALVES>(a, threadIdx.x % LPR);
  const uint32_t tokens = (uint32_t)(a.B * a.T);
  float w[2][8], dw[2][8];
  load_weights(a.wq, at, w[0]);
  load_weights(a.wk, at, w[1]);
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
  for (uint32_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
    const uint32_t group = piece / runs, token = group * (256 / LPR) + threadIdx.x / LPR;
    const int first = (int)(piece - group * runs) * per, last = min(first + per, a.Hq + a.Hk);
    const bool row = token < tokens, on = row && at.on;
    const uint32_t b = token / (uint32_t)a.T, t = token - b * (uint32_t)a.T;
    Turn r{};
    if (row) r = turn_of(a, at, token, tokens, t);
    auto heads = [&](auto which, int h0, int h1, int H, const void* in, int64_t stride, const void* dy, void* dx) {
      constexpr int W = which.value;
      const E* src = reinterpret_cast<const E*>(in) + (int64_t)token * stride;
      const E* grad = reinterpret_cast<const E*>(dy) + ((int64_t)b * H * a.T + t) * a.d;
      E* dst = reinterpret_cast<E*>(dx) + (int64_t)token * H * a.d;
#pragma unroll 2
      for (int h = h0; h < h1; ++h) {
        float x[8], g[8];
        load_row(src + (int64_t)h * a.d, at, on, x);
        load_row(grad + (int64_t)h * a.T * a.d, at, on, g);
        // past the last token the norm of zeros would be infinite where eps is 0, and dw not a number
        const float rstd = row ? row_rstd<LPR>(a, x) : 0.f;
        turn<HALVES>(g, r, -1.f);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= rstd;
          dw[W][e] = fmaf(g[e], x[e], dw[W][e]);
          g[e] *= w[W][e];
          dot = fmaf(g[e], x[e], dot);
        }
        dot = a.norm == GDN_QK_NONE ? 0.f : lanes_sum<LPR>(dot);
        if (a.norm == GDN_QK_RMS) dot /= (float)a.d;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = rstd * (g[e] - x[e] * dot);
        store_row(dst + (int64_t)h * a.d, at, on, x);
      }
    };
    heads(std::integral_constant<int, 0>{}, first, min(last, a.Hq), a.Hq, a.Q_in, a.q_stride, a.dQ, a.Q);
    heads(std::integral_constant<int, 1>{}, max(first - a.Hq, 0), last - a.Hq, a.Hk, a.K_in, a.k_stride, a.dK, a.K);
  }
  if (!part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at.on) sums[threadIdx.x / LPR][(e < 4 ? at.at0 : at.at1 - 4) + e] = dw[which][e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += 256) {
      float s = 0.f;
      for (int k = 0; k < 256 / LPR; ++k) s += sums[k][i];
      part[((int64_t)blockIdx.x * 2 + which) * a.d + i] = s;
    }
  }
}

// ---- host side ----------------------------------------------------------------------------

namespace {

int row_lanes(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

template <class F>
int by_kind(const QkLaunch& p, F&& f) {
  auto pairs = [&](auto lpr, auto e) {
    return p.halves ? f(lpr, e, std::integral_constant<bool, true>{}) : f(lpr, e, std::integral_constant<bool, false>{});
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
int64_t bwd_groups(const QkLaunch& p) {
  const int64_t n = token_groups(p) * head_runs(p);
  return n < 1024 ? n : 1024;
}

}  // namespace

size_t qk_bwd_workspace(const QkLaunch& p) { return (size_t)bwd_groups(p) * 2 * p.d * 4; }

int launch_qk(const QkLaunch& p, hipStream_t s) {
  return by_kind(p, [&](auto lpr, auto e, auto halves) {
    const dim3 grid((unsigned)token_groups(p), (unsigned)head_runs(p)), block(256);
    hipLaunchKernelGGL((qk_kernel<lpr.value, std::remove_pointer_t<decltype(e)>, halves.value>), grid, block, 0, s, p,
                       heads_per_group(p));
    return 0;
  });
}

int launch_qk_bwd(const QkLaunch& p, void* workspace, hipStream_t s) {
  float* part = p.dwq || p.dwk ? reinterpret_cast<float*>(workspace) : nullptr;
  const bool rows = (int64_t)p.B * p.T > 0 && p.Hq + p.Hk > 0;
  const int64_t n = rows ? bwd_groups(p) : 0;
  if (rows)
    by_kind(p, [&](auto lpr, auto e, auto halves) {
      const dim3 grid((unsigned)n), block(256);
      const int runs = head_runs(p);
      hipLaunchKernelGGL((qk_bwd_kernel<lpr.value, std::remove_pointer_t<decltype(e)>, halves.value>), grid, block, 0, s,
                         p, heads_per_group(p), (uint32_t)runs, (uint32_t)(token_groups(p) * runs), part);
      return 0;
    });
  if (p.dwq || p.dwk) launch_column_sum(part, n, p.d, 2, p.dwq, p.dwk, s);  // no rows: zeros
  return 0;
}

}  // namespace gdn
