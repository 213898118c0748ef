// norm.hip -- the norms around the token mixer, fused with its gate and its residual scale.
//
// Gated norm of the head outputs (rows of d, one per token and head):
//   y = n * w * act(z),  n = o * rstd,  rstd = (mean(o^2) + eps)^-1/2
//   dz = dy * n * w * act'(z);  with u = dy * act(z):  dw = sum_rows u * n,
//   do = rstd (u w - n mean(u w n))
// Residual norm (rows of D, one per token; every factor but alpha may be absent):
//   r = x + alpha s * (rms(y) * w_post),   n = rms(r) * w_pre
//   dr' = dr + rms'(dn; r, w_pre),  dx = dr',  dy = rms'(alpha s dr'; y, w_post),
//   and with p = sum_rows alpha dr' * y / sqrt(mean(y^2) + eps):  ds = p w_post, dw_post = p s
//
// All of it is bound by bytes: each row is read once into registers, the sums over it are
// formed there and its results written, with 16-byte accesses.  Sums and norms are fp32; each
// output is rounded once.  Gradients of the weights are sums over rows: every workgroup walks
// a fixed set of rows with its column sums in registers and writes one partial row, and a
// second kernel adds the partial rows in order (no atomics: the same call gives the same bits).
//
// Measured (a copy of 1 GiB reaches 5.2 TB/s): gated norm B4 H16 T8192 d128 bf16, 403 MB, 74 us,
// 5.4 TB/s (its vector instructions, the exponentials mostly, take as long); backward B3 H16
// T4099, 252 MB, 57 us, 4.4 TB/s, of which the column sum 4.7; residual norm backward, 16384 rows of 4096,
// fp32 and bf16, 1208 MB, 226 us, 5.4 TB/s; forward, 64 rows of 2048, 3.4 us, latency.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

// 8 consecutive elements as fp32
__device__ __forceinline__ void load8(const __bf16* p, float (&x)[8]) {
  const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a[e];
    x[4 + e] = b[e];
  }
}
__device__ __forceinline__ void store8(__bf16* p, const float (&x)[8]) {
  *reinterpret_cast<bf16x8*>(p) = pack8(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void fill8(float (&x)[8], float v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = v;
}

// act(z) and its derivative; 1 / (1 + e^-z) is 0 or 1 where e^-z overflows or vanishes.  What it
// leaves of 1 is e^-z times itself for z >= 0, where the difference would cancel (17 % of the
// sigmoid's derivative at z = 15, all of it from 17 on)
__device__ __forceinline__ void gate(int act, float z, float& f, float& df) {
  const float ez = __expf(-z), sg = 1.f / (1.f + ez), rest = z < 0.f ? 1.f - sg : ez * sg;
  if (act == GDN_GATE_SILU) {
    f = z * sg;
    df = sg * fmaf(z, rest, 1.f);
  } else {
    f = sg;
    df = sg * rest;
  }
}

// rows are taken token by token, head by head: row r of Y, of Z's token r / H, head r % H
__device__ __forceinline__ void gate_row(const GateNormLaunch& a, uint32_t r, int64_t& o, int64_t& z) {
  const uint32_t H = a.H, T = (uint32_t)a.T;
  const uint32_t tok = r / H, h = r - tok * H, b = tok / T, t = tok - b * T;
  o = ((int64_t)(b * H + h) * a.T + t) * a.d;
  z = (int64_t)tok * a.z_stride + (int64_t)h * a.d;
}

}  // namespace

template <int LPR, class E>
__global__ __launch_bounds__(256) void gate_norm_kernel(GateNormLaunch a, uint32_t rows) {
  const int col = 8 * (threadIdx.x % LPR);
  const uint32_t r = (uint32_t)(blockIdx.x * (256 / LPR)) + threadIdx.x / LPR;
  const bool on = r < rows && col < a.d;
  int64_t oo = 0, zo = 0;
  if (r < rows) gate_row(a, r, oo, zo);
  float x[8], z[8], w[8];
  fill8(x, 0.f);
  fill8(z, 0.f);
  fill8(w, 1.f);
  if (on) {
    load8(reinterpret_cast<const E*>(a.O) + oo + col, x);
    load8(reinterpret_cast<const E*>(a.Z) + zo + col, z);
    if (a.w) load8(a.w + col, w);
  }
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  const float rstd = 1.f / sqrtf(group_sum<LPR>(ss) / (float)a.d + a.eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float f, df;
    gate(a.act, z[e], f, df);
    x[e] = x[e] * rstd * w[e] * f;
  }
  if (on) store8(reinterpret_cast<E*>(a.Y) + (int64_t)r * a.d + col, x);
}

template <int LPR, class E>
__global__ __launch_bounds__(256) void gate_norm_bwd_kernel(GateNormLaunch a, uint32_t rows, float* part) {
  __shared__ float sums[256 / LPR][8 * LPR];
  const int col = 8 * (threadIdx.x % LPR);
  const uint32_t step = gridDim.x * (256 / LPR);
  float w[8], dw[8];
  fill8(w, 1.f);
  fill8(dw, 0.f);
  if (a.w && col < a.d) load8(a.w + col, w);
  for (uint32_t r0 = blockIdx.x * (256 / LPR); r0 < rows; r0 += step) {
    const uint32_t r = r0 + threadIdx.x / LPR;
    const bool on = r < rows && col < a.d;
    int64_t oo = 0, zo = 0;
    if (r < rows) gate_row(a, r, oo, zo);
    float x[8], z[8], dy[8];
    fill8(x, 0.f);
    fill8(z, 0.f);
    fill8(dy, 0.f);
    if (on) {
      load8(reinterpret_cast<const E*>(a.O) + oo + col, x);
      load8(reinterpret_cast<const E*>(a.Z) + zo + col, z);
      load8(reinterpret_cast<const E*>(a.dY) + (int64_t)r * a.d + col, dy);
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    // past the last row the norm of zeros would be infinite where eps is 0, and dw not a number
    const float norm = group_sum<LPR>(ss) / (float)a.d + a.eps;
    const float rstd = r < rows ? 1.f / sqrtf(norm) : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float f, df;
      gate(a.act, z[e], f, df);
      const float n = x[e] * rstd, u = dy[e] * f;
      z[e] = dy[e] * n * w[e] * df;
      dw[e] = fmaf(u, n, dw[e]);
      x[e] = n;
      dy[e] = u * w[e];
      dot = fmaf(dy[e], n, dot);
    }
    dot = group_sum<LPR>(dot) / (float)a.d;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = rstd * (dy[e] - x[e] * dot);
    if (on) {
      store8(reinterpret_cast<E*>(a.dO) + oo + col, x);
      store8(reinterpret_cast<E*>(a.dZ) + (int64_t)r * a.d + col, z);
    }
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[threadIdx.x / LPR][col + e] = dw[e];
  __syncthreads();
  for (int i = threadIdx.x; i < a.d; i += 256) {
    float s = 0.f;
    for (int k = 0; k < 256 / LPR; ++k) s += sums[k][i];
    part[(int64_t)blockIdx.x * a.d + i] = s;
  }
}

// sums over k < n of part[k][j][i], in order: 16 columns a workgroup, 64 threads a column (each
// a fixed run of k), joined in order.  j = 0 gives out0; j = 1 times f1 (NULL = 1) out1, times f2 out2
struct ColumnSum {
  float *out0, *out1, *out2;
  const float *f1, *f2;
};
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* part, int n, int D, int n_in, ColumnSum o) {
  constexpr int RUNS = 64;
  __shared__ double red[RUNS][17];
  const int c = threadIdx.x % 16, k0 = threadIdx.x / 16, i = blockIdx.x * 16 + c;
  const int j = blockIdx.y;
  if (j == 0 ? !o.out0 : !o.out1 && !o.out2) return;
  const int run = (n + RUNS - 1) / RUNS, k1 = min(n, (k0 + 1) * run);
  double x = 0.0;
  if (i < D)
#pragma unroll 8
    for (int k = k0 * run; k < k1; ++k) x += (double)part[((int64_t)k * n_in + j) * D + i];
  red[k0][c] = x;
  __syncthreads();
  // 16 neighbouring runs, then those four sums
  if (k0 < 4) {
    x = 0.0;
#pragma unroll
    for (int k = 0; k < 16; ++k) x += red[16 * k0 + k][c];
  }
  __syncthreads();
  if (k0 < 4) red[k0][c] = x;
  __syncthreads();
  if (k0 > 0 || i >= D) return;
  x = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
  if (j == 0) {
    o.out0[i] = (float)x;
  } else {
    if (o.out1) o.out1[i] = (float)(o.f1 ? x * (double)o.f1[i] : x);
    if (o.out2) o.out2[i] = (float)(o.f2 ? x * (double)o.f2[i] : x);
  }
}

// ---- residual norm ----------------------------------------------------------------------
// WPR waves a row, 8 V columns a lane: column 8 (lane + 64 WPR v) + e

namespace {

template <int WPR>
struct RowSum {
  // sum over the row; every wave of the workgroup calls it together.  Two buffers of WPR values
  // (the memory behind red, taken flat) in turn
  float (*red)[2];
  int phase = 0;
  __device__ __forceinline__ float operator()(float x) {
    x = group_sum<64>(x);
    if constexpr (WPR > 1) {
      const int wave = threadIdx.x / WAVE;
      float* r = &red[0][0] + phase * WPR;
      if (lane_id() == 0) r[wave] = x;
      __syncthreads();
      x = 0.f;
#pragma unroll
      for (int k = 0; k < WPR; ++k) x += r[k];
      phase ^= 1;  // the next sum writes the other half: its barrier comes after these reads
    }
    return x;
  }
};

}  // namespace

template <int WPR, int V, class EX, class EY>
__global__ __launch_bounds__(WPR * WAVE < 256 ? 256 : WPR * WAVE) void res_norm_kernel(ResNormLaunch a) {
  constexpr int ROWS = WPR == 1 ? 4 : 1;  // rows of a workgroup at a time
  constexpr int TPR = WPR * WAVE;
  __shared__ float red[WPR][2];
  RowSum<WPR> row_sum{red};
  const int tid = threadIdx.x % TPR;
  const float inv = 1.f / (float)a.D;
  float wq[V][8], ws[V][8], wp[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = 8 * (tid + TPR * v);
    fill8(wq[v], 1.f);
    fill8(ws[v], a.alpha);
    fill8(wp[v], 1.f);
    if (col < a.D) {
      if (a.w_post) load8(a.w_post + col, wq[v]);
      if (a.s) {
        load8(a.s + col, ws[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ws[v][e] *= a.alpha;
      }
      if (a.w_pre) load8(a.w_pre + col, wp[v]);
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t r = r0 + (ROWS > 1 ? threadIdx.x / TPR : 0);
    const bool row_on = r < a.rows;
    const int64_t at = r * a.D;
    float x[V][8], y[V][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = 8 * (tid + TPR * v);
      fill8(x[v], 0.f);
      fill8(y[v], 0.f);
      if (row_on && col < a.D) {
        load8(reinterpret_cast<const EX*>(a.X) + at + col, x[v]);
        load8(reinterpret_cast<const EY*>(a.Y) + at + col, y[v]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[v][e], y[v][e], ss);
    }
    const float ry = a.w_post ? 1.f / sqrtf(row_sum(ss) * inv + a.eps) : 1.f;
    ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[v][e] = fmaf(ws[v][e], y[v][e] * ry * wq[v][e], x[v][e]);
        ss = fmaf(x[v][e], x[v][e], ss);
      }
    const float rr = a.N ? 1.f / sqrtf(row_sum(ss) * inv + a.eps) : 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = 8 * (tid + TPR * v);
      if (row_on && col < a.D) {
        store8(reinterpret_cast<EX*>(a.R) + at + col, x[v]);
        if (a.N) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[v][e] *= rr * wp[v][e];
          store8(reinterpret_cast<EY*>(a.N) + at + col, x[v]);
        }
      }
    }
  }
}

template <int WPR, int V, class EX, class EY>
__global__ __launch_bounds__(WPR * WAVE < 256 ? 256 : WPR * WAVE) void res_norm_bwd_kernel(ResNormLaunch a,
                                                                                          float* part) {
  constexpr int ROWS = WPR == 1 ? 4 : 1;
  constexpr int TPR = WPR * WAVE;
  __shared__ float red[WPR][2];
  __shared__ float cols[ROWS > 1 ? ROWS * 512 * V : 1];
  RowSum<WPR> row_sum{red};
  const int tid = threadIdx.x % TPR;
  const float inv = 1.f / (float)a.D;
  float wp[V][8], wb[V][8], g_pre[V][8], g_y[V][8];
  // the weights of vector v: w_pre, and s w_post.  With two vectors they do not fit beside the row
  // and come anew from the caches where they are used: 36 to 53 registers still go to scratch
  // memory (108 to 120 bytes a lane), with the weights kept it would be 130.
  auto weights = [&](int v) {
    const int col = 8 * (tid + TPR * v);
    fill8(wp[v], 1.f);
    fill8(wb[v], 1.f);
    if (col < a.D) {
      if (a.w_pre) load8(a.w_pre + col, wp[v]);
      if (a.w_post) load8(a.w_post + col, wb[v]);
      if (a.s) {
        float ws[8];
        load8(a.s + col, ws);
#pragma unroll
        for (int e = 0; e < 8; ++e) wb[v][e] *= ws[e];
      }
    }
  };
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (V == 1) weights(v);
    fill8(g_pre[v], 0.f);
    fill8(g_y[v], 0.f);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t r = r0 + (ROWS > 1 ? threadIdx.x / TPR : 0);
    const bool row_on = r < a.rows;
    const int64_t at = r * a.D;
    float x[V][8], y[V][8], dn[V][8], dr[V][8];
    float ssx = 0.f, ssy = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = 8 * (tid + TPR * v);
      if constexpr (V > 1) weights(v);
      fill8(x[v], 0.f);
      fill8(y[v], 0.f);
      fill8(dn[v], 0.f);
      fill8(dr[v], 0.f);
      if (row_on && col < a.D) {
        if (a.dN) {
          load8(reinterpret_cast<const EX*>(a.X) + at + col, x[v]);
          load8(reinterpret_cast<const EY*>(a.dN) + at + col, dn[v]);
        }
        if (a.w_post || a.ds) load8(reinterpret_cast<const EY*>(a.Y) + at + col, y[v]);
        if (a.dR) load8(reinterpret_cast<const EX*>(a.dR) + at + col, dr[v]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ssx = fmaf(x[v][e], x[v][e], ssx);
        ssy = fmaf(y[v][e], y[v][e], ssy);
        dot = fmaf(dn[v][e] * wp[v][e], x[v][e], dot);
      }
    }
    if (a.dN) {
      const float norm = row_sum(ssx) * inv + a.eps;
      const float rstd = row_on ? 1.f / sqrtf(norm) : 0.f;  // a row past the last adds nothing, eps 0 or not
      const float m = row_sum(dot) * inv * rstd;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (V > 1) weights(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = x[v][e] * rstd;
          g_pre[v][e] = fmaf(dn[v][e], n, g_pre[v][e]);
          dr[v][e] += rstd * (dn[v][e] * wp[v][e] - n * m);
        }
      }
    }
    float ry = 1.f;
    if (a.w_post) {
      const float norm = row_sum(ssy) * inv + a.eps;
      ry = row_on ? 1.f / sqrtf(norm) : 0.f;
    }
    dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = 8 * (tid + TPR * v);
      if constexpr (V > 1) weights(v);
      if (row_on && col < a.D) store8(reinterpret_cast<EX*>(a.dX) + at + col, dr[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = a.alpha * dr[v][e], n = y[v][e] * ry;
        g_y[v][e] = fmaf(d, n, g_y[v][e]);
        dr[v][e] = d * wb[v][e];
        dot = fmaf(dr[v][e], n, dot);
      }
    }
    if (a.w_post) {
      const float m = row_sum(dot) * inv;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) dr[v][e] = ry * (dr[v][e] - y[v][e] * ry * m);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = 8 * (tid + TPR * v);
      if (row_on && col < a.D) store8(reinterpret_cast<EY*>(a.dY) + at + col, dr[v]);
    }
  }
  // partial sums of this workgroup: [2][D]
  float* out = part + (int64_t)blockIdx.x * 2 * a.D;
  auto put = [&](int which, float (&x)[V][8]) {
    if constexpr (ROWS > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) cols[(threadIdx.x / TPR) * 512 * V + 8 * (tid + TPR * v) + e] = x[v][e];
      __syncthreads();
      for (int i = threadIdx.x; i < a.D; i += ROWS * TPR) {
        float s = 0.f;
        for (int k = 0; k < ROWS; ++k) s += cols[k * 512 * V + i];
        out[(int64_t)which * a.D + i] = s;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = 8 * (tid + TPR * v);
        if (col < a.D) store8(out + (int64_t)which * a.D + col, x[v]);
      }
    }
  };
  if (a.dw_pre) put(0, g_pre);
  if (a.dw_post || a.ds) put(1, g_y);
}

// ---- host side ----------------------------------------------------------------------------

namespace {

uint32_t gate_rows(const GateNormLaunch& p) { return (uint32_t)(p.B * p.T * p.H); }
int lanes_per_row(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }
// workgroups of the gated norm's backward pass: four for each CU, each over many rows
int64_t gate_bwd_groups(const GateNormLaunch& p) {
  const int per = 256 / lanes_per_row(p.d);
  const int64_t n = ((int64_t)gate_rows(p) + per - 1) / per;
  return n < 1024 ? n : 1024;
}

template <class F>
int by_lanes(int d, F&& f) {
  switch (lanes_per_row(d)) {
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    default: return f(std::integral_constant<int, 32>{});
  }
}

// Waves and vectors of a row by its length: 8 values a lane where 16 waves hold the row, so that
// the row's tensors and, backwards, two column sums fit the registers; 16 values above 8192.
// Backwards one such row takes more registers than a CU has for it, so some go to scratch memory
// and nothing hides its latency: 4096 rows of 16384 run at 2.7 TB/s, 8192 rows of 8192 at 5.1
// (forwards 4.9 and 5.4).
template <class F>
int by_row(int D, F&& f) {
  using std::integral_constant;
  if (D <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (D <= 1024) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (D <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (D <= 4096) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (D <= 8192) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}
template <class F>
int by_types(int x_bf16, int y_bf16, F&& f) {
  if (x_bf16) return y_bf16 ? f((__bf16*)nullptr, (__bf16*)nullptr) : f((__bf16*)nullptr, (float*)nullptr);
  return y_bf16 ? f((float*)nullptr, (__bf16*)nullptr) : f((float*)nullptr, (float*)nullptr);
}

int64_t res_groups(const ResNormLaunch& p, int64_t most) {
  const int64_t n = p.D <= 512 ? (p.rows + 3) / 4 : p.rows;
  return n < most ? n : most;
}
constexpr int64_t RES_FWD_GROUPS = 2048, RES_BWD_GROUPS = 512;

void column_sum(const float* part, int64_t n, int D, int n_in, const ColumnSum& o, hipStream_t s) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((D + 15) / 16), (unsigned)n_in), dim3(1024), 0, s, part, (int)n,
                     D, n_in, o);
}

}  // namespace

void launch_column_sum(const float* part, int64_t n, int D, int n_in, float* out0, float* out1, hipStream_t s) {
  column_sum(part, n, D, n_in, {out0, out1, nullptr, nullptr, nullptr}, s);
}

size_t gate_norm_bwd_workspace(const GateNormLaunch& p) { return (size_t)gate_bwd_groups(p) * p.d * 4; }

int launch_gate_norm(const GateNormLaunch& p, hipStream_t s) {
  const uint32_t rows = gate_rows(p);
  return by_lanes(p.d, [&](auto lpr) {
    constexpr int L = lpr.value, per = 256 / L;
    const dim3 grid((rows + per - 1) / per), block(256);
    if (p.bf16)
      hipLaunchKernelGGL((gate_norm_kernel<L, __bf16>), grid, block, 0, s, p, rows);
    else
      hipLaunchKernelGGL((gate_norm_kernel<L, float>), grid, block, 0, s, p, rows);
    return 0;
  });
}

int launch_gate_norm_bwd(const GateNormLaunch& p, void* workspace, hipStream_t s) {
  const uint32_t rows = gate_rows(p);
  const int64_t n = gate_bwd_groups(p);
  float* part = p.dw ? reinterpret_cast<float*>(workspace) : nullptr;
  const int rc = rows == 0 ? 0 : by_lanes(p.d, [&](auto lpr) {  // no rows: dw = 0
    constexpr int L = lpr.value;
    const dim3 grid((unsigned)n), block(256);
    if (p.bf16)
      hipLaunchKernelGGL((gate_norm_bwd_kernel<L, __bf16>), grid, block, 0, s, p, rows, part);
    else
      hipLaunchKernelGGL((gate_norm_bwd_kernel<L, float>), grid, block, 0, s, p, rows, part);
    return 0;
  });
  if (p.dw) column_sum(part, n, p.d, 1, {p.dw, nullptr, nullptr, nullptr, nullptr}, s);
  return rc;
}

size_t res_norm_bwd_workspace(const ResNormLaunch& p) { return (size_t)res_groups(p, RES_BWD_GROUPS) * 2 * p.D * 4; }

int launch_res_norm(const ResNormLaunch& p, hipStream_t s) {
  return by_row(p.D, [&](auto wpr, auto v) {
    return by_types(p.x_bf16, p.y_bf16, [&](auto ex, auto ey) {
      constexpr int W = wpr.value;
      const dim3 grid((unsigned)res_groups(p, RES_FWD_GROUPS)), block(W == 1 ? 256 : W * WAVE);
      hipLaunchKernelGGL((res_norm_kernel<W, v.value, std::remove_pointer_t<decltype(ex)>,
                                          std::remove_pointer_t<decltype(ey)>>), grid, block, 0, s, p);
      return 0;
    });
  });
}

int launch_res_norm_bwd(const ResNormLaunch& p, void* workspace, hipStream_t s) {
  const int64_t n = res_groups(p, RES_BWD_GROUPS);
  float* part = reinterpret_cast<float*>(workspace);
  const int rc = p.rows == 0 ? 0 : by_row(p.D, [&](auto wpr, auto v) {  // no rows: zero sums
    return by_types(p.x_bf16, p.y_bf16, [&](auto ex, auto ey) {
      constexpr int W = wpr.value;
      const dim3 grid((unsigned)n), block(W == 1 ? 256 : W * WAVE);
      hipLaunchKernelGGL((res_norm_bwd_kernel<W, v.value, std::remove_pointer_t<decltype(ex)>,
                                              std::remove_pointer_t<decltype(ey)>>), grid, block, 0, s, p, part);
      return 0;
    });
  });
  if (p.dw_pre || p.dw_post || p.ds) column_sum(part, n, p.D, 2, {p.dw_pre, p.dw_post, p.ds, p.s, p.w_post}, s);
  return rc;
}

}  // namespace gdn
