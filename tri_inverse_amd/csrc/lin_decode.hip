// lin_decode.hip -- linear attention with a decay for each head, one token at a time.
//
// Per (b, h) and token t, a = e^{g_t}, the state S [d_k][d_v] fp32:
//   S <- a S + k v^T,     o = scale S^T q
// A call reads and writes the state once and keeps it in registers for all its n tokens, so
// its bytes bound it: 2 x 4 d_k d_v per head.
//
// One wave per (b, h, 32 columns of d_v).  Lane l = 8 rg + cg holds columns 4 cg .. + 3 of
// rows RPL rg .. + RPL - 1 (RPL = d_k / 8); every access to S moves 8 rows of 128 bytes.
// The output's sum over d_k runs over a lane's rows, then over the 8 row groups.  A wave for
// each 32 columns and not for a head: one token is all latency, and 8 KB of state a wave keeps
// enough loads in flight.
//
// Measured: 64 sequences, 32 heads, d = 128, one token: 47.5 us for 270 MB, 5.7 TB/s (a copy of
// 1 GiB reaches 5.2); one sequence 4.3 us, launch and the latency of one round of loads.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

template <int N>
__device__ __forceinline__ void widen(const __bf16* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const bf16x8 v = *reinterpret_cast<const bf16x8*>(p + 8 * i);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[8 * i + e] = (float)v[e];
  }
}
template <int N>
__device__ __forceinline__ void widen(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
  }
}
__device__ __forceinline__ f32x4 widen4(const __bf16* p) { return unpack4(*reinterpret_cast<const bf16x4*>(p)); }
__device__ __forceinline__ f32x4 widen4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// sum over lanes l ^ 8m, in every lane
__device__ __forceinline__ float sum_rows(float x) {
  x += dpp_f<0x128>(x);
  float a, b;
  self_swap_f<16>(x, a, b);
  x = a + b;
  self_swap_f<32>(x, a, b);
  return a + b;
}

}  // namespace

template <int DK, class TI>
__global__ __launch_bounds__(512) void lin_decode_kernel(LinDecodeLaunch a) {
  constexpr int RPL = DK / 8;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int64_t bh = blockIdx.x;
  const int h = (int)(bh % a.H), group = a.H / a.H_qk;
  const int64_t bq = bh / group;  // (b H + h) / group = b H_qk + h / group
  const int l = lane_id(), rg = l >> 3, cg = l & 7;
  const int dv = a.d_v;
  const int col = 32 * wave + 4 * cg, row0 = RPL * rg;
  const TI* Qp = reinterpret_cast<const TI*>(a.Q) + bq * a.n * DK + row0;
  const TI* Kp = reinterpret_cast<const TI*>(a.K) + bq * a.n * DK + row0;
  const TI* Vp = reinterpret_cast<const TI*>(a.V) + bh * a.n * dv + col;
  const float* gp = a.g_per_head ? a.g + h : a.g + bh * a.n;

  // streamed once: non-temporal
  const int64_t sbase = (bh * DK + row0) * dv + col;
  f32x4 S[RPL];
#pragma unroll
  for (int i = 0; i < RPL; ++i)
    S[i] = a.S_in ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(a.S_in + sbase + (int64_t)i * dv))
                  : zero4();
  for (int t = 0; t < a.n; ++t) {
    float k[RPL], q[RPL];
    widen<RPL>(Kp + (int64_t)t * DK, k);
    widen<RPL>(Qp + (int64_t)t * DK, q);
    const f32x4 v = widen4(Vp + (int64_t)t * dv);
    const float av = expf(gp[a.g_per_head ? 0 : t]);
    f32x4 o = zero4();
#pragma unroll
    for (int i = 0; i < RPL; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        S[i][c] = fmaf(k[i], v[c], av * S[i][c]);
        o[c] = fmaf(S[i][c], q[i], o[c]);
      }
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = sum_rows(o[c]) * a.scale;
    if (rg == 0) {
      const int64_t oo = (bh * a.n + t) * dv + col;
      if (a.o_bf16)
        *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(a.O) + oo) = pack4(o);
      else
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.O) + oo) = o;
    }
  }
#pragma unroll
  for (int i = 0; i < RPL; ++i)
    __builtin_nontemporal_store(S[i], reinterpret_cast<f32x4*>(a.S_out + sbase + (int64_t)i * dv));
}

int launch_lin_decode(const LinDecodeLaunch& p, hipStream_t s) {
  if (p.d_v % 32 != 0 || p.d_v > 256 || p.d_v <= 0) return -1;
  const dim3 grid((unsigned)(p.B * p.H)), block((unsigned)(WAVE * (p.d_v / 32)));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, s, p);
    return 0;
  };
  switch (p.d_k) {
    case 64: return p.in_bf16 ? go(lin_decode_kernel<64, __bf16>) : go(lin_decode_kernel<64, float>);
    case 128: return p.in_bf16 ? go(lin_decode_kernel<128, __bf16>) : go(lin_decode_kernel<128, float>);
    default: return -1;
  }
}

}  // namespace gdn
