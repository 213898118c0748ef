// abi.cpp -- the C ABI of libgdn (declared in include/gdn.h): argument validation,
// status codes, and the hand-off to the kernel launchers on the caller's stream.
// Validation happens entirely on the host and returns before any HIP call, so every
// error path can be exercised without a GPU.
#include "gdn.h"

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "gdn_kernels.hpp"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool chunk_ok(int C) { return C == 16 || C == 32 || C == 64 || C == 128 || C == 256; }
bool chunk_small(int C) { return C == 16 || C == 32 || C == 64; }
bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128 || d == 256; }

gdn_status launch_result(int rc) {
  if (rc < 0) return GDN_ERR_UNSUPPORTED;
  hipError_t e = hipGetLastError();
  return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

// validates a gdn_blocks descriptor; src_out: 0 = A given, 1 = K bf16, 2 = K fp32.
// An empty batch (n_blocks == 0) only needs valid sizes: its pointers may be NULL.
gdn_status check_blocks(const gdn_blocks* in, bool allow_A, bool allow_k_f32, int* src_out) {
  if (!in) return GDN_ERR_NULL_POINTER;
  if (in->n_blocks < 0 || in->C <= 0) return GDN_ERR_BAD_SHAPE;
  if (!chunk_ok(in->C)) return GDN_ERR_UNSUPPORTED;
  const bool empty = in->n_blocks == 0;
  if (in->A) {
    if (!allow_A) return GDN_ERR_UNSUPPORTED;
    if (!aligned16(in->A)) return GDN_ERR_BAD_ALIGNMENT;
    *src_out = 0;
    return GDN_OK;
  }
  if (in->d_k <= 0) {
    if (empty && !in->K) {  // empty batch given as A == NULL, K == NULL
      *src_out = 0;
      return GDN_OK;
    }
    return GDN_ERR_BAD_SHAPE;
  }
  if (!head_dim_ok(in->d_k)) return GDN_ERR_UNSUPPORTED;
  if (in->k_dtype == GDN_BF16) {
    *src_out = 1;
  } else if (in->k_dtype == GDN_F32) {
    if (!allow_k_f32) return GDN_ERR_UNSUPPORTED;
    *src_out = 2;
  } else {
    return GDN_ERR_BAD_DTYPE;
  }
  if (empty) return GDN_OK;
  if (!in->K || !in->beta || !in->g) return GDN_ERR_NULL_POINTER;
  if (!aligned16(in->K) || !aligned16(in->beta) || !aligned16(in->g)) return GDN_ERR_BAD_ALIGNMENT;
  return GDN_OK;
}

gdn::BlocksArgs to_args(const gdn_blocks* in) {
  gdn::BlocksArgs a;
  a.A = in->A;
  a.K = in->K;
  a.beta = in->beta;
  a.g = in->g;
  a.n_blocks = in->n_blocks;
  a.C = in->C;
  a.d_k = in->d_k;
  a.g_cumulative = in->g_cumulative;
  return a;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int gdn_abi_version(void) { return GDN_ABI_VERSION; }

const char* gdn_status_string(int32_t s) {
  switch (s) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_NULL_POINTER: return "GDN_ERR_NULL_POINTER: a required pointer is NULL";
    case GDN_ERR_BAD_SHAPE: return "GDN_ERR_BAD_SHAPE: a size or order argument is out of range";
    case GDN_ERR_BAD_DTYPE: return "GDN_ERR_BAD_DTYPE: dtype code not accepted for this argument";
    case GDN_ERR_BAD_ALIGNMENT: return "GDN_ERR_BAD_ALIGNMENT: a tensor pointer is not 16-byte aligned";
    case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED: configuration not implemented by this build";
    case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE: workspace missing or smaller than the query returned";
    case GDN_ERR_HIP: return "GDN_ERR_HIP: the HIP runtime reported an error at launch";
    default: return "unknown gdn_status";
  }
}

gdn_status gdn_build_A(const gdn_blocks* in, float* A_out, void* stream) {
  int src = 0;
  if (in && in->A) return GDN_ERR_UNSUPPORTED;  // A is the output here
  gdn_status st = check_blocks(in, false, true, &src);
  if (st != GDN_OK) return st;
  if (!chunk_small(in->C)) return GDN_ERR_UNSUPPORTED;
  if (in->n_blocks == 0) return GDN_OK;
  if (!A_out) return GDN_ERR_NULL_POINTER;
  if (!aligned16(A_out)) return GDN_ERR_BAD_ALIGNMENT;
  return launch_result(gdn::launch_build_A(to_args(in), src, A_out, as_stream(stream)));
}

gdn_status gdn_tri_inverse_neumann(const gdn_blocks* in, int32_t N, int32_t mask, int32_t compute,
                                   void* T_out, int32_t t_dtype, gdn_fp8_stats* stats, void* stream) {
  int src = 0;
  gdn_status st = check_blocks(in, true, false, &src);
  if (st != GDN_OK) return st;
  if (N < 1 || N >= in->C) return GDN_ERR_BAD_SHAPE;
  if (mask != 0 && mask != 1) return GDN_ERR_BAD_SHAPE;
  if (compute != GDN_F32 && compute != GDN_BF16 && compute != GDN_FP8_E4M3 && compute != GDN_INT8 &&
      compute != GDN_INT16)
    return GDN_ERR_BAD_DTYPE;
  if (t_dtype != GDN_F32 && t_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  // C >= 128 (bf16 keys and products): the band kernel for the masked sum with N <= 16,
  // the full-triangle kernel otherwise
  const bool large = !chunk_small(in->C);
  if (large && (src != 1 || compute != GDN_BF16)) return GDN_ERR_UNSUPPORTED;
  const bool band = large && mask && N <= 16;
  if (stats && !aligned16(stats)) return GDN_ERR_BAD_ALIGNMENT;
  if (in->n_blocks > 0) {
    if (!T_out) return GDN_ERR_NULL_POINTER;
    if (!aligned16(T_out)) return GDN_ERR_BAD_ALIGNMENT;
  }
  hipStream_t s = as_stream(stream);
  auto* st64 = reinterpret_cast<unsigned long long*>(stats);
  if (st64) {
    gdn::launch_zero_stats(st64, s);
    if (hipGetLastError() != hipSuccess) return GDN_ERR_HIP;
  }
  if (in->n_blocks == 0) return GDN_OK;
  if (band)
    return launch_result(gdn::launch_band(to_args(in), nullptr, 0, N, 0, T_out, t_dtype == GDN_BF16,
                                          nullptr, nullptr, 0, s));
  if (large)
    return launch_result(gdn::launch_dense(to_args(in), nullptr, 0, 0, N, mask, nullptr, 0, 0, T_out,
                                           t_dtype == GDN_BF16, nullptr, nullptr, 0, s));
  return launch_result(gdn::launch_neumann(to_args(in), src, N, mask, compute, T_out,
                                           t_dtype == GDN_BF16, st64, s));
}

gdn_status gdn_tri_inverse_exact(const gdn_blocks* in, int32_t compute, void* T_out,
                                 int32_t t_dtype, void* stream) {
  int src = 0;
  gdn_status st = check_blocks(in, true, false, &src);
  if (st != GDN_OK) return st;
  if (compute == GDN_FP8_E4M3 || compute == GDN_INT8 || compute == GDN_INT16) return GDN_ERR_UNSUPPORTED;
  if (compute != GDN_F32 && compute != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  if (t_dtype != GDN_F32 && t_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  const bool large = !chunk_small(in->C);
  if (large && (src != 1 || compute != GDN_BF16)) return GDN_ERR_UNSUPPORTED;
  if (in->n_blocks == 0) return GDN_OK;
  if (!T_out) return GDN_ERR_NULL_POINTER;
  if (!aligned16(T_out)) return GDN_ERR_BAD_ALIGNMENT;
  if (large)
    return launch_result(gdn::launch_dense(to_args(in), nullptr, 0, 1, 0, 0, nullptr, 0, 0, T_out,
                                           t_dtype == GDN_BF16, nullptr, nullptr, 0, as_stream(stream)));
  return launch_result(gdn::launch_exact(to_args(in), src, compute, T_out, t_dtype == GDN_BF16,
                                         as_stream(stream)));
}

gdn_status gdn_tri_inverse_residual(const gdn_blocks* in, int32_t N, int32_t mask, int32_t S,
                                    int32_t compute, void* T_out, int32_t t_dtype, void* stream) {
  int src = 0;
  gdn_status st = check_blocks(in, true, false, &src);
  if (st != GDN_OK) return st;
  if (N < 1 || N >= in->C) return GDN_ERR_BAD_SHAPE;
  if (mask != 0 && mask != 1) return GDN_ERR_BAD_SHAPE;
  if (S < 0 || S > 64) return GDN_ERR_BAD_SHAPE;
  if (compute != GDN_F32 && compute != GDN_BF16 && compute != GDN_FP8_E4M3 && compute != GDN_INT8 &&
      compute != GDN_INT16)
    return GDN_ERR_BAD_DTYPE;
  if (t_dtype != GDN_F32 && t_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  if (compute != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (!chunk_small(in->C)) return GDN_ERR_UNSUPPORTED;
  if (in->n_blocks == 0) return GDN_OK;
  if (!T_out) return GDN_ERR_NULL_POINTER;
  if (!aligned16(T_out)) return GDN_ERR_BAD_ALIGNMENT;
  return launch_result(gdn::launch_residual(to_args(in), src, N, mask, S, T_out, t_dtype == GDN_BF16,
                                            as_stream(stream)));
}

gdn_status gdn_tri_inverse_fs(const gdn_blocks* in, void* T_out, int32_t t_dtype, void* stream) {
  int src = 0;
  gdn_status st = check_blocks(in, true, false, &src);
  if (st != GDN_OK) return st;
  if (t_dtype != GDN_F32 && t_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  const bool c128 = in->C == 128;
  if (!chunk_small(in->C) && !c128) return GDN_ERR_UNSUPPORTED;
  if (c128 && src == 2) return GDN_ERR_UNSUPPORTED;  // fp32 keys: C <= 64 only
  if (c128 && src == 1 && !(in->d_k == 64 || in->d_k == 128)) return GDN_ERR_UNSUPPORTED;
  if (in->n_blocks == 0) return GDN_OK;
  if (!T_out) return GDN_ERR_NULL_POINTER;
  if (!aligned16(T_out)) return GDN_ERR_BAD_ALIGNMENT;
  if (c128)
    return launch_result(gdn::launch_fs128(to_args(in), src, T_out, t_dtype == GDN_BF16, as_stream(stream)));
  return launch_result(gdn::launch_fs(to_args(in), src, T_out, t_dtype == GDN_BF16, as_stream(stream)));
}

gdn_status gdn_wy(const gdn_blocks* in, const void* T, int32_t t_dtype, const gdn_inverse_cfg* inv,
                  const void* V, int32_t d_v, int32_t gate_k, void* W_out, void* U_out,
                  int32_t out_dtype, void* stream) {
  int src = 0;
  if (in && in->A) return GDN_ERR_UNSUPPORTED;  // the products need K itself
  gdn_status st = check_blocks(in, false, false, &src);
  if (st != GDN_OK) return st;
  if (T) {
    if (t_dtype != GDN_F32 && t_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  } else {
    if (!inv) return GDN_ERR_NULL_POINTER;
    if (inv->mode != GDN_INV_NEUMANN && inv->mode != GDN_INV_EXACT) return GDN_ERR_BAD_SHAPE;
    if (inv->mode == GDN_INV_NEUMANN && (inv->N < 1 || inv->N >= in->C)) return GDN_ERR_BAD_SHAPE;
    if (inv->mask != 0 && inv->mask != 1) return GDN_ERR_BAD_SHAPE;
    if (inv->compute != GDN_BF16) {
      if (inv->compute == GDN_F32 || inv->compute == GDN_FP8_E4M3 || inv->compute == GDN_INT8 ||
          inv->compute == GDN_INT16)
        return GDN_ERR_UNSUPPORTED;
      return GDN_ERR_BAD_DTYPE;
    }
  }
  if (d_v <= 0) return GDN_ERR_BAD_SHAPE;
  if (gate_k != 0 && gate_k != 1) return GDN_ERR_BAD_SHAPE;
  if (out_dtype != GDN_F32 && out_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  // C >= 128: the band kernel when T is formed as the masked sum with N <= 16, the
  // full-triangle kernel otherwise (T formed, or given)
  const bool large = in->C == 128 || in->C == 256;
  const bool band = large && !T && inv->mode == GDN_INV_NEUMANN && inv->mask && inv->N <= 16;
  if (!(large || in->C == 32 || in->C == 64)) return GDN_ERR_UNSUPPORTED;
  if (!(in->d_k == 64 || in->d_k == 128) || !(d_v == 64 || d_v == 128)) return GDN_ERR_UNSUPPORTED;
  if (in->n_blocks == 0) return GDN_OK;
  if (!V || !W_out || !U_out) return GDN_ERR_NULL_POINTER;
  if (!aligned16(V) || !aligned16(W_out) || !aligned16(U_out) || (T && !aligned16(T)))
    return GDN_ERR_BAD_ALIGNMENT;
  const int mode = T ? 0 : inv->mode, N = T ? 0 : inv->N, mask = T ? 0 : inv->mask;
  if (band)
    return launch_result(gdn::launch_band(to_args(in), V, d_v, N, gate_k, nullptr, 0, W_out, U_out,
                                          out_dtype == GDN_BF16, as_stream(stream)));
  if (large)
    return launch_result(gdn::launch_dense(to_args(in), T, t_dtype == GDN_BF16, mode, N, mask, V, d_v,
                                           gate_k, nullptr, 0, W_out, U_out, out_dtype == GDN_BF16,
                                           as_stream(stream)));
  return launch_result(gdn::launch_wy(to_args(in), T, t_dtype == GDN_BF16, mode, N, mask, V, d_v,
                                      gate_k, W_out, U_out, out_dtype == GDN_BF16,
                                      as_stream(stream)));
}

// argument checks of gdn_chunk_fwd that need no pointer (shared with the workspace query)
static gdn_status check_chunk_args(int32_t qkv_dtype, int32_t o_dtype, int32_t B, int32_t H, int64_t T, int32_t d_k,
                            int32_t d_v, int32_t C, const gdn_inverse_cfg* inv) {
  if (!inv) return GDN_ERR_NULL_POINTER;
  if (B < 0 || H < 0 || T < 0 || d_k <= 0 || d_v <= 0 || C <= 0) return GDN_ERR_BAD_SHAPE;
  if (qkv_dtype != GDN_BF16) return (qkv_dtype == GDN_F32) ? GDN_ERR_UNSUPPORTED : GDN_ERR_BAD_DTYPE;
  if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  if (!chunk_ok(C)) return GDN_ERR_UNSUPPORTED;
  if (T % C != 0) return GDN_ERR_BAD_SHAPE;
  if (inv->mode != GDN_INV_NEUMANN && inv->mode != GDN_INV_EXACT && inv->mode != GDN_INV_NEUMANN_PRODUCTS)
    return GDN_ERR_BAD_SHAPE;
  if (inv->mode != GDN_INV_EXACT && (inv->N < 1 || inv->N >= C)) return GDN_ERR_BAD_SHAPE;
  if (inv->mask != 0 && inv->mask != 1) return GDN_ERR_BAD_SHAPE;
  if (inv->compute != GDN_BF16 && inv->compute != GDN_FP8_E4M3 && inv->compute != GDN_F32 &&
      inv->compute != GDN_INT8 && inv->compute != GDN_INT16)
    return GDN_ERR_BAD_DTYPE;
  if (inv->compute == GDN_F32 || inv->compute == GDN_INT8 || inv->compute == GDN_INT16) return GDN_ERR_UNSUPPORTED;
  if (inv->compute == GDN_FP8_E4M3 && inv->mode == GDN_INV_EXACT) return GDN_ERR_UNSUPPORTED;
  if (C != 64) return GDN_ERR_UNSUPPORTED;
  if (!(d_k == 64 || d_k == 128)) return GDN_ERR_UNSUPPORTED;
  if (d_v % 32 != 0 || d_v > 256) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

static size_t chunk_workspace(int32_t B, int32_t H, int64_t T, int32_t C, const gdn_inverse_cfg* inv) {
  if (inv->mode == GDN_INV_NEUMANN && gdn::chunk_fwd_band_path(inv->mode, inv->N, inv->mask, inv->compute))
    return 0;
  const size_t chunks = (size_t)B * (size_t)H * (size_t)(T / C);
  if (inv->mode == GDN_INV_NEUMANN && gdn::chunk_fwd_fp8_band(inv->mode, inv->N, inv->mask, inv->compute))
    return chunks * gdn::BAND_ROW_BYTES;
  return chunks * gdn::T_PACK_BYTES;
}

size_t gdn_chunk_fwd_workspace_bytes(int32_t B, int32_t H, int64_t T, int32_t d_k, int32_t d_v,
                                     int32_t C, const gdn_inverse_cfg* inv) {
  if (check_chunk_args(GDN_BF16, GDN_BF16, B, H, T, d_k, d_v, C, inv) != GDN_OK) return 0;
  return chunk_workspace(B, H, T, C, inv);
}

gdn_status gdn_chunk_fwd(const void* Q, const void* K, const void* V, int32_t qkv_dtype,
                         const float* beta, const float* g, const float* S0, void* O,
                         int32_t o_dtype, float* S_out, int32_t B, int32_t H, int64_t T,
                         int32_t d_k, int32_t d_v, int32_t C, float scale,
                         const gdn_inverse_cfg* inv, void* workspace, size_t workspace_bytes,
                         gdn_fp8_stats* stats, void* stream) {
  return gdn::chunk_fwd_impl(Q, K, V, qkv_dtype, beta, g, S0, O, o_dtype, S_out, B, H, T, d_k, d_v, C,
                             scale, inv, workspace, workspace_bytes, nullptr, stats, stream);
}

gdn_status gdn_decode(const void* Q, const void* K, const void* V, int32_t qkv_dtype,
                      const float* beta, const float* g, const float* S_in, float* S_out,
                      void* O, int32_t o_dtype, int32_t B, int32_t H, int32_t n,
                      int32_t d_k, int32_t d_v, float scale, void* stream) {
  if (B < 0 || H < 0 || n < 0 || d_k <= 0 || d_v <= 0) return GDN_ERR_BAD_SHAPE;
  if (qkv_dtype != GDN_BF16 && qkv_dtype != GDN_F32) return GDN_ERR_BAD_DTYPE;
  if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  if (!(d_k == 64 || d_k == 128)) return GDN_ERR_UNSUPPORTED;
  if (d_v % 32 != 0 || d_v > 256) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)B * H == 0) return GDN_OK;
  if (!S_out) return GDN_ERR_NULL_POINTER;
  if (n > 0 && (!Q || !K || !V || !beta || !g || !O)) return GDN_ERR_NULL_POINTER;
  for (const void* p : {Q, K, V, (const void*)beta, (const void*)g, (const void*)S_in,
                        (const void*)S_out, (const void*)O})
    if (p && !aligned16(p)) return GDN_ERR_BAD_ALIGNMENT;
  gdn::DecodeLaunch p;
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.beta = beta;
  p.g = g;
  p.S_in = S_in;
  p.S_out = S_out;
  p.O = O;
  p.B = B;
  p.H = H;
  p.n = n;
  p.d_k = d_k;
  p.d_v = d_v;
  p.in_bf16 = qkv_dtype == GDN_BF16;
  p.o_bf16 = o_dtype == GDN_BF16;
  p.scale = scale;
  return launch_result(gdn::launch_decode(p, as_stream(stream)));
}

// ---- linear attention with a decay for each head --------------------------------------

// sizes of a gdn_lin_shape (pointers are the entry points' matter)
static gdn_status check_lin(const gdn_lin_shape* s, bool bwd) {
  if (!s) return GDN_ERR_NULL_POINTER;
  if (s->B < 0 || s->H < 0 || s->H_qk < 0 || s->T < 0 || s->d_k <= 0 || s->d_v <= 0) return GDN_ERR_BAD_SHAPE;
  if (s->H > 0 && (s->H_qk == 0 || s->H % s->H_qk != 0)) return GDN_ERR_BAD_SHAPE;
  if (s->g_per_head != 0 && s->g_per_head != 1) return GDN_ERR_BAD_SHAPE;
  if (!(s->d_k == 64 || s->d_k == 128)) return GDN_ERR_UNSUPPORTED;
  if (bwd ? !(s->d_v == 64 || s->d_v == 128) : (s->d_v % 32 != 0 || s->d_v > 256)) return GDN_ERR_UNSUPPORTED;
  if (s->T > INT32_MAX - 64) return GDN_ERR_UNSUPPORTED;  // token indices within a sequence are 32 bits
  if ((int64_t)s->B * s->H > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

static gdn::LinLaunch lin_launch(const gdn_lin_shape* s) {
  gdn::LinLaunch p{};
  p.offsets = s->offsets;
  p.scale = s->scale;
  p.g_per_head = s->g_per_head;
  p.n_seq = s->B;
  p.H = s->H;
  p.H_qk = s->H_qk;
  p.d_k = s->d_k;
  p.d_v = s->d_v;
  p.T = s->T;
  return p;
}

static gdn_status check_workspace(size_t need, const void* workspace, size_t bytes) {
  if (need == 0) return GDN_OK;
  if (!workspace || bytes < need) return GDN_ERR_WORKSPACE;
  return aligned16(workspace) ? GDN_OK : GDN_ERR_BAD_ALIGNMENT;
}

static bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}

size_t gdn_lin_chunk_fwd_workspace_bytes(const gdn_lin_shape* s) {
  if (check_lin(s, false) != GDN_OK || s->B == 0 || s->H == 0 || !gdn::lin_grid_ok(lin_launch(s), false)) return 0;
  return gdn::lin_workspace(lin_launch(s), false);
}

size_t gdn_lin_chunk_bwd_workspace_bytes(const gdn_lin_shape* s) {
  if (check_lin(s, true) != GDN_OK || s->B == 0 || s->H == 0 || !gdn::lin_grid_ok(lin_launch(s), true)) return 0;
  return gdn::lin_workspace(lin_launch(s), true);
}

gdn_status gdn_lin_chunk_fwd(const gdn_lin_shape* s, const void* Q, const void* K, const void* V,
                             int32_t qkv_dtype, const float* g, const float* S0, void* O, int32_t o_dtype,
                             float* S_out, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_lin(s, false);
  if (st != GDN_OK) return st;
  if (qkv_dtype != GDN_BF16) return qkv_dtype == GDN_F32 ? GDN_ERR_UNSUPPORTED : GDN_ERR_BAD_DTYPE;
  if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  if (s->B == 0 || s->H == 0) return GDN_OK;
  if (s->T > 0 && (!Q || !K || !V || !g || !O)) return GDN_ERR_NULL_POINTER;
  if (!all_aligned16({Q, K, V, g, S0, O, S_out, s->offsets})) return GDN_ERR_BAD_ALIGNMENT;
  gdn::LinLaunch p = lin_launch(s);
  if (!gdn::lin_grid_ok(p, false)) return GDN_ERR_UNSUPPORTED;
  st = check_workspace(gdn::lin_workspace(p, false), workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.g = g;
  p.S0 = S0;
  p.O = O;
  p.o_bf16 = o_dtype == GDN_BF16;
  p.S_out = S_out;
  return launch_result(gdn::launch_lin_fwd(p, workspace, as_stream(stream)));
}

gdn_status gdn_lin_chunk_bwd(const gdn_lin_shape* s, const void* Q, const void* K, const void* V,
                             int32_t qkv_dtype, const float* g, const float* S0, const void* dO,
                             const float* dS, void* dQ, void* dK, void* dV, int32_t grad_dtype, float* dg,
                             float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_lin(s, true);
  if (st != GDN_OK) return st;
  if (qkv_dtype != GDN_BF16) return qkv_dtype == GDN_F32 ? GDN_ERR_UNSUPPORTED : GDN_ERR_BAD_DTYPE;
  if (grad_dtype != GDN_F32 && grad_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  if (s->H == 0) return GDN_OK;
  // without a sequence all rows' gradients are zero, and so are those of the heads' decays
  const bool rows = s->T > 0 && (s->B > 0 || s->offsets);
  if (rows && (!Q || !K || !V || !g || !dO || !dQ || !dK || !dV)) return GDN_ERR_NULL_POINTER;
  if (s->B == 0 && !rows && !(dg && s->g_per_head)) return GDN_OK;
  if (!all_aligned16({Q, K, V, g, S0, dO, dS, dQ, dK, dV, dg, dS0, s->offsets})) return GDN_ERR_BAD_ALIGNMENT;
  gdn::LinLaunch p = lin_launch(s);
  if (!gdn::lin_grid_ok(p, true)) return GDN_ERR_UNSUPPORTED;
  st = check_workspace(s->B > 0 ? gdn::lin_workspace(p, true) : 0, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.g = g;
  p.S0 = S0;
  p.dO = dO;
  p.dS = dS;
  p.dQ = dQ;
  p.dK = dK;
  p.dV = dV;
  p.grad_bf16 = grad_dtype == GDN_BF16;
  p.dg = dg;
  p.dS0 = dS0;
  return launch_result(gdn::launch_lin_bwd(p, workspace, as_stream(stream)));
}

gdn_status gdn_lin_decode(const gdn_lin_shape* s, const void* Q, const void* K, const void* V, int32_t qkv_dtype,
                          const float* g, const float* S_in, float* S_out, void* O, int32_t o_dtype,
                          void* stream) {
  gdn_status st = check_lin(s, false);
  if (st != GDN_OK) return st;
  if (qkv_dtype != GDN_BF16 && qkv_dtype != GDN_F32) return GDN_ERR_BAD_DTYPE;
  if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_BAD_DTYPE;
  if (s->offsets) return GDN_ERR_UNSUPPORTED;
  if (s->B == 0 || s->H == 0) return GDN_OK;
  if (!S_out || (s->T > 0 && (!Q || !K || !V || !g || !O))) return GDN_ERR_NULL_POINTER;
  if (!all_aligned16({Q, K, V, g, S_in, S_out, O})) return GDN_ERR_BAD_ALIGNMENT;
  gdn::LinDecodeLaunch p{};
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.g = g;
  p.S_in = S_in;
  p.S_out = S_out;
  p.O = O;
  p.g_per_head = s->g_per_head;
  p.B = s->B;
  p.H = s->H;
  p.H_qk = s->H_qk;
  p.n = (int)s->T;
  p.d_k = s->d_k;
  p.d_v = s->d_v;
  p.in_bf16 = qkv_dtype == GDN_BF16;
  p.o_bf16 = o_dtype == GDN_BF16;
  p.scale = s->scale;
  return launch_result(gdn::launch_lin_decode(p, as_stream(stream)));
}

// ---- the norms around the token mixer ---------------------------------------------------

static bool float_dtype(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }

static gdn_status check_gate(int32_t dtype, int32_t B, int32_t H, int64_t T, int32_t d, int64_t z_stride, int32_t act,
                             float eps) {
  if (B < 0 || H < 0 || T < 0 || d <= 0 || !(eps >= 0.f)) return GDN_ERR_BAD_SHAPE;
  if (!float_dtype(dtype)) return GDN_ERR_BAD_DTYPE;
  if (act != GDN_GATE_SILU && act != GDN_GATE_SIGMOID) return GDN_ERR_BAD_SHAPE;
  if (z_stride < (int64_t)H * d) return GDN_ERR_BAD_SHAPE;
  if (z_stride % 8 != 0) return GDN_ERR_BAD_ALIGNMENT;
  if (d % 32 != 0 || d > 256) return GDN_ERR_UNSUPPORTED;
  // row indices and the threads of a launch (at most d / 4 a row) are 32 bits
  if (H > 0 && B > 0 && T > (((int64_t)1 << 34) - 1) / d / ((int64_t)B * H)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

static gdn::GateNormLaunch gate_launch(int32_t dtype, int32_t B, int32_t H, int64_t T, int32_t d) {
  gdn::GateNormLaunch p{};
  p.bf16 = dtype == GDN_BF16;
  p.B = B;
  p.H = H;
  p.T = T;
  p.d = d;
  return p;
}

gdn_status gdn_gate_norm_fwd(const void* O, const void* Z, int64_t z_stride, const float* w, void* Y, int32_t dtype,
                             int32_t B, int32_t H, int64_t T, int32_t d, int32_t act, float eps, void* stream) {
  const gdn_status st = check_gate(dtype, B, H, T, d, z_stride, act, eps);
  if (st != GDN_OK) return st;
  if (B == 0 || H == 0 || T == 0) return GDN_OK;
  if (!O || !Z || !Y) return GDN_ERR_NULL_POINTER;
  if (!all_aligned16({O, Z, w, Y})) return GDN_ERR_BAD_ALIGNMENT;
  gdn::GateNormLaunch p = gate_launch(dtype, B, H, T, d);
  p.O = O;
  p.Z = Z;
  p.z_stride = z_stride;
  p.w = w;
  p.Y = Y;
  p.act = act;
  p.eps = eps;
  return launch_result(gdn::launch_gate_norm(p, as_stream(stream)));
}

size_t gdn_gate_norm_bwd_workspace_bytes(int32_t B, int32_t H, int64_t T, int32_t d) {
  if (H < 0 || d <= 0 || check_gate(GDN_BF16, B, H, T, d, (int64_t)H * d, GDN_GATE_SILU, 0.f) != GDN_OK) return 0;
  return gdn::gate_norm_bwd_workspace(gate_launch(GDN_BF16, B, H, T, d));
}

gdn_status gdn_gate_norm_bwd(const void* dY, const void* O, const void* Z, int64_t z_stride, const float* w, void* dO,
                             void* dZ, float* dw, int32_t dtype, int32_t B, int32_t H, int64_t T, int32_t d,
                             int32_t act, float eps, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_gate(dtype, B, H, T, d, z_stride, act, eps);
  if (st != GDN_OK) return st;
  gdn::GateNormLaunch p = gate_launch(dtype, B, H, T, d);
  const bool empty = B == 0 || H == 0 || T == 0;
  if (empty && !dw) return GDN_OK;
  if (!empty && (!dY || !O || !Z || !dO || !dZ)) return GDN_ERR_NULL_POINTER;
  if (!all_aligned16({dY, O, Z, w, dO, dZ, dw})) return GDN_ERR_BAD_ALIGNMENT;
  st = check_workspace(dw ? gdn::gate_norm_bwd_workspace(p) : 0, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  p.dY = dY;
  p.O = O;
  p.Z = Z;
  p.z_stride = z_stride;
  p.w = w;
  p.dO = dO;
  p.dZ = dZ;
  p.dw = dw;
  p.act = act;
  p.eps = eps;
  return launch_result(gdn::launch_gate_norm_bwd(p, workspace, as_stream(stream)));
}

static gdn_status check_res(int32_t x_dtype, int32_t y_dtype, int64_t rows, int32_t D, float eps) {
  if (rows < 0 || D <= 0 || !(eps >= 0.f)) return GDN_ERR_BAD_SHAPE;
  if (!float_dtype(x_dtype) || !float_dtype(y_dtype)) return GDN_ERR_BAD_DTYPE;
  if (D % 8 != 0 || D > 16384) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

static gdn::ResNormLaunch res_launch(int32_t x_dtype, int32_t y_dtype, int64_t rows, int32_t D, float alpha,
                                     float eps) {
  gdn::ResNormLaunch p{};
  p.x_bf16 = x_dtype == GDN_BF16;
  p.y_bf16 = y_dtype == GDN_BF16;
  p.rows = rows;
  p.D = D;
  p.alpha = alpha;
  p.eps = eps;
  return p;
}

gdn_status gdn_residual_norm_fwd(const void* X, int32_t x_dtype, const void* Y, int32_t y_dtype, const float* w_post,
                                 const float* s, float alpha, const float* w_pre, void* R, void* N, int64_t rows,
                                 int32_t D, float eps, void* stream) {
  const gdn_status st = check_res(x_dtype, y_dtype, rows, D, eps);
  if (st != GDN_OK) return st;
  if (rows == 0) return GDN_OK;
  if (!X || !Y || !R) return GDN_ERR_NULL_POINTER;
  if (!all_aligned16({X, Y, w_post, s, w_pre, R, N})) return GDN_ERR_BAD_ALIGNMENT;
  gdn::ResNormLaunch p = res_launch(x_dtype, y_dtype, rows, D, alpha, eps);
  p.X = X;
  p.Y = Y;
  p.w_post = w_post;
  p.s = s;
  p.w_pre = w_pre;
  p.R = R;
  p.N = N;
  return launch_result(gdn::launch_res_norm(p, as_stream(stream)));
}

size_t gdn_residual_norm_bwd_workspace_bytes(int64_t rows, int32_t D) {
  if (check_res(GDN_F32, GDN_F32, rows, D, 0.f) != GDN_OK) return 0;
  return gdn::res_norm_bwd_workspace(res_launch(GDN_F32, GDN_F32, rows, D, 0.f, 0.f));
}

gdn_status gdn_residual_norm_bwd(const void* dN, const void* dR, const void* R, int32_t x_dtype, const void* Y,
                                 int32_t y_dtype, const float* w_post, const float* s, float alpha,
                                 const float* w_pre, void* dX, void* dY, float* dw_pre, float* dw_post, float* ds,
                                 int64_t rows, int32_t D, float eps, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  gdn_status st = check_res(x_dtype, y_dtype, rows, D, eps);
  if (st != GDN_OK) return st;
  if ((dw_post && !w_post) || (ds && !s)) return GDN_ERR_NULL_POINTER;
  const bool sums = dw_pre || dw_post || ds;
  if (rows == 0 && !sums) return GDN_OK;
  if (rows > 0 && (!dX || !dY || (dN && !R) || ((w_post || ds) && !Y))) return GDN_ERR_NULL_POINTER;
  if (!all_aligned16({dN, dR, R, Y, w_post, s, w_pre, dX, dY, dw_pre, dw_post, ds})) return GDN_ERR_BAD_ALIGNMENT;
  gdn::ResNormLaunch p = res_launch(x_dtype, y_dtype, rows, D, alpha, eps);
  st = check_workspace(sums ? gdn::res_norm_bwd_workspace(p) : 0, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  p.dN = dN;
  p.dR = dR;
  p.X = R;
  p.Y = Y;
  p.w_post = w_post;
  p.s = s;
  p.w_pre = w_pre;
  p.dX = dX;
  p.dY = dY;
  p.dw_pre = dw_pre;
  p.dw_post = dw_post;
  p.ds = ds;
  return launch_result(gdn::launch_res_norm_bwd(p, workspace, as_stream(stream)));
}

}  // extern "C"

namespace gdn {

gdn_status chunk_fwd_impl(const void* Q, const void* K, const void* V, int32_t qkv_dtype,
                          const float* beta, const float* g, const float* S0, void* O,
                          int32_t o_dtype, float* S_out, int32_t B, int32_t H, int64_t T,
                          int32_t d_k, int32_t d_v, int32_t C, float scale,
                          const gdn_inverse_cfg* inv, void* workspace, size_t workspace_bytes,
                          void* (*workspace_of_device)(size_t need), gdn_fp8_stats* stats, void* stream) {
  gdn_status st = check_chunk_args(qkv_dtype, o_dtype, B, H, T, d_k, d_v, C, inv);
  if (st != GDN_OK) return st;
  if (stats && !aligned16(stats)) return GDN_ERR_BAD_ALIGNMENT;
  hipStream_t s = as_stream(stream);
  auto* st64 = reinterpret_cast<unsigned long long*>(stats);
  const bool empty = (int64_t)B * H == 0 || T == 0;
  const size_t need = empty ? 0 : chunk_workspace(B, H, T, C, inv);
  // the masked fp8 chain with N <= 3: its band pre-pass instead of the row packs
  const bool fp8_band =
      inv->mode == GDN_INV_NEUMANN && gdn::chunk_fwd_fp8_band(inv->mode, inv->N, inv->mask, inv->compute);
  if (!empty) {
    if (!Q || !K || !V || !beta || !g || !O || !S_out) return GDN_ERR_NULL_POINTER;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(beta) || !aligned16(g) ||
        !aligned16(O) || !aligned16(S_out) || (S0 && !aligned16(S0)))
      return GDN_ERR_BAD_ALIGNMENT;
    if (need > 0) {
      if (workspace_of_device) {
        // no workspace argument: the caller's resolver supplies it (NULL if need exceeds
        // what it holds, or if the HIP runtime failed; it reports which)
        if (need > workspace_bytes) return GDN_ERR_WORKSPACE;
        workspace = workspace_of_device(need);
        if (!workspace) return GDN_ERR_HIP;
      } else if (!workspace || workspace_bytes < need) {
        return GDN_ERR_WORKSPACE;
      }
      if (!aligned16(workspace)) return GDN_ERR_BAD_ALIGNMENT;
    }
  }
  if (st64) {
    gdn::launch_zero_stats(st64, s);
    if (hipGetLastError() != hipSuccess) return GDN_ERR_HIP;
  }
  if (empty) return GDN_OK;
  if (need > 0) {
    // pre-pass: T - I of every chunk as row packs, each chunk a block of the keys
    gdn::BlocksArgs ba;
    ba.A = nullptr;
    ba.K = K;
    ba.beta = beta;
    ba.g = g;
    ba.n_blocks = (int64_t)B * H * (T / C);
    ba.C = C;
    ba.d_k = d_k;
    ba.g_cumulative = 0;
    const int mode = inv->mode == GDN_INV_EXACT ? 1 : 0;  // the products of either Neumann mode
    const gdn_status pre =
        launch_result(fp8_band ? gdn::launch_band_fp8(ba, inv->N, workspace, st64, s)
                               : gdn::launch_T_packs(ba, mode, inv->N, inv->mask, inv->compute, workspace, st64, s));
    if (pre != GDN_OK) return pre;
  }
  gdn::ChunkLaunch p;
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.beta = beta;
  p.g = g;
  p.S0 = S0;
  p.O = O;
  p.S_out = S_out;
  p.packs = need > 0 ? workspace : nullptr;
  p.band_rows = fp8_band ? 1 : 0;
  p.T = T;
  p.B = B;
  p.H = H;
  p.d_k = d_k;
  p.d_v = d_v;
  p.o_bf16 = o_dtype == GDN_BF16;
  p.mode = inv->mode == GDN_INV_EXACT ? 1 : 0;
  p.N = inv->N;
  p.mask = inv->mask;
  p.cmp = inv->compute;
  p.scale = scale;
  return launch_result(gdn::launch_chunk_fwd(p, s));
}

}  // namespace gdn
