// gdn_kernels.hpp -- host-visible launch interface between the C-ABI layer (abi.cpp)
// and the kernel translation units.  Arguments are validated by abi.cpp before any
// launcher is called; launchers return 0 on success, -1 for a configuration they
// have no instantiation for (reported as GDN_ERR_UNSUPPORTED).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace gdn {

struct BlocksArgs {
  const float* A;
  const void* K;
  const float* beta;
  const float* g;
  int64_t n_blocks;
  int C;
  int d_k;
  int g_cumulative;
};

// src: 0 = A given, 1 = K bf16, 2 = K fp32.  cmp: 0 = f32, 1 = bf16, 2 = fp8.
int launch_build_A(const BlocksArgs& a, int src, float* A_out, hipStream_t s);
int launch_neumann(const BlocksArgs& a, int src, int N, int mask, int cmp, void* T_out, int t_bf16,
                   unsigned long long* stats, hipStream_t s);
int launch_exact(const BlocksArgs& a, int src, int cmp, void* T_out, int t_bf16, hipStream_t s);
void launch_zero_stats(unsigned long long* stats, hipStream_t s);
// truncated sum refined by the parallel residual correction (S Horner steps in E), fp32
int launch_residual(const BlocksArgs& a, int src, int N, int mask, int S, void* T_out, int t_bf16,
                    hipStream_t s);
// forward substitution (fp32), the sequential baseline, C <= 64
int launch_fs(const BlocksArgs& a, int src, void* T_out, int t_bf16, hipStream_t s);
// forward substitution at C = 128 (A given in fp32, or built from bf16 keys, d_k 64 or 128)
int launch_fs128(const BlocksArgs& a, int src, void* T_out, int t_bf16, hipStream_t s);

// WY products; T given (t_bf16 selects its dtype) or formed with (mode, N, mask);
// C in {32, 64}, d_k and d_v in {64, 128}
int launch_wy(const BlocksArgs& a, const void* T, int t_bf16, int mode, int N, int mask,
              const void* V, int d_v, int gate_k, void* W_out, void* U_out, int out_bf16,
              hipStream_t s);

// masked truncated Neumann with band N <= 16 for C a multiple of 64 (d_k in {64, 128}):
// T (T_out non-NULL, row-major [C][C]) or the WY products (d_v in {64, 128}); one
// wave per 16-row tile, each on its own 32-row window
int launch_band(const BlocksArgs& a, const void* V, int d_v, int N, int gate_k, void* T_out, int t_bf16,
                void* W_out, void* U_out, int out_bf16, hipStream_t s);

// full lower triangle at C in {128, 256} (d_k in {64, 128}): Neumann (any N, masked or
// not) or exact doubling, as T (T_out) or as the WY products (d_v in {64, 128}); WY
// of a given T (T_in, fp32 or bf16) too.  One workgroup of C/32 waves per block.
int launch_dense(const BlocksArgs& a, const void* T_in, int t_in_bf16, int mode, int N, int mask,
                 const void* V, int d_v, int gate_k, void* T_out, int t_bf16, void* W_out, void* U_out,
                 int out_bf16, hipStream_t s);

// T - I of every 64 x 64 block as the chunk forward's row packs (6 x 64 x 16 bytes per
// block, store_T_packs): the pre-pass of every chunk-forward variant but the band path
int launch_T_packs(const BlocksArgs& a, int mode, int N, int mask, int cmp, void* packs,
                   unsigned long long* stats, hipStream_t s);
constexpr size_t T_PACK_BYTES = 6 * 64 * 16;

struct ChunkLaunch {
  const void* Q;
  const void* K;
  const void* V;
  const float* beta;
  const float* g;
  const float* S0;
  void* O;
  float* S_out;
  const void* packs;  // T - I from the pre-pass (NULL on the band path): row packs, or
                      // with band_rows the fp8 band pre-pass's rows
  int band_rows;
  int64_t T;
  int B, H, d_k, d_v;
  int o_bf16;
  int mode, N, mask, cmp;
  float scale;
};
// chunk-wise forward, C = 64; d_k in {64, 128}; d_v a multiple of 32.  The band path
// (Neumann, mask, N <= 3, bf16) forms T - I itself; the masked fp8 chain with N <= 3 reads
// the band rows of launch_band_fp8 (p.packs, p.band_rows); every other variant reads the
// row packs of launch_T_packs (p.packs).
bool chunk_fwd_band_path(int mode, int N, int mask, int cmp);
bool chunk_fwd_fp8_band(int mode, int N, int mask, int cmp);
// the band of T - I of every 64-row chunk for the masked fp8 chain, N <= 3 (bf16 keys,
// d_k 64 or 128, raw log-gates): 64 rows x 8 bytes per chunk; stats: its counters (or NULL)
int launch_band_fp8(const BlocksArgs& a, int N, void* out, unsigned long long* stats, hipStream_t s);
constexpr size_t BAND_ROW_BYTES = 64 * 8;
int launch_chunk_fwd(const ChunkLaunch& p, hipStream_t s);
}  // namespace gdn

#include "gdn.h"
namespace gdn {
// gdn_chunk_fwd's validation and launches.  With workspace_of_device == NULL the
// workspace arguments are the caller's; otherwise workspace_bytes is the most the
// resolver can supply and the resolver returns device memory of at least `need` bytes
// for the current device (NULL if the HIP runtime failed).
gdn_status chunk_fwd_impl(const void* Q, const void* K, const void* V, int32_t qkv_dtype,
                          const float* beta, const float* g, const float* S0, void* O,
                          int32_t o_dtype, float* S_out, int32_t B, int32_t H, int64_t T,
                          int32_t d_k, int32_t d_v, int32_t C, float scale,
                          const gdn_inverse_cfg* inv, void* workspace, size_t workspace_bytes,
                          void* (*workspace_of_device)(size_t need), gdn_fp8_stats* stats, void* stream);

struct DecodeLaunch {
  const void* Q;
  const void* K;
  const void* V;
  const float* beta;
  const float* g;
  const float* S_in;  // NULL = zeros; may equal S_out
  float* S_out;
  void* O;
  int B, H, n, d_k, d_v;
  int in_bf16, o_bf16;
  float scale;
};
// gated delta rule token by token with the state resident on chip for all n tokens;
// d_k in {64, 128}, d_v a multiple of 32 up to 256
int launch_decode(const DecodeLaunch& p, hipStream_t s);

// linear attention with a decay for each head (offsets: packed sequences, n_seq of them in
// T tokens; NULL: n_seq sequences of T tokens each); d_k in {64, 128}, d_v a multiple of 32
// up to 256 (backward: in {64, 128})
struct LinLaunch {
  const void* Q;
  const void* K;
  const void* V;
  const float* g;
  const float* S0;  // NULL = zeros
  const int32_t* offsets;
  float scale;
  int g_per_head;
  int n_seq, H, H_qk, d_k, d_v;
  int64_t T;
  // forward
  void* O;
  int o_bf16;
  float* S_out;  // NULL = not wanted
  // backward
  const void* dO;
  const float* dS;  // NULL = zeros
  void* dQ;
  void* dK;
  void* dV;
  int grad_bf16;
  float* dg;
  float* dS0;  // NULL = not wanted
};
size_t lin_workspace(const LinLaunch& p, bool bwd);
bool lin_grid_ok(const LinLaunch& p, bool bwd);  // the launches' grids stay within their limits
int launch_lin_fwd(const LinLaunch& p, void* workspace, hipStream_t s);
int launch_lin_bwd(const LinLaunch& p, void* workspace, hipStream_t s);

struct LinDecodeLaunch {
  const void* Q;
  const void* K;
  const void* V;
  const float* g;
  const float* S_in;  // NULL = zeros; may equal S_out
  float* S_out;
  void* O;
  int g_per_head, B, H, H_qk, n, d_k, d_v;
  int in_bf16, o_bf16;
  float scale;
};
int launch_lin_decode(const LinDecodeLaunch& p, hipStream_t s);

// gated norm of head outputs: O [B][H][T][d], Z and dZ [B][T] rows of H * d (Z's at stride
// z_stride), Y and dY [B][T][H][d]; d a multiple of 32 up to 256
struct GateNormLaunch {
  const void* O;
  const void* Z;
  const float* w;  // NULL = ones
  void* Y;
  const void* dY;
  void* dO;
  void* dZ;
  float* dw;  // NULL = not wanted
  int bf16;
  int act;
  int B, H, d;
  int64_t T, z_stride;
  float eps;
};
size_t gate_norm_bwd_workspace(const GateNormLaunch& p);
int launch_gate_norm(const GateNormLaunch& p, hipStream_t s);
int launch_gate_norm_bwd(const GateNormLaunch& p, void* workspace, hipStream_t s);

// residual sum with the norms before and after: [rows][D], D a multiple of 8 up to 16384
struct ResNormLaunch {
  const void* X;  // backward: R
  const void* Y;
  const float* w_post;
  const float* s;
  const float* w_pre;
  void* R;
  void* N;
  const void* dN;
  const void* dR;
  void* dX;
  void* dY;
  float* dw_pre;
  float* dw_post;
  float* ds;
  int x_bf16, y_bf16;
  int64_t rows;
  int D;
  float alpha, eps;
};
size_t res_norm_bwd_workspace(const ResNormLaunch& p);
int launch_res_norm(const ResNormLaunch& p, hipStream_t s);
int launch_res_norm_bwd(const ResNormLaunch& p, void* workspace, hipStream_t s);
// out0, out1 [D] = the sums over k < n of part[k][0][i] and part[k][1][i] (n_in 1 or 2), in order, in fp64
// (norm.hip; NULL = not wanted)
void launch_column_sum(const float* part, int64_t n, int D, int n_in, float* out0, float* out1, hipStream_t s);

// gated linear recurrence of every channel (offsets: packed sequences, n_seq of them in T tokens;
// NULL: n_seq sequences of T tokens each); D a multiple of 8
constexpr int64_t REC_MAX_STRIDE = (int64_t)1 << 24;  // values between tokens
struct RecLaunch {
  const void* X;
  const void* A;
  const void* I;       // NULL = no input gate
  const float* w;      // decay GDN_DECAY_POWER
  const float* h0;     // NULL = zeros
  const int32_t* offsets;
  int64_t x_stride, a_stride, i_stride;
  int64_t T, n_states; // of a row: T tokens, the states at every GDN_REC_TILE-th of them
  int n_seq, D;
  int decay, norm, bf16;
  // forward and step
  void* H;
  float* h_out;        // NULL = not wanted
  float* states;       // [rows][n_states][D]; forward: NULL = not wanted, backward: NULL = not given
  // backward
  const void* dH;
  const float* dh;     // NULL = zeros
  void* dX;
  void* dA;
  void* dI;
  float* dw;           // NULL = not wanted
  float* dh0;          // NULL = not wanted
  // set by the launchers: a row's tiles and, in the workspace, what links them
  int64_t tiles;
  uint64_t* chain_tiles;
  uint64_t* chain_eights;
  uint64_t* chain_states;
  uint32_t* tickets;
  float* part;
};
size_t rec_workspace(const RecLaunch& p, bool bwd);
bool rec_grid_ok(const RecLaunch& p);  // the launches' grids stay within their limits
bool rec_step_grid_ok(const RecLaunch& p);
int launch_rec_fwd(const RecLaunch& p, void* workspace, hipStream_t s);
int launch_rec_bwd(const RecLaunch& p, void* workspace, hipStream_t s);
int launch_rec_step(const RecLaunch& p, hipStream_t s);

// norm and rotation of query and key heads: Q_in, K_in [B][T] rows of heads at their strides, Q, K
// [B][H][T][d]; d a multiple of 32 up to 256, rot a multiple of 8 up to d
struct QkLaunch {
  const void* Q_in;
  const void* K_in;
  int64_t q_stride, k_stride;
  const float* wq;  // NULL = ones
  const float* wk;
  const double* freqs;
  const int32_t* positions;  // NULL = the token's index
  void* Q;  // backward: dQ_in, dK_in [B][T][H][d]
  void* K;
  const void* dQ;  // [B][H][T][d]
  const void* dK;
  float* dwq;  // NULL = not wanted
  float* dwk;
  int64_t T;
  int B, Hq, Hk, d;
  int norm, rot, halves, bf16;
  float eps;
  uint8_t axis[GDN_QK_MAX_PAIRS];
};
size_t qk_bwd_workspace(const QkLaunch& p);
int launch_qk(const QkLaunch& p, hipStream_t s);
int launch_qk_bwd(const QkLaunch& p, void* workspace, hipStream_t s);
}  // namespace gdn
