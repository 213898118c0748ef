// lin.hip -- linear attention with a decay for each head, chunk-wise: forward and backward.
//
// Per sequence and value head, tokens in order, g_t the log-decays, S [d_k][d_v] fp32:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,     o_t = scale S_t^T q_t
// (the gated recurrence without the delta correction).  In chunks of 64 tokens, with G the
// in-chunk cumulative sum of g, S the state before the chunk and D the gradient of the loss
// with respect to the state after it:
//   O_i  = scale (sum_{j<=i} e^{G_i-G_j} (q_i . k_j)  v_j  + e^{G_i} q_i S)
//   dQ_i = scale (sum_{j<=i} e^{G_i-G_j} (do_i . v_j) k_j  + e^{G_i} do_i S^T)
//   dV_i = scale sum_{j>=i} e^{G_j-G_i} (k_i . q_j)  do_j + e^{G_C-G_i} k_i D
//   dK_i = scale sum_{j>=i} e^{G_j-G_i} (v_i . do_j) q_j  + e^{G_C-G_i} v_i D^T
//   S   <- e^{G_C} S + sum_j e^{G_C-G_j} k_j v_j^T
//   D   <- e^{G_C} D + scale sum_j e^{G_j} q_j do_j^T          (chunks from last to first)
// All four are one scan over row operands a, column operands b and values c,
//   out_i = sum_j w_ij (a_i . b_j) c_j + row_i a_i X,   X <- e^{G_C} X + sum_j col_j b_j c_j^T,
// run forwards for O and dQ and backwards for dV and dK; one kernel serves them all.
//
// Gradient of the log-decays: with r_t = q_t . dq_t - k_t . dk_t, dg_t = sum_{s>=t} r_s over
// the rest of the sequence + <dS_out, S_out>.  Summed over a whole long sequence the
// differences r_s would lose digits, so the sum runs within a segment of at most 1024 tokens,
// between <D, S> at the segment's two ends, formed from the states there.  The products q . dq and
// k . dk are summed in fp64 from four terms on.
//
// Precision: a, b and c are bf16 as given, so a . b is exact up to the fp32 sums of the MFMA.
// The fp32 factor of every other product (col c of the state, X and w (a . b) of the outputs)
// enters as a sum of three bf16 parts, which hold all 24 bits.  The state is carried from chunk
// to chunk in fp32 and returned so, and an output in bf16 is the one in fp32 rounded once: its
// type changes no product.  For bf16 outputs one part of X and two of w (a . b) would take 169
// instead of 217 us on the prefill workload, two of both 203; but where decays are slow one part
// leaves O at 0.0023 in the norm (0.0017 is its own rounding), and two leave 1e-5 in dg, the
// small difference of products with q and k, where three leave 4e-7.  G is summed in fp64 and
// handed over as two floats: the exponent of w is a difference of two sums that can both be
// large.
//
// Work split: one workgroup per (segment, head, W columns of c), W = 32, 64 or 128.
//   column waves  32 columns each at W = 128, else 16: they keep their columns of X in
//                 registers, form a X, then split col c and update X, and after the barrier in
//                 the middle of a chunk add w (a . b) c and store.
//   weight waves  two: w (a . b) for row tiles 0 and 3, 1 and 2, handed over through LDS.
//   one wave forms the next chunk's decay factors, one loads its rows of a, b and c straight
//   into LDS.
// What a workgroup does per chunk whatever its columns (w (a . b), the rows of a and b) is
// shared by W columns, so wide workgroups take fewer instructions: B4 H16 T8192 d128 takes 305 us
// as 256 workgroups of 32 columns over whole sequences, 217 as 256 of 128 columns over quarters,
// their states formed first.  A segment is a run of chunks of one sequence: where sequences and
// heads alone fill the GPU a segment is a whole sequence; else each segment's own state is
// formed first (the same kernel without outputs), the segments are joined in order, and every
// segment then starts from its state.
//
// What bounds it: the issue of the column waves, and where they wait for the weights in the middle
// of a chunk.  A chunk of a column wave of 32 columns at d_k = 128 is 228 MFMA (3650 cycles) on one
// SIMD, which its vector instructions overlap little, and takes 4.2 us (10000 cycles).  256 heads of
// 2048 tokens, whole sequences (537 MB), take 158 us, 3.4 TB/s; the states alone reach 3.6 to 3.9.
// Measured, whole calls:
//   forward   B4 H16 T8192 d128                212-220 us (800 MB moved; the segments' states, which
//                                              read K and V again, 56)
//             B1 H8 T32768 d128                111-122 us
//             13 packed, 11171 tokens, H16 128 x 256   189-194 us (uneven segments)
//   backward  B4 H16 T4096 d128                320-334 us
//             7 packed, 5003 tokens, H12 64 x 128      113 us (one round of 5 chunks in each of
//                                              five scans, ten launches)
#include "gdn_kernels.hpp"
#include "gdn_device.hpp"

namespace gdn {

namespace {

constexpr int LC = 64;     // tokens of a chunk
constexpr int LNT = 4;     // 16-row tiles of a chunk
constexpr int PARTS = 3;   // bf16 parts of an fp32 factor: 24 bits
constexpr int BWD_SEG_CHUNKS = 16;  // at most 1024 tokens are summed into dg from one pair of states
constexpr int JOIN_GROUPS = 2048;    // 256 CUs with eight workgroups each
constexpr double LOG2E = 1.4426950408889634;

// How sequences are cut into segments, runs of chunks that one workgroup (for some columns) walks
struct Cut {
  const int32_t* offsets;  // packed sequences
  int64_t T;
  int n_seq;
  int chunks;    // of a segment
  int segments;  // of a sequence (packed: at most, not used)
  int n_seg;     // of all sequences (packed: at most)
};

struct ScanArgs {
  const __bf16* a;
  const __bf16* b;
  const __bf16* c;
  const float* g;
  const float* init;   // states given per sequence (NULL: zeros)
  float* fin;          // states returned per sequence (NULL: not wanted)
  float* slot;         // states of the segments (workspace); written without OUT, read with
  float* slot_decay;   // [segment][head] decay over the segment, written without OUT
  void* out;
  const __bf16* dotw;  // rows whose product with the output rows goes to dots,
  double* dots;        // [head row] (one slice)
  int H, group_a, group_b, group_c, dc;
  Cut cut;
  int g_per_head;
  int skip;            // without OUT: a sequence's end segment is not wanted
  float s_intra, s_inter, s_state;
};

// 64 rows of D values in LDS, without padding (they arrive by direct loads, 1 KB an instruction
// in lane order).  The 16-byte pieces of row r are permuted by r so that the readers spread over
// the banks: 16 consecutive rows at one piece, and 4 rows x 4 pieces by the transpose read.
template <int D>
struct alignas(16) LinRows {
  __bf16 v[LC * D];
  static __device__ __forceinline__ int mix(int r) {
    // low two bits by r / 4: 0, 2, 3, 1, so that rows r and r ^ 4 at neighbouring pieces do not
    // meet either (in order: three times the bank conflicts, and 1 % of the prefill's time)
    const int b = (r >> 2) & 3, low = ((b ^ (b << 1)) & 2) | (b >> 1);
    return D == 128 ? ((r & 3) << 2) | low : D == 64 ? (((r >> 1) & 1) << 2) | low : (r >> 1) & 2;
  }
  // where element d of row r lies (d a multiple of 4: the rest of its piece follows)
  static __device__ __forceinline__ int at(int r, int d) { return r * D + 8 * ((d >> 3) ^ mix(r)) + (d & 7); }
  // byte offset in memory of what lane l of load i brings, rows being stride values apart
  static __device__ __forceinline__ int source(int i, int l, int stride) {
    const int e = i * 512 + l * 8, r = e / D, piece = (e % D) / 8;
    return (r * stride + 8 * (piece ^ mix(r))) * 2;
  }
};

struct alignas(16) LinGates {
  float hi[LC], lo[LC];         // G in units of log 2, as a sum of two floats
  float row[LC];                // factor of a_i X
  float col[LC];                // factor of b_j c_j^T
  float from[LNT - 1][LC];      // w of j to the boundary of a tile,
  float to[LC];                 // and from the row's boundary to the row, with the scale
  float end;                    // e^{G_C}
};

// one segment: nc chunks from chunk c0 on of a sequence of len tokens from token tok0 on
struct Span {
  int64_t tok0;
  int len, seq, c0, nc;
  bool first, last;
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ int wave_scan_int(int v) {
#pragma unroll
  for (int d = 1; d < WAVE; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane_id() >= d) v += o;
  }
  return v;
}

// offsets outside [0, T] or out of order are clamped, so that no access leaves the tensors
__device__ __forceinline__ void seq_bounds(const int32_t* off, int s, int64_t T, int& o0, int& o1) {
  const int t = (int)T;
  o0 = min(max(off[s], 0), t);
  o1 = min(max(off[s + 1], o0), t);
}

__device__ __forceinline__ int segment_count(int len, int chunks) {
  const int nch = (len + LC - 1) / LC;
  return max(1, (nch + chunks - 1) / chunks);
}

__device__ __forceinline__ void cut_span(const Cut& c, int k, int n, Span& sp) {
  const int nch = (sp.len + LC - 1) / LC;
  sp.c0 = k * c.chunks;
  sp.nc = min(c.chunks, nch - sp.c0);
  sp.first = k == 0;
  sp.last = k == n - 1;
}

// the segment of index seg; false: there are fewer (packed sequences: the grid is an upper
// bound), or offsets out of order make more than there can be
__device__ __forceinline__ bool find_segment(const Cut& c, int seg, Span& sp) {
  if (!c.offsets) {
    sp.seq = seg / c.segments;
    sp.tok0 = 0;
    sp.len = (int)c.T;
    cut_span(c, seg % c.segments, c.segments, sp);
    return true;
  }
  int base = 0;
  for (int s0 = 0; s0 < c.n_seq; s0 += WAVE) {
    const int s = s0 + lane_id();
    int o0 = 0, o1 = 0, n = 0;
    if (s < c.n_seq) {
      seq_bounds(c.offsets, s, c.T, o0, o1);
      n = segment_count(o1 - o0, c.chunks);
    }
    const int inc = wave_scan_int(n);
    const uint64_t m = __builtin_amdgcn_ballot_w64(base + inc > seg);
    if (m) {
      const int src = __builtin_ctzll(m);
      const int a0 = __builtin_amdgcn_readlane(o0, src), a1 = __builtin_amdgcn_readlane(o1, src);
      const int ns = __builtin_amdgcn_readlane(n, src), end = base + __builtin_amdgcn_readlane(inc, src);
      sp.seq = s0 + src;
      sp.tok0 = a0;
      sp.len = a1 - a0;
      cut_span(c, seg - (end - ns), ns, sp);
      return end <= c.n_seg;
    }
    base += __builtin_amdgcn_readlane(inc, WAVE - 1);
  }
  return false;
}

// index of a sequence's first segment, and how many it has
__device__ __forceinline__ int first_segment(const Cut& c, int seq, int& ns) {
  if (!c.offsets) {
    ns = c.segments;
    return seq * c.segments;
  }
  int base = 0;
  for (int s0 = 0; s0 < seq; s0 += WAVE) {
    const int s = s0 + lane_id();
    int n = 0, o0, o1;
    if (s < seq) {
      seq_bounds(c.offsets, s, c.T, o0, o1);
      n = segment_count(o1 - o0, c.chunks);
    }
    base += __builtin_amdgcn_readlane(wave_scan_int(n), WAVE - 1);
  }
  int o0, o1;
  seq_bounds(c.offsets, seq, c.T, o0, o1);
  ns = segment_count(o1 - o0, c.chunks);
  return base;
}

template <int CTRL>
__device__ __forceinline__ double dpp_d(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  const unsigned lo = w[0], hi = w[1];
  return __builtin_bit_cast(double, u32x2{dpp_u<CTRL>(lo), dpp_u<CTRL>(hi)});
}
__device__ __forceinline__ double readlane_d(double x, int lane) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  const int lo = (int)w[0], hi = (int)w[1];
  return __builtin_bit_cast(double, u32x2{(unsigned)__builtin_amdgcn_readlane(lo, lane),
                                          (unsigned)__builtin_amdgcn_readlane(hi, lane)});
}
// inclusive prefix sum over the 64 lanes: shifts within each row of 16 (lanes that would read
// across its start add 0), then the totals of the rows before
__device__ __forceinline__ double wave_scan_f64(double v) {
  v += dpp_d<0x111>(v);
  v += dpp_d<0x112>(v);
  v += dpp_d<0x114>(v);
  v += dpp_d<0x118>(v);
  const double t0 = readlane_d(v, 15), t1 = readlane_d(v, 31), t2 = readlane_d(v, 47);
  const int row = lane_id() >> 4;
  return v + ((row >= 1 ? t0 : 0.0) + (row >= 2 ? t1 : 0.0) + (row >= 3 ? t2 : 0.0));
}

// sum over lanes l ^ W (16 or 32)
template <int W>
__device__ __forceinline__ double swap_sum_d(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  uint32_t lo[2], hi[2];
  self_swap<W>(w[0], lo[0], lo[1]);
  self_swap<W>(w[1], hi[0], hi[1]);
  return __builtin_bit_cast(double, u32x2{lo[0], hi[0]}) + __builtin_bit_cast(double, u32x2{lo[1], hi[1]});
}

// log-decays below 2^-512 are e^g = 0 in every product: clamped, so that -inf (a state that is
// forgotten) keeps the differences of G finite.  A NaN stays one.
__device__ __forceinline__ double clamp_log2(double x) { return x < -512.0 ? -512.0 : x; }

__device__ __forceinline__ float exp2_f32(float x) { return __builtin_amdgcn_exp2f(x); }
// 2^x with the whole part set apart before the fraction becomes a float: rounding an exponent
// of -10 to a float alone costs 3e-7 of the result
__device__ __forceinline__ float exp2_f64(double x) {
  const double n = rint(x);
  return ldexpf(exp2_f32((float)(x - n)), (int)n);
}

__device__ __forceinline__ f32x4 lo4(const bf16x8& v) { return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]}; }
__device__ __forceinline__ f32x4 hi4(const bf16x8& v) { return f32x4{(float)v[4], (float)v[5], (float)v[6], (float)v[7]}; }

// two tiles as the sum of N bf16 operands
template <int N>
__device__ __forceinline__ void split(f32x4 a, f32x4 b, bf16x8 (&s)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    s[k] = pack8(a, b);
    if (k + 1 < N) {
      a = a - lo4(s[k]);
      b = b - hi4(s[k]);
    }
  }
}

// x as the sum of three bf16 values, exactly: each part is the upper half of what is left (no
// rounding, so 8 + 8 + 8 bits hold all 24), and one byte permute packs the parts of two values
__device__ __forceinline__ void split3_exact(const float (&x)[8], bf16x8 (&s)[3]) {
  uint32_t w[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t ua = __builtin_bit_cast(uint32_t, a), ub = __builtin_bit_cast(uint32_t, b);
      w[k][i] = __builtin_amdgcn_perm(ub, ua, 0x07060302);
      a -= __builtin_bit_cast(float, ua & 0xffff0000u);
      b -= __builtin_bit_cast(float, ub & 0xffff0000u);
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) s[k] = __builtin_bit_cast(bf16x8, u32x4{w[k][0], w[k][1], w[k][2], w[k][3]});
}

// A run of rows as a buffer: loads past its end give 0 and stores there do nothing, so the
// last, shorter chunk of a sequence needs no code of its own.  base and bytes are uniform.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t r, int off) {
  const unsigned x = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  return __builtin_bit_cast(float, x);
}
__device__ __forceinline__ void store16b(__amdgpu_buffer_rsrc_t r, int off, const u32x4& x) {
  __builtin_amdgcn_raw_buffer_store_b128(x, r, off, 0, 0);
}
__device__ __forceinline__ void store8b(__amdgpu_buffer_rsrc_t r, int off, const bf16x4& x) {
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), r, off, 0, 0);
}
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, int off, double x) {
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), r, off, 0, 0);
}
// 16 bytes a lane straight to LDS, at p + 16 bytes x lane (p uniform)
__device__ __forceinline__ void load16_lds(__amdgpu_buffer_rsrc_t r, __bf16* p, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)p, 16, off, 0, 0, 0);
}
// until all of this wave's vector memory operations are done
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// two adjacent 16-column tiles of a row as bf16, 16 contiguous bytes per lane: group g then
// holds columns 16(g % 2) + 8(g / 2) .. + 7
__device__ __forceinline__ u32x4 pair_bf16(const f32x4& a0, const f32x4& a1) {
  const bf16x4 h0 = pack4(a0), h1 = pack4(a1);
  const u32x2 w0 = __builtin_bit_cast(u32x2, h0), w1 = __builtin_bit_cast(u32x2, h1);
  u32x4 v;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const unsigned x0 = w0[k], x1 = w1[k];  // vector elements to scalars before any bit cast
    const auto sw = __builtin_amdgcn_permlane16_swap(x0, x1, false, false);
    const unsigned y0 = sw[0], y1 = sw[1];
    v[k] = y0;
    v[2 + k] = y1;
  }
  return v;
}

// d of the state tile's row 4g + r: two tiles 2p, 2p + 1 of a lane are then the natural-order
// operand (slot t <-> d = 32p + 8g + t)
__device__ __forceinline__ int state_dim(int a, int g, int r) { return 32 * (a >> 1) + 8 * g + 4 * (a & 1) + r; }

__device__ __forceinline__ void lds_handover() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace

// waves of a workgroup of W columns: column waves, two that form w (a . b) (with outputs), one
// for the decay factors, one for the loads.  A column wave of 32 columns reads the rows of a
// and b once for both 16-column tiles; below 128 columns the waves would be too few.
constexpr int scan_tiles(int W) { return W == 128 ? 2 : 1; }
constexpr int scan_waves(int W, bool out) { return W / (16 * scan_tiles(W)) + (out ? 4 : 2); }
// waves a SIMD has to hold: those of one workgroup, of two without outputs
constexpr int scan_per_simd(int W, bool out) { return (scan_waves(W, out) * (out ? 1 : 2) + 3) / 4; }

template <int DK, int W, bool REV, bool OUT, bool DOTS, class TO>
__global__ __launch_bounds__(scan_waves(W, OUT) * WAVE, scan_per_simd(W, OUT)) void lin_scan_kernel(ScanArgs A) {
  // two slots of everything: one in use, one being filled
  __shared__ LinRows<DK> rows_a[OUT ? 2 : 1], rows_b[2];
  __shared__ LinRows<W> rows_c[2], rows_w[DOTS ? 2 : 1];
  __shared__ LinGates gates[2];
  __shared__ bf16x8 weights[OUT ? PARTS : 1][LNT][2][WAVE];  // w (a . b) as operands: [part][row tile][32-wide step]
  __shared__ double dot_part[DOTS ? W / (16 * scan_tiles(W)) : 1][LC];
  constexpr int HC = scan_tiles(W), COLS = W / (16 * HC), NP = DK / 32;
  constexpr int W_GATES = COLS + (OUT ? 2 : 0), W_ROWS = W_GATES + 1;

  // workgroup -> (segment, head, slice).  Workgroups are dealt round-robin over the 8 XCDs;
  // those that share rows (the slices of a head, the heads of a group) come one after another
  // on one XCD, so that its L2 has the rows once, and such families alternate between XCDs, so
  // that long and short segments mix.
  const int n_slices = A.dc / W;
  const int family = n_slices * (A.group_a > A.group_c ? A.group_a : A.group_c);
  const int turn = (int)(blockIdx.x / 8);
  const int idx = (turn / family * 8 + (int)(blockIdx.x % 8)) * family + turn % family;
  if (idx >= A.cut.n_seg * A.H * n_slices) return;
  const int slice = idx % n_slices, head = (idx / n_slices) % A.H, seg = idx / (n_slices * A.H);
  Span sp;
  if (!find_segment(A.cut, seg, sp)) return;
  if (!OUT && A.skip && (REV ? sp.first : sp.last)) return;

  const int wave = uniform(threadIdx.x / WAVE);
  const int l = lane_id(), g = l >> 4, c = l & 15;
  const int n = sp.nc;
  // first row of the sequence in each tensor ([B][heads][T][.], or [heads][T][.] packed)
  const int64_t batch = A.cut.offsets ? 0 : sp.seq;
  auto row_of = [&](int group) {
    const int heads = A.H / group;
    return (batch * heads + head / group) * A.cut.T + sp.tok0;
  };
  // chunk j of the scan: its first token, clamped to the segment, and the rows it has
  auto token_of = [&](int j) {
    j = min(j, n - 1);
    return LC * (REV ? sp.c0 + n - 1 - j : sp.c0 + j);
  };
  auto chunk_rows = [&](const void* base, int64_t row0, int j, int row_bytes) {
    const int t0 = token_of(j);
    return row_buffer(reinterpret_cast<const char*>(base) + (row0 + t0) * row_bytes, min(LC, sp.len - t0) * row_bytes);
  };
  const int64_t head_state = (int64_t)DK * A.dc;
  const int64_t crow = row_of(A.group_c), orow = row_of(1);

  if (wave < COLS) {
    // ---- column waves: their columns of X, in registers from the segment's start to its end --
    constexpr int NA = DK / 16;  // 16-row state tiles
    const int col0 = 16 * HC * wave;
    const int64_t col = slice * W + col0 + c;
    const float* from = nullptr;  // the state this segment starts from (NULL: zeros)
    float* to = nullptr;
    if (!OUT) {
      to = A.slot + ((int64_t)seg * A.H + head) * head_state;
    } else {
      if (!(REV ? sp.last : sp.first))
        from = A.slot + ((int64_t)(REV ? seg + 1 : seg - 1) * A.H + head) * head_state;
      else if (A.init)
        from = A.init + ((int64_t)sp.seq * A.H + head) * head_state;
      if ((REV ? sp.first : sp.last) && A.fin) to = A.fin + ((int64_t)sp.seq * A.H + head) * head_state;
    }
    // states lie [d_k][d_v]: rows of X by columns, or (dQ, dK) columns of X by rows, where a
    // lane's four rows are 16 contiguous bytes
    f32x4 X[HC][NA];
#pragma unroll
    for (int h = 0; h < HC; ++h)
#pragma unroll
      for (int t = 0; t < NA; ++t) {
        X[h][t] = zero4();
        if (!from) continue;
        if constexpr (DOTS) {
          X[h][t] = *reinterpret_cast<const f32x4*>(from + (col + 16 * h) * DK + state_dim(t, g, 0));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) X[h][t][r] = from[(int64_t)state_dim(t, g, r) * A.dc + col + 16 * h];
        }
      }
    if (n > 0) {
      // rows of a as operands: lane (g, c) reads row 16I + c, 16 bytes at 32p + 8g
      int a_at[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) a_at[p] = LinRows<DK>::at(c, 32 * p + 8 * g);
      // transposed rows of b: lane addresses of state tiles (t, t + 1) for even t; of c
      const int tr_row = 4 * g + (c >> 2);
      int bt_at[NA / 2], ct_at[HC], w_at[HC];
#pragma unroll
      for (int t = 0; t < NA / 2; ++t) bt_at[t] = LinRows<DK>::at(tr_row, 32 * t + 8 * (c & 3));
#pragma unroll
      for (int h = 0; h < HC; ++h) {
        ct_at[h] = LinRows<W>::at(tr_row, col0 + 16 * h + 4 * (c & 3));
        w_at[h] = LinRows<W>::at(c, col0 + 16 * h + 4 * g);
      }
      constexpr bool PAIR = HC == 2 && sizeof(TO) == 2;  // 16 bytes a lane from two tiles
      const int ooff = (c * A.dc + slice * W + col0 + (PAIR ? 16 * (g & 1) + 8 * (g >> 1) : 4 * g)) * (int)sizeof(TO);
      lds_handover();
      for (int it = 0; it < n; ++it) {
        const LinGates& GT = gates[it & 1];
        const __bf16* bs = rows_b[it & 1].v;
        const __bf16* cs = rows_c[it & 1].v;
        // a X: lane (g, c) holds row 16I + c, columns 4g + r of each tile.  The smaller parts have
        // sums of their own, so that the sums of the first part round only as often as they have
        // terms (dg on the training workload: 1.2e-6 with one sum).
        f32x4 o[HC][LNT], low[HC][LNT];
        if constexpr (OUT) {
          const __bf16* as = rows_a[it & 1].v;
#pragma unroll
          for (int h = 0; h < HC; ++h)
#pragma unroll
            for (int I = 0; I < LNT; ++I) o[h][I] = low[h][I] = zero4();
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            bf16x8 s[HC][PARTS];
#pragma unroll
            for (int h = 0; h < HC; ++h) split<PARTS>(X[h][2 * p], X[h][2 * p + 1], s[h]);
#pragma unroll
            for (int I = 0; I < LNT; ++I) {
              const bf16x8 af = *reinterpret_cast<const bf16x8*>(as + a_at[p] + 16 * I * DK);
#pragma unroll
              for (int h = 0; h < HC; ++h) {
#pragma unroll
                for (int k = PARTS - 1; k > 0; --k) low[h][I] = mma_bf16(s[h][k], af, low[h][I]);
                o[h][I] = mma_bf16(s[h][0], af, o[h][I]);
              }
            }
          }
        }
        // X <- e^{G_C} X + b^T (col c), col c as three parts
        const float end = GT.end;
        bf16x8 cf[HC][2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const f32x4 w0 = *reinterpret_cast<const f32x4*>(&GT.col[32 * p + 4 * g]);
          const f32x4 w1 = *reinterpret_cast<const f32x4*>(&GT.col[32 * p + 16 + 4 * g]);
          bf16x8 u[HC][3];
#pragma unroll
          for (int h = 0; h < HC; ++h) {
            const bf16x4 c0 = lds_read_tr4(cs + ct_at[h] + 32 * p * W), c1 = lds_read_tr4(cs + ct_at[h] + (32 * p + 16) * W);
            cf[h][p] = join8(c0, c1);
            const f32x4 y0 = unpack4(c0) * w0, y1 = unpack4(c1) * w1;
            const float y[8] = {y0[0], y0[1], y0[2], y0[3], y1[0], y1[1], y1[2], y1[3]};
            split3_exact(y, u[h]);
          }
#pragma unroll
          for (int t = 0; t < NA; ++t) {
            const __bf16* q = bs + bt_at[t / 2] + 32 * p * DK + 4 * (t & 1);
            const bf16x8 bt = join8(lds_read_tr4(q), lds_read_tr4(q + 16 * DK));
#pragma unroll
            for (int h = 0; h < HC; ++h) {
              if (p == 0) X[h][t] = X[h][t] * end;
#pragma unroll
              for (int k = 2; k >= 0; --k) X[h][t] = mma_bf16(bt, u[h][k], X[h][t]);
            }
          }
        }
        if constexpr (OUT) {
#pragma unroll
          for (int I = 0; I < LNT; ++I) {
            const float rw = GT.row[16 * I + c];
#pragma unroll
            for (int h = 0; h < HC; ++h) {
              o[h][I] = o[h][I] * rw;
              low[h][I] = low[h][I] * rw;
            }
          }
          lds_handover();  // the weights are there
          // Rows of V behind row i reach it with weight 0, which leaves a finite row out but not
          // an infinity or a NaN (the rows that pad a batch may hold anything).  Any such value is
          // in every row of its column of the new state; the sums then run row by row.
          bool plain = true;
          if constexpr (!REV && !DOTS) {
            float x = X[0][0][0];
            if constexpr (HC > 1) x += X[1][0][0];
            plain = __builtin_amdgcn_ballot_w64(!(fabsf(x) < __builtin_inff())) == 0;
          }
          if (plain) {
#pragma unroll
            for (int I = 0; I < LNT; ++I)
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                if (REV ? 2 * p + 1 < I : 2 * p > I) continue;
#pragma unroll
                for (int k = PARTS - 1; k >= 0; --k) {
                  const bf16x8 wf = weights[k][I][p][l];
#pragma unroll
                  for (int h = 0; h < HC; ++h) {
                    f32x4& sum = k > 0 ? low[h][I] : o[h][I];
                    sum = mma_bf16(cf[h][p], wf, sum);
                  }
                }
              }
          } else {
            for (int j = 0; j < LC; ++j)
#pragma unroll
              for (int I = 0; I < LNT; ++I) {
                if (j > 16 * I + 15) continue;
                float wj = 0.f;
#pragma unroll
                for (int k = PARTS - 1; k >= 0; --k)
                  wj += (float)weights[k][I][j / 32][16 * (j % 16 / 4) + c][4 * (j % 32 / 16) + j % 4];
#pragma unroll
                for (int h = 0; h < HC; ++h) {
                  const f32x4 v = unpack4(*reinterpret_cast<const bf16x4*>(cs + LinRows<W>::at(j, col0 + 16 * h + 4 * g)));
                  if (j <= 16 * I + c) o[h][I] = o[h][I] + wj * v;
                }
              }
          }
#pragma unroll
          for (int h = 0; h < HC; ++h)
#pragma unroll
            for (int I = 0; I < LNT; ++I) o[h][I] = o[h][I] + low[h][I];
          const auto r = chunk_rows(A.out, orow, it, (int)sizeof(TO) * A.dc);  // rows past the end are not stored
#pragma unroll
          for (int I = 0; I < LNT; ++I) {
            if constexpr (DOTS) {
              // four terms in fp32, the sums of these in fp64 (dg on the training workload: 1.07e-6
              // with fp32 throughout)
              double s = 0.0;
#pragma unroll
              for (int h = 0; h < HC; ++h) {
                const f32x4 w = unpack4(*reinterpret_cast<const bf16x4*>(rows_w[it & 1].v + w_at[h] + 16 * I * W));
                float four = w[0] * o[h][I][0];
#pragma unroll
                for (int q = 1; q < 4; ++q) four = fmaf(w[q], o[h][I][q], four);
                s += (double)four;
              }
              s = swap_sum_d<32>(swap_sum_d<16>(s));
              if (g == 0) dot_part[wave][16 * I + c] = s;
            }
            const int at = ooff + 16 * I * A.dc * (int)sizeof(TO);
            if constexpr (PAIR) {
              store16b(r, at, pair_bf16(o[0][I], o[HC - 1][I]));
            } else {
#pragma unroll
              for (int h = 0; h < HC; ++h) {
                if constexpr (sizeof(TO) == 2)
                  store8b(r, at + 32 * h, pack4(o[h][I]));
                else
                  store16b(r, at + 64 * h, __builtin_bit_cast(u32x4, o[h][I]));
              }
            }
          }
        }
        lds_handover();
      }
    }
    if (!DOTS && to) {
#pragma unroll
      for (int h = 0; h < HC; ++h)
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) to[(int64_t)state_dim(t, g, r) * A.dc + col + 16 * h] = X[h][t][r];
    }
    return;
  }
  if (wave == W_GATES) {
    // ---- decay factors, one chunk ahead (lane = token) ----------------------------------
    double decay = 0.0;  // sum of G_C over the segment
    const float g_head = n > 0 && A.g_per_head ? A.g[head] : 0.f;  // without tokens g may be NULL
    auto load = [&](int j) {
      const int t0 = token_of(j);
      if (A.g_per_head) return t0 + l < sp.len ? g_head : 0.f;
      return load4(row_buffer(A.g + orow + t0, min(LC, sp.len - t0) * 4), 4 * l);  // 0 past the end
    };
    auto store = [&](float gl, LinGates& GT) {
      const double G = wave_scan_f64(clamp_log2((double)gl * LOG2E)), GC = readlane_d(G, WAVE - 1);
      const float hi = (float)G;
      const float eG = exp2_f64(G), eR = exp2_f64(GC - G);
      GT.col[l] = (REV ? eG : eR) * A.s_state;
      if (l == 0) GT.end = exp2_f64(GC);
      if constexpr (OUT) {
        GT.hi[l] = hi;
        GT.lo[l] = (float)(G - (double)hi);
        GT.row[l] = (REV ? eR : eG) * A.s_inter;
        // between tiles w factors at the boundary next to the row's tile: forwards G at the end
        // of tile I - 1, backwards at the end of tile I; both exponents are <= 0 there
#pragma unroll
        for (int B = 0; B < LNT - 1; ++B) {
          const double Gb = readlane_d(G, 16 * B + 15);
          const float e = exp2_f64(REV ? G - Gb : Gb - G);
          if (REV ? l > 16 * B + 15 : l <= 16 * B + 15) GT.from[B][l] = e;
          if ((l >> 4) == (REV ? B : B + 1)) GT.to[l] = exp2_f64(REV ? Gb - G : G - Gb) * A.s_intra;
        }
      }
      decay += GC;
    };
    // products of a chunk's output rows with those of dotw: the column waves' parts in order
    auto sum_dots = [&](int j) {
      double s = 0.0;
#pragma unroll
      for (int w = 0; w < COLS; ++w) s += dot_part[w][l];
      store8(chunk_rows(A.dots, orow, j, 8), 8 * l, s);
    };
    if (n > 0) {
      store(load(0), gates[0]);
      float gl = load(1);
      lds_handover();
      for (int it = 0; it < n; ++it) {
        if constexpr (DOTS) {
          if (it > 0) sum_dots(it - 1);  // the column waves write the next ones after the coming barrier
        }
        if (it + 1 < n) {
          store(gl, gates[(it + 1) & 1]);
          gl = load(it + 2);
        }
        if (OUT) lds_handover();
        lds_handover();
      }
      if constexpr (DOTS) sum_dots(n - 1);
    }
    if (!OUT && slice == 0 && l == 0) A.slot_decay[(int64_t)seg * A.H + head] = exp2_f64(decay);
    return;
  }
  if (wave == W_ROWS) {
    // ---- rows of a, b, c straight into LDS, one chunk ahead -------------------------------
    if (n <= 0) return;
    constexpr int NB = LC * DK * 2 / 1024, NC = LC * W * 2 / 1024;  // 1 KB an instruction
    const int64_t arow = row_of(A.group_a), brow = row_of(A.group_b);
    int boff[NB], coff[NC];
#pragma unroll
    for (int i = 0; i < NB; ++i) boff[i] = LinRows<DK>::source(i, l, DK);
#pragma unroll
    for (int i = 0; i < NC; ++i) coff[i] = LinRows<W>::source(i, l, A.dc) + slice * W * 2;
    auto load = [&](int j, int s) {
      const auto rb = chunk_rows(A.b, brow, j, 2 * DK);
#pragma unroll
      for (int i = 0; i < NB; ++i) load16_lds(rb, rows_b[s].v + 512 * i, boff[i]);
      const auto rc = chunk_rows(A.c, crow, j, 2 * A.dc);
#pragma unroll
      for (int i = 0; i < NC; ++i) load16_lds(rc, rows_c[s].v + 512 * i, coff[i]);
      if constexpr (OUT) {
        const auto ra = chunk_rows(A.a, arow, j, 2 * DK);
#pragma unroll
        for (int i = 0; i < NB; ++i) load16_lds(ra, rows_a[s].v + 512 * i, boff[i]);
      }
      if constexpr (DOTS) {
        const auto rw = chunk_rows(A.dotw, crow, j, 2 * A.dc);
#pragma unroll
        for (int i = 0; i < NC; ++i) load16_lds(rw, rows_w[s].v + 512 * i, coff[i]);
      }
    };
    load(0, 0);
    wait_loads();
    lds_handover();
    for (int it = 0; it < n; ++it) {
      if (it + 1 < n) load(it + 1, (it + 1) & 1);
      if (OUT) lds_handover();
      wait_loads();
      lds_handover();
    }
    return;
  }
  if constexpr (OUT) {
    // ---- weight waves: row tiles 0 and 3, or 1 and 2 (equal numbers of products) ----------
    if (n <= 0) return;
    auto weigh = [&](auto tile0, auto tile1) {
      constexpr int TI[2] = {tile0.value, tile1.value};
      // tiles J of b that have a weight for row tile I
      constexpr auto used = [](int I, int J) { return REV ? J >= I : J <= I; };
      int row_at[NP];  // row c of a tile, 16 bytes at 32p + 8g
#pragma unroll
      for (int p = 0; p < NP; ++p) row_at[p] = LinRows<DK>::at(c, 32 * p + 8 * g);
      lds_handover();
      for (int it = 0; it < n; ++it) {
        const LinGates& GT = gates[it & 1];
        const __bf16* as = rows_a[it & 1].v;
        const __bf16* bs = rows_b[it & 1].v;
        // P_ij = w_ij (a_i . b_j): lane (g, c) holds row i = 16I + c, columns 16J + 4g + r
        f32x4 P[2][LNT];
        bf16x8 af[2][NP];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int p = 0; p < NP; ++p)
            af[i][p] = *reinterpret_cast<const bf16x8*>(as + row_at[p] + 16 * TI[i] * DK);
#pragma unroll
        for (int J = 0; J < LNT; ++J) {
          P[0][J] = P[1][J] = zero4();
          if (!used(TI[0], J) && !used(TI[1], J)) continue;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const bf16x8 bf = *reinterpret_cast<const bf16x8*>(bs + row_at[p] + 16 * J * DK);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (used(TI[i], J)) P[i][J] = mma_bf16(bf, af[i][p], P[i][J]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int I = TI[i];
          const float to = GT.to[16 * I + c];
#pragma unroll
          for (int J = 0; J < LNT; ++J) {
            if (!used(I, J)) continue;
            if (J != I) {
              const f32x4 f = *reinterpret_cast<const f32x4*>(&GT.from[REV ? I : I - 1][16 * J + 4 * g]);
              P[i][J] = P[i][J] * (f * to);
            } else {
              const float hi = GT.hi[16 * I + c], lo = GT.lo[16 * I + c];
              const f32x4 hj = *reinterpret_cast<const f32x4*>(&GT.hi[16 * J + 4 * g]);
              const f32x4 lj = *reinterpret_cast<const f32x4*>(&GT.lo[16 * J + 4 * g]);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float e = REV ? (hj[q] - hi) + (lj[q] - lo) : (hi - hj[q]) + (lo - lj[q]);
                const bool keep = REV ? 4 * g + q >= c : 4 * g + q <= c;
                P[i][J][q] = keep ? P[i][J][q] * (exp2_f32(e) * A.s_intra) : 0.f;
              }
            }
          }
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            if (REV ? 2 * p + 1 < I : 2 * p > I) continue;
            bf16x8 s[PARTS];
            split<PARTS>(P[i][2 * p], P[i][2 * p + 1], s);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) weights[k][I][p][l] = s[k];
          }
        }
        lds_handover();
        lds_handover();
      }
    };
    using std::integral_constant;
    if (wave == COLS)
      weigh(integral_constant<int, 0>{}, integral_constant<int, 3>{});
    else
      weigh(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  }
}

struct JoinArgs {
  float* slot;
  const float* decay;
  const float* init;
  int skip, back;
};
// The segments' own states joined in order, from the states given per sequence: slot[k] becomes
// the state after segment k, or before it (back).  Threads take four values of a state at a time;
// per workgroups share a state.
__global__ __launch_bounds__(256) void lin_join_kernel(JoinArgs a0, JoinArgs a1, Cut cut, int H, int size, int per) {
  const JoinArgs a = blockIdx.y ? a1 : a0;
  const int head = (int)(blockIdx.x / per) % H, seq = (int)(blockIdx.x / per) / H;
  int ns;
  const int s0 = first_segment(cut, seq, ns);
  if (s0 + ns > cut.n_seg) return;  // offsets out of order: more segments than there can be
  const int n = ns - a.skip;
  // eight segments' values asked for together: the loads do not wait for the sums
  constexpr int N = 8;
  for (int e = 4 * (int)((blockIdx.x % per) * 256 + threadIdx.x); n > 0 && e < size; e += 1024 * per) {
    f32x4 x = a.init ? *reinterpret_cast<const f32x4*>(a.init + ((int64_t)seq * H + head) * size + e) : zero4();
    for (int i0 = 0; i0 < n; i0 += N) {
      f32x4* at[N];
      f32x4 v[N];
      float d[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int i = min(i0 + k, n - 1);
        const int64_t sh = (int64_t)(a.back ? s0 + ns - 1 - i : s0 + i) * H + head;
        at[k] = reinterpret_cast<f32x4*>(a.slot + sh * size + e);
        v[k] = *at[k];
        d[k] = a.decay[sh];
      }
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (i0 + k < n) {
          x = x * d[k] + v[k];
          *at[k] = x;
        }
    }
  }
}

// dg of one (segment, head).  From the segment's end backwards dg_t = <D, S> there + sum_{s>=t}
// (q_s . dq_s - k_s . dk_s), and at the segment's first token dg is <D, S> before it.  The
// rounding errors of the sum grow like a random walk; what it misses the second product by is
// taken back in proportion to the tokens summed, which leaves a bridge between two exact ends (a
// third of the mean square error).  Bound by memory: four states a segment (B4 H16 T4096 d128: 67
// MB in 13 us).  All sums in fp64.  Per-head decays: the segment's sum.
__global__ __launch_bounds__(256) void lin_dgate_kernel(const double* dot_q, const double* dot_k, const float* slot_s,
                                                        const float* slot_d, const float* S0, const float* dS0,
                                                        const float* dS, float* dg, double* dg_seg, Cut cut, int H,
                                                        int size) {
  __shared__ double red[4][2];
  const int head = (int)blockIdx.x % H;
  const int l = lane_id(), wave = threadIdx.x / WAVE;
  Span sp;
  const int64_t seg = blockIdx.x / H;
  if (!find_segment(cut, (int)seg, sp)) return;
  auto wave_sum = [&](double x) {
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) x += __shfl_xor(x, d);
    return x;
  };
  auto block_sum = [&](double x, double y, double& sx, double& sy) {
    x = wave_sum(x);
    y = wave_sum(y);
    __syncthreads();
    if (l == 0) {
      red[wave][0] = x;
      red[wave][1] = y;
    }
    __syncthreads();
    sx = (red[0][0] + red[1][0]) + (red[2][0] + red[3][0]);
    sy = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
  };
  // thread i holds tokens t1 - 1 - i - 256 k: all are asked for before anything is summed
  constexpr int RUNS = BWD_SEG_CHUNKS * LC / 256;
  const int64_t row0 = ((cut.offsets ? 0 : (int64_t)sp.seq * H) + head) * cut.T + sp.tok0;
  const int t0 = sp.c0 * LC, t1 = min(sp.len, (sp.c0 + sp.nc) * LC);
  double rq[RUNS], rk[RUNS];
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    const int t = t1 - 1 - (int)threadIdx.x - 256 * k;
    rq[k] = t >= t0 ? dot_q[row0 + t] : 0.0;
    rk[k] = t >= t0 ? dot_k[row0 + t] : 0.0;
  }
  // the states at the segment's two ends (none given: zeros, and so is their product)
  auto of = [&](const float* p, int64_t i) { return p ? p + (i * H + head) * size : nullptr; };
  const float* De = sp.last ? of(dS, sp.seq) : of(slot_d, seg + 1);
  const float* Se = De ? of(slot_s, seg) : nullptr;
  const float* Sb = sp.first ? of(S0, sp.seq) : of(slot_s, seg - 1);
  const float* Db = sp.first ? of(dS0, sp.seq) : of(slot_d, seg);
  double end = 0.0, begin = 0.0;
#pragma unroll 2
  for (int e = 4 * (int)threadIdx.x; e < size; e += 1024) {
    f32x4 a = zero4(), b = zero4(), c = zero4(), d = zero4();
    if (De) {
      a = *reinterpret_cast<const f32x4*>(De + e);
      b = *reinterpret_cast<const f32x4*>(Se + e);
    }
    if (Sb && Db) {
      c = *reinterpret_cast<const f32x4*>(Db + e);
      d = *reinterpret_cast<const f32x4*>(Sb + e);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      end = fma((double)a[r], (double)b[r], end);
      begin = fma((double)c[r], (double)d[r], begin);
    }
  }
  block_sum(end, begin, end, begin);
  // sums from the segment's end, this thread's tokens
  double run = end, at[RUNS];
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    const double r = wave_scan_f64(rq[k] - rk[k]);
    __syncthreads();
    if (l == WAVE - 1) red[wave][0] = r;
    __syncthreads();
    at[k] = run + r;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at[k] += red[w][0];
      run += red[w][0];
    }
  }
  // a state given whose gradient is not formed: nothing to compare the sum with
  const double miss = Sb && !Db ? 0.0 : begin - run;
  const double share = t1 > t0 ? miss / (double)(t1 - t0) : 0.0;
  double sum = 0.0, unused;
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    const int t = t1 - 1 - (int)threadIdx.x - 256 * k;
    if (t >= t0) {
      const double x = at[k] + share * (double)(t1 - t);
      if (dg) dg[row0 + t] = (float)x;
      sum += x;
    }
  }
  if (dg_seg) {
    block_sum(sum, 0.0, sum, unused);
    if (threadIdx.x == 0) dg_seg[seg * H + head] = sum;
  }
}

// per-head decays: the segments' sums in order
__global__ __launch_bounds__(64) void lin_dgate_head_kernel(const double* dg_seg, float* dg, Cut cut, int H) {
  int ns = 0;
  const int n = cut.n_seq > 0 ? min(cut.n_seg, first_segment(cut, cut.n_seq - 1, ns) + ns) : 0;
  double x = 0.0;
  for (int s = lane_id(); s < n; s += WAVE) x += dg_seg[(int64_t)s * H + blockIdx.x];
#pragma unroll
  for (int d = 1; d < WAVE; d <<= 1) x += __shfl_xor(x, d);
  if (lane_id() == 0) dg[blockIdx.x] = (float)x;
}

// rows before the first and behind the last packed sequence: their gradients are zero
struct Outside {
  char* p[4];
  int heads[4];
  int row_bytes[4];  // a multiple of 4
};
__global__ __launch_bounds__(256) void lin_outside_kernel(Outside o, const int32_t* offsets, int n_seq, int64_t T) {
  int lo = (int)T, hi = (int)T, unused;
  if (n_seq > 0) {
    seq_bounds(offsets, 0, T, lo, unused);
    seq_bounds(offsets, n_seq - 1, T, unused, hi);
  }
  if (hi < lo) hi = lo;
  const int64_t rows = lo + (T - hi);
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  for (int k = 0; k < 4; ++k) {
    const int words = o.row_bytes[k] / 4;
    if (!o.p[k]) continue;
    for (int64_t i = at; i < rows * o.heads[k] * words; i += step) {
      const int64_t r = i / words % rows, head = i / words / rows;
      const int64_t row = r < lo ? r : hi + (r - lo);
      reinterpret_cast<uint32_t*>(o.p[k])[(head * T + row) * words + i % words] = 0u;
    }
  }
}

// gradients of shared heads: the group's fp32 parts summed in order and rounded once; rows
// before the first and behind the last packed sequence are left as they are
__global__ __launch_bounds__(256) void lin_group_sum_kernel(const float* part_q, const float* part_k, void* out_q,
                                                            void* out_k, int out_bf16, int64_t n, int64_t head_size,
                                                            int d, int group, const int32_t* offsets, int n_seq) {
  const float* part = blockIdx.y ? part_k : part_q;
  void* out = blockIdx.y ? out_k : out_q;
  const int64_t e = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (e >= n) return;
  const int64_t hd = e / head_size, in = e % head_size;
  if (offsets && (in < (int64_t)offsets[0] * d || in >= (int64_t)offsets[n_seq] * d)) return;
  f32x4 x = zero4();
  for (int i = 0; i < group; ++i)
    x = x + *reinterpret_cast<const f32x4*>(part + (hd * group + i) * head_size + in);
  if (out_bf16)
    *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(out) + e) = pack4(x);
  else
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + e) = x;
}

// ---- host side -----------------------------------------------------------------------

namespace {

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// how a call is cut and where its workspace holds what
struct LinPlan {
  Cut cut;
  int64_t n_seg;
  int width;   // columns of c per workgroup, of d_v
  bool ahead;  // the segments' states are formed ahead
  size_t slot_s, slot_d, decay_s, decay_d, dot_q, dot_k, dg_seg, part_q, part_k, bytes;
};

bool fits(int d, int width) { return d % width == 0; }
// of a scan for the segments' states: without outputs there is no w (a . b) to share, and more,
// smaller workgroups spread better (9 us less than at 128 columns on the prefill workload, 11 less
// on 13 packed sequences)
int state_width(int width) { return width < 64 ? width : 64; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Microseconds of one scan, after whole launches at d = 128: a workgroup of 128 / 64 / 32 columns
// takes 4.2 / 2.6 / 2.35 a chunk with outputs (one workgroup a CU) and 1.7 / 1.5 at 64 / 32
// columns without (two a CU; a third fits, but then memory sets the rate: 256, 512, 768 and 1024
// workgroups of 64 columns take 1.4, 2.2, 3.2 and 4.1 a chunk), starts and ends in 8, and memory
// gives 4.5 MB a microsecond.
// Segments of equal length run in whole rounds; packed sequences leave segments of all lengths,
// and whichever CU is free takes the next.  groups workgroups of at most len chunks, all chunks.
double scan_cost(const LinLaunch& p, int width, double groups, double len, double all, bool out, double bytes) {
  const double chunk = (out ? (width == 128 ? 4.2 : width == 64 ? 2.6 : 2.35) : width == 64 ? 1.7 : 1.5) *
                       (p.d_k == 128 ? 1.0 : 0.7);
  const double rounds = groups / (out ? 256 : 512);
  const double work = rounds <= 1.0 || !p.offsets
                          ? ceil(rounds) * (len * chunk + 8.0)
                          : (all / groups * rounds + 0.5 * len) * chunk + 8.0 * rounds;
  const double memory = bytes / 4.5e6 + 6.0;
  return work > memory ? work : memory;
}

// Microseconds of a whole pass over segments of len chunks by workgroups of width columns
double plan_cost(const LinLaunch& p, bool bwd, int width, int64_t len) {
  const int64_t longest = ceil_div(p.T, LC), per = ceil_div(longest, len);
  // packed: sequences end half a chunk and half a segment before the next on average; one of
  // them may hold nearly all tokens
  const double seqs = p.offsets ? 1.0 : p.n_seq, ends = p.offsets ? 0.5 * p.n_seq : 0.0;
  const double all = (double)longest * seqs + ends;
  double n = p.offsets ? all / (double)len + ends : (double)(per * p.n_seq);
  if (n < p.n_seq) n = p.n_seq;
  const double slices = p.d_v / width, H = p.H;
  const double bytes = seqs * (double)p.T * 2.0 * ((double)p.H_qk * p.d_k + H * p.d_v);  // K and V
  // dQ and dK, with their products for dg, take 5.2 a chunk, dV 4.2: 1.15 on average
  double cost = bwd ? 3.0 * scan_cost(p, width, n * H, 1.15 * (double)len, 1.15 * all * H, true, 3.0 * bytes)
                    : scan_cost(p, width, n * H * slices, (double)len, all * H * slices, true, 2.0 * bytes);
  if (per > 1) {
    const int w = state_width(width);
    const double inner = (n - seqs) * H * (p.d_v / w), most = all * H * (p.d_v / w);
    const double state = 4.0 * p.H * p.d_k * p.d_v, share = (double)(per - 1) / (double)per;
    // the segments' states, and joining them: read and written (backwards both kinds, and read
    // once more for dg)
    cost += (bwd ? 2.0 : 1.0) * scan_cost(p, w, inner, (double)len, most * share, false, bytes * share) + 8.0 +
            (bwd ? 8.0 : 2.0) * n * state / 6e6;
  }
  return cost;
}

LinPlan make_plan(const LinLaunch& p, bool bwd) {
  LinPlan q{};
  const int64_t nch = ceil_div(p.T, LC), longest = nch > 0 ? nch : 1;
  const int64_t all = p.offsets ? nch + p.n_seq : longest * p.n_seq;  // chunks, at most
  q.width = bwd ? p.d_v : fits(p.d_v, 128) ? 128 : fits(p.d_v, 64) ? 64 : 32;
  // Whole sequences, or segments for more workgroups: their own states cost another reading of K
  // and V, and the launches and the joining some more.  B4 H16 T8192 d128: four segments a
  // sequence 217 us, eight 238, whole sequences in two slices of 64 columns 314, in four of 32 305;
  // 128 heads of 4096: two slices 184, two segments 210.  Backwards (12 heads, 7 packed sequences,
  // 5003 tokens) segments of 4 chunks 130 us, 5 113, 6 120, 8 136.  There a segment also bounds
  // the sums of dg.
  int64_t chunks = longest;
  double best = 1e300;
  const int widest = q.width;
  auto consider = [&](int width, int64_t len) {
    const double cost = plan_cost(p, bwd, width, len);
    if (cost < best) {
      best = cost;
      q.width = width;
      chunks = len;
    }
  };
  if (bwd) {
    for (int64_t len = BWD_SEG_CHUNKS < longest ? BWD_SEG_CHUNKS : longest; len >= (longest < 2 ? 1 : 2); --len)
      consider(widest, len);
  } else if (longest > 4) {
    for (int w = widest; w >= 32; w /= 2) {
      consider(w, longest);
      if (p.offsets) {
        for (int64_t len = 4; len < longest; len += 1 + len / 4) consider(w, len);
      } else {
        for (int rounds = 1; rounds <= 4; ++rounds) {
          const int64_t len = ceil_div(all * p.H * (p.d_v / w), 256 * rounds);
          if (len < longest) consider(w, len < 2 ? 2 : len);
        }
      }
    }
  }
  q.cut.offsets = p.offsets;
  q.cut.T = p.T;
  q.cut.n_seq = p.n_seq;
  q.cut.chunks = (int)chunks;
  q.cut.segments = (int)ceil_div(longest, chunks);
  // packed: sum over sequences of max(1, ceil(len / (64 chunks))) <= T / (64 chunks) + sequences
  q.n_seg = p.offsets ? nch / chunks + p.n_seq : (int64_t)q.cut.segments * p.n_seq;
  q.cut.n_seg = (int)q.n_seg;  // lin_grid_ok: it is one
  q.ahead = q.cut.segments > 1;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t x = at;
    at += up256(n);
    return x;
  };
  const size_t one = (size_t)p.d_k * p.d_v * 4, sh = (size_t)q.n_seg * p.H;
  const size_t tokens = (size_t)(p.offsets ? 1 : p.n_seq) * p.H * p.T;
  if (q.ahead || bwd) {
    q.slot_s = take(sh * one);
    q.decay_s = take(sh * 4);
  }
  if (bwd) {
    q.slot_d = take(sh * one);
    q.decay_d = take(sh * 4);
    q.dot_q = take(tokens * 8);
    q.dot_k = take(tokens * 8);
    if (p.g_per_head) q.dg_seg = take(sh * 8);
    if (p.H != p.H_qk) {
      q.part_q = take(tokens * p.d_k * 4);
      q.part_k = take(tokens * p.d_k * 4);
    }
  }
  q.bytes = at;
  return q;
}

template <bool REV, bool OUT, bool DOTS, class TO>
int scan(int dk, int width, const ScanArgs& a, hipStream_t s) {
  const int64_t family = (int64_t)(a.dc / width) * (a.group_a > a.group_c ? a.group_a : a.group_c);
  const int64_t total = (int64_t)a.cut.n_seg * a.H * (a.dc / width);
  const dim3 grid((unsigned)(8 * family * ceil_div(total, 8 * family)));
  auto go = [&](auto d, auto w) {
    hipLaunchKernelGGL((lin_scan_kernel<d.value, w.value, REV, OUT, DOTS, TO>), grid,
                       dim3(scan_waves(w.value, OUT) * WAVE), 0, s, a);
    return 0;
  };
  using std::integral_constant;
  auto by_width = [&](auto d) {
    if constexpr (OUT)
      if (width == 128) return go(d, integral_constant<int, 128>{});
    if (width == 64) return go(d, integral_constant<int, 64>{});
    // the backward pass has d_k and d_v of 64 and 128 only
    if constexpr (!REV && !DOTS) return go(d, integral_constant<int, 32>{});
    return -1;
  };
  if (dk == 64) return by_width(integral_constant<int, 64>{});
  if (dk == 128) return by_width(integral_constant<int, 128>{});
  return -1;
}

ScanArgs base_args(const LinLaunch& p, const LinPlan& q) {
  ScanArgs a{};
  a.g = p.g;
  a.cut = q.cut;
  a.H = p.H;
  a.group_a = a.group_b = a.group_c = 1;
  a.g_per_head = p.g_per_head;
  return a;
}

// joins n (1 or 2) sets of segment states
void join(const JoinArgs* a, int n, const LinLaunch& p, const LinPlan& q, hipStream_t s) {
  const int size = p.d_k * p.d_v, heads = p.H * p.n_seq;
  // a state's values over as many workgroups as keep the GPU in one round of them: each has to
  // find its segments first (13 packed sequences, 16 heads, 128 x 256: the call takes 145.3 us,
  // 146.6 with 32 workgroups each, 149.4 with half as many as here)
  int per = JOIN_GROUPS / heads;
  per = per < 1 ? 1 : per > (size + 1023) / 1024 ? (size + 1023) / 1024 : per;
  const dim3 grid((unsigned)(per * heads), (unsigned)n), block(256);
  hipLaunchKernelGGL(lin_join_kernel, grid, block, 0, s, a[0], a[n - 1], q.cut, p.H, size, per);
}

const __bf16* bf(const void* p) { return reinterpret_cast<const __bf16*>(p); }

}  // namespace

size_t lin_workspace(const LinLaunch& p, bool bwd) { return make_plan(p, bwd).bytes; }

bool lin_grid_ok(const LinLaunch& p, bool bwd) {
  const LinPlan q = make_plan(p, bwd);
  // threads of a launch are below 2^32; all factors are, and the doubles round by far less than
  // their products are away from overflow
  const double most = 4294967295.0, cols = p.d_k > p.d_v ? p.d_k : p.d_v, H = p.H, n_seq = p.n_seq;
  const double scan = ((double)q.n_seg + 8.0) * H * cols * 12.0;  // 6 waves for 32 columns, the last round of families full
  const double sum = (p.offsets ? 1.0 : n_seq) * H * (double)p.T * p.d_k / 4.0;
  return scan < most && (!bwd || p.H == p.H_qk || sum < most);
}

int launch_lin_fwd(const LinLaunch& p, void* workspace, hipStream_t s) {
  const LinPlan q = make_plan(p, false);
  char* ws = reinterpret_cast<char*>(workspace);
  ScanArgs a = base_args(p, q);
  a.a = bf(p.Q);
  a.b = bf(p.K);
  a.c = bf(p.V);
  a.group_a = a.group_b = p.H / p.H_qk;
  a.dc = p.d_v;
  a.init = p.S0;
  a.fin = p.S_out;
  a.out = p.O;
  a.s_intra = a.s_inter = p.scale;
  a.s_state = 1.f;
  if (q.ahead) {
    a.slot = reinterpret_cast<float*>(ws + q.slot_s);
    a.slot_decay = reinterpret_cast<float*>(ws + q.decay_s);
    a.skip = 1;
    const int rc = scan<false, false, false, float>(p.d_k, state_width(q.width), a, s);
    if (rc) return rc;
    const JoinArgs j{a.slot, a.slot_decay, p.S0, 1, 0};
    join(&j, 1, p, q, s);
  }
  return p.o_bf16 ? scan<false, true, false, __bf16>(p.d_k, q.width, a, s)
                  : scan<false, true, false, float>(p.d_k, q.width, a, s);
}

int launch_lin_bwd(const LinLaunch& p, void* workspace, hipStream_t s) {
  const LinPlan q = make_plan(p, true);
  char* ws = reinterpret_cast<char*>(workspace);
  const int group = p.H / p.H_qk;
  const bool end = p.dS != nullptr && p.dg != nullptr;  // <dS, S> at the sequences' ends is wanted
  float* slot_s = reinterpret_cast<float*>(ws + q.slot_s);
  float* slot_d = reinterpret_cast<float*>(ws + q.slot_d);
  if (p.offsets && p.T > 0) {
    const int size = p.grad_bf16 ? 2 : 4;
    const Outside o{{(char*)p.dQ, (char*)p.dK, (char*)p.dV, p.g_per_head ? nullptr : (char*)p.dg},
                    {p.H_qk, p.H_qk, p.H, p.H},
                    {p.d_k * size, p.d_k * size, p.d_v * size, 4}};
    hipLaunchKernelGGL(lin_outside_kernel, dim3(128), dim3(256), 0, s, o, p.offsets, p.n_seq, p.T);
  }
  if (p.n_seq == 0) {  // no sequence: nothing but zeros
    if (p.dg && p.g_per_head)
      hipLaunchKernelGGL(lin_dgate_head_kernel, dim3((unsigned)p.H), dim3(64), 0, s, nullptr, p.dg, q.cut, p.H);
    return 0;
  }
  int rc = 0, n_joins = 0;
  JoinArgs joins[2];
  // states after the segments
  if (q.ahead || end) {
    ScanArgs f = base_args(p, q);
    f.b = bf(p.K);
    f.c = bf(p.V);
    f.group_a = f.group_b = group;
    f.dc = p.d_v;
    f.s_state = 1.f;
    f.slot = slot_s;
    f.slot_decay = reinterpret_cast<float*>(ws + q.decay_s);
    f.skip = end ? 0 : 1;
    rc = scan<false, false, false, float>(p.d_k, state_width(q.width), f, s);
    if (rc) return rc;
    joins[n_joins++] = {f.slot, f.slot_decay, p.S0, f.skip, 0};
  }
  // gradients of the states before the segments; dV, and the gradient of the states given
  ScanArgs r = base_args(p, q);
  r.a = bf(p.K);
  r.b = bf(p.Q);
  r.c = bf(p.dO);
  r.group_a = r.group_b = group;
  r.dc = p.d_v;
  r.s_state = p.scale;
  r.slot = slot_d;
  r.slot_decay = reinterpret_cast<float*>(ws + q.decay_d);
  r.skip = 1;
  if (q.ahead) {
    rc = scan<true, false, false, float>(p.d_k, state_width(q.width), r, s);
    if (rc) return rc;
    joins[n_joins++] = {r.slot, r.slot_decay, p.dS, 1, 1};
  }
  if (n_joins) join(joins, n_joins, p, q, s);
  r.init = p.dS;
  r.fin = p.dS0;
  r.out = p.dV;
  r.s_intra = p.scale;
  r.s_inter = 1.f;
  rc = p.grad_bf16 ? scan<true, true, false, __bf16>(p.d_k, q.width, r, s)
                   : scan<true, true, false, float>(p.d_k, q.width, r, s);
  if (rc) return rc;
  // dK and dQ: the transposed states, contraction over d_v
  ScanArgs k = base_args(p, q);
  k.dc = p.d_k;
  k.a = bf(p.V);
  k.b = bf(p.dO);
  k.c = bf(p.Q);
  k.group_c = group;
  k.init = p.dS;
  k.slot = slot_d;
  k.dotw = bf(p.K);
  k.dots = reinterpret_cast<double*>(ws + q.dot_k);
  k.out = group > 1 ? (void*)(ws + q.part_k) : p.dK;
  const bool part_bf16 = group == 1 && p.grad_bf16;
  k.s_intra = k.s_state = p.scale;
  k.s_inter = 1.f;
  rc = part_bf16 ? scan<true, true, true, __bf16>(p.d_v, p.d_k, k, s) : scan<true, true, true, float>(p.d_v, p.d_k, k, s);
  if (rc) return rc;
  k.a = bf(p.dO);
  k.b = bf(p.V);
  k.c = bf(p.K);
  k.init = p.S0;
  k.slot = slot_s;
  k.dotw = bf(p.Q);
  k.dots = reinterpret_cast<double*>(ws + q.dot_q);
  k.out = group > 1 ? (void*)(ws + q.part_q) : p.dQ;
  k.s_intra = k.s_inter = p.scale;
  k.s_state = 1.f;
  rc = part_bf16 ? scan<false, true, true, __bf16>(p.d_v, p.d_k, k, s)
                 : scan<false, true, true, float>(p.d_v, p.d_k, k, s);
  if (rc) return rc;
  if (group > 1 && p.T > 0) {
    const int64_t n = (int64_t)(p.offsets ? 1 : p.n_seq) * p.H_qk * p.T * p.d_k;
    const dim3 grid((unsigned)ceil_div(n / 4, 256), 2), block(256);
    hipLaunchKernelGGL(lin_group_sum_kernel, grid, block, 0, s, reinterpret_cast<const float*>(ws + q.part_q),
                       reinterpret_cast<const float*>(ws + q.part_k), p.dQ, p.dK, p.grad_bf16, n, p.T * p.d_k, p.d_k,
                       group, p.offsets, p.n_seq);
  }
  if (!p.dg) return 0;
  double* dg_seg = p.g_per_head ? reinterpret_cast<double*>(ws + q.dg_seg) : nullptr;
  hipLaunchKernelGGL(lin_dgate_kernel, dim3((unsigned)(p.H * q.cut.n_seg)), dim3(256), 0, s,
                     reinterpret_cast<const double*>(ws + q.dot_q), reinterpret_cast<const double*>(ws + q.dot_k), slot_s,
                     slot_d, p.S0, p.dS0, p.dS, p.g_per_head ? nullptr : p.dg, dg_seg, q.cut, p.H, p.d_k * p.d_v);
  if (p.g_per_head)
    hipLaunchKernelGGL(lin_dgate_head_kernel, dim3((unsigned)p.H), dim3(64), 0, s, dg_seg, p.dg, q.cut, p.H);
  return 0;
}

}  // namespace gdn
