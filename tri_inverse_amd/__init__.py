"""tri_inverse_amd -- Python binding of libgdn (include/gdn.h) for MI355X (gfx950).

Thin ctypes layer: every function here has the name of the C entry point it calls,
checks the tensors' device, dtype, shape and contiguity, and passes data pointers and
the current HIP stream.  Every step of the computation runs in libgdn's HIP kernels;
there is no CPU or PyTorch fallback.  If libgdn.so has not been built, importing this
package raises ImportError (build it with ``python tri_inverse_amd/build.py``).

PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libgdn.so is not built (run `python tri_inverse_amd/build.py`); "
                      "tri_inverse_amd has no fallback path")

_lib = ctypes.CDLL(LIB_PATH)

# dtype and mode codes (gdn.h)
GDN_F32, GDN_BF16, GDN_FP8_E4M3, GDN_INT8, GDN_INT16 = 0, 1, 2, 3, 4
GDN_INV_NEUMANN, GDN_INV_EXACT, GDN_INV_NEUMANN_PRODUCTS = 0, 1, 2
GDN_GATE_SILU, GDN_GATE_SIGMOID = 0, 1
GDN_OK = 0
GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_HIP = 5, 6, 7
FP8_STATS_FIELDS = ("nonfinite", "sat_dynamic", "sat_static", "underflow")

_COMPUTE = {"f32": GDN_F32, "fp32": GDN_F32, "bf16": GDN_BF16, "fp8": GDN_FP8_E4M3,
            "e4m3": GDN_FP8_E4M3, "int8": GDN_INT8, "int16": GDN_INT16}
_TORCH_DTYPE = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


class gdn_blocks(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("K", ctypes.c_void_p), ("k_dtype", ctypes.c_int32),
                ("g_cumulative", ctypes.c_int32), ("beta", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("n_blocks", ctypes.c_int64), ("C", ctypes.c_int32),
                ("d_k", ctypes.c_int32)]


class gdn_inverse_cfg(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("N", ctypes.c_int32), ("mask", ctypes.c_int32),
                ("compute", ctypes.c_int32)]


class gdn_lin_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("B", ctypes.c_int32),
                ("H", ctypes.c_int32), ("H_qk", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("g_per_head", ctypes.c_int32), ("scale", ctypes.c_float)]


_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_P = ctypes.POINTER
_lib.gdn_abi_version.restype = ctypes.c_int
_lib.gdn_status_string.restype = ctypes.c_char_p
_lib.gdn_status_string.argtypes = [_i32]
_lib.gdn_build_A.restype = _i32
_lib.gdn_build_A.argtypes = [_P(gdn_blocks), _vp, _vp]
_lib.gdn_tri_inverse_neumann.restype = _i32
_lib.gdn_tri_inverse_neumann.argtypes = [_P(gdn_blocks), _i32, _i32, _i32, _vp, _i32, _vp, _vp]
_lib.gdn_tri_inverse_exact.restype = _i32
_lib.gdn_tri_inverse_exact.argtypes = [_P(gdn_blocks), _i32, _vp, _i32, _vp]
_lib.gdn_tri_inverse_residual.restype = _i32
_lib.gdn_tri_inverse_residual.argtypes = [_P(gdn_blocks), _i32, _i32, _i32, _i32, _vp, _i32, _vp]
_lib.gdn_tri_inverse_fs.restype = _i32
_lib.gdn_tri_inverse_fs.argtypes = [_P(gdn_blocks), _vp, _i32, _vp]
_lib.gdn_wy.restype = _i32
_lib.gdn_wy.argtypes = [_P(gdn_blocks), _vp, _i32, _P(gdn_inverse_cfg), _vp, _i32, _i32, _vp, _vp,
                        _i32, _vp]
_lib.gdn_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
_lib.gdn_chunk_fwd_workspace_bytes.argtypes = [_i32, _i32, _i64, _i32, _i32, _i32, _P(gdn_inverse_cfg)]
_lib.gdn_chunk_fwd.restype = _i32
_lib.gdn_chunk_fwd.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                               _i64, _i32, _i32, _i32, _f32, _P(gdn_inverse_cfg), _vp, ctypes.c_size_t,
                               _vp, _vp]
_lib.gdn_chunk_fwd_noalloc.restype = _i32
_lib.gdn_chunk_fwd_noalloc.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                       _i64, _i32, _i32, _i32, _f32, _P(gdn_inverse_cfg), _vp, _vp]
_lib.gdn_decode.restype = _i32
_lib.gdn_decode.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                            _i32, _i32, _f32, _vp]
_sz = ctypes.c_size_t
_lib.gdn_lin_chunk_fwd_workspace_bytes.restype = _sz
_lib.gdn_lin_chunk_fwd_workspace_bytes.argtypes = [_P(gdn_lin_shape)]
_lib.gdn_lin_chunk_bwd_workspace_bytes.restype = _sz
_lib.gdn_lin_chunk_bwd_workspace_bytes.argtypes = [_P(gdn_lin_shape)]
_lib.gdn_lin_chunk_fwd.restype = _i32
_lib.gdn_lin_chunk_fwd.argtypes = [_P(gdn_lin_shape), _vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _sz, _vp]
_lib.gdn_lin_chunk_bwd.restype = _i32
_lib.gdn_lin_chunk_bwd.argtypes = [_P(gdn_lin_shape), _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                   _vp, _vp, _vp, _sz, _vp]
_lib.gdn_lin_decode.restype = _i32
_lib.gdn_lin_decode.argtypes = [_P(gdn_lin_shape), _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp]
_lib.gdn_gate_norm_fwd.restype = _i32
_lib.gdn_gate_norm_fwd.argtypes = [_vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i64, _i32, _i32, _f32, _vp]
_lib.gdn_gate_norm_bwd_workspace_bytes.restype = _sz
_lib.gdn_gate_norm_bwd_workspace_bytes.argtypes = [_i32, _i32, _i64, _i32]
_lib.gdn_gate_norm_bwd.restype = _i32
_lib.gdn_gate_norm_bwd.argtypes = [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i64, _i32, _i32, _f32,
                                   _vp, _sz, _vp]
_lib.gdn_residual_norm_fwd.restype = _i32
_lib.gdn_residual_norm_fwd.argtypes = [_vp, _i32, _vp, _i32, _vp, _vp, _f32, _vp, _vp, _vp, _i64, _i32, _f32, _vp]
_lib.gdn_residual_norm_bwd_workspace_bytes.restype = _sz
_lib.gdn_residual_norm_bwd_workspace_bytes.argtypes = [_i64, _i32]
_lib.gdn_residual_norm_bwd.restype = _i32
_lib.gdn_residual_norm_bwd.argtypes = [_vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _i64, _i32, _f32, _vp, _sz, _vp]

EXPORTED = ("gdn_abi_version", "gdn_status_string", "gdn_build_A", "gdn_tri_inverse_neumann",
            "gdn_tri_inverse_exact", "gdn_tri_inverse_residual", "gdn_tri_inverse_fs", "gdn_wy",
            "gdn_chunk_fwd_workspace_bytes", "gdn_chunk_fwd", "gdn_chunk_fwd_noalloc", "gdn_decode",
            "gdn_lin_chunk_fwd_workspace_bytes", "gdn_lin_chunk_bwd_workspace_bytes", "gdn_lin_chunk_fwd",
            "gdn_lin_chunk_bwd", "gdn_lin_decode", "gdn_gate_norm_fwd", "gdn_gate_norm_bwd_workspace_bytes",
            "gdn_gate_norm_bwd", "gdn_residual_norm_fwd", "gdn_residual_norm_bwd_workspace_bytes",
            "gdn_residual_norm_bwd")
GDN_NOALLOC_SCRATCH_BYTES = 64 << 20


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s" % (where, gdn_status_string(status)))


def gdn_abi_version() -> int:
    return int(_lib.gdn_abi_version())


def gdn_status_string(status: int) -> str:
    return _lib.gdn_status_string(int(status)).decode()


def _check(st: int, where: str) -> None:
    if st != GDN_OK:
        raise GdnError(st, where)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, name, dtypes=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    return t


def _compute_code(compute) -> int:
    if isinstance(compute, int):
        return compute
    return _COMPUTE[str(compute)]


def _blocks(A=None, K=None, beta=None, g=None, C=64, g_cumulative=False):
    """Build the gdn_blocks descriptor; returns (desc, n_blocks, d_k)."""
    d = gdn_blocks()
    if A is not None:
        _dev(A, "A", (torch.float32,))
        if A.dim() < 2 or A.shape[-1] != C or A.shape[-2] != C:
            raise ValueError("A must end in [C, C]")
        nb = A.numel() // (C * C)
        d.A, d.n_blocks, d.C, d.d_k = A.data_ptr(), nb, C, 0
        return d, nb, 0
    _dev(K, "K", (torch.bfloat16, torch.float32))
    _dev(beta, "beta", (torch.float32,))
    _dev(g, "g", (torch.float32,))
    dk = K.shape[-1]
    rows = K.numel() // dk
    if rows % C != 0:
        raise ValueError("K has %d rows, not a multiple of C=%d" % (rows, C))
    nb = rows // C
    if beta.numel() != rows or g.numel() != rows:
        raise ValueError("beta and g need one value per K row")
    d.A = None
    d.K = K.data_ptr()
    d.k_dtype = _TORCH_DTYPE[K.dtype]
    d.g_cumulative = int(bool(g_cumulative))
    d.beta, d.g = beta.data_ptr(), g.data_ptr()
    d.n_blocks, d.C, d.d_k = nb, C, dk
    return d, nb, dk


def gdn_build_A(K, beta, g, C: int = 64, g_cumulative: bool = False, out=None, stream=None):
    """A = -tril(diag(beta)(K K^T .* exp(G_i - G_j)), -1) per C-row block -> [n_blocks, C, C] fp32."""
    d, nb, _ = _blocks(K=K, beta=beta, g=g, C=C, g_cumulative=g_cumulative)
    if out is None:
        out = torch.empty((nb, C, C), device=K.device, dtype=torch.float32)
    _dev(out, "out", (torch.float32,))
    _check(_lib.gdn_build_A(ctypes.byref(d), _ptr(out), _stream(stream)), "gdn_build_A")
    return out


def gdn_tri_inverse_neumann(A=None, K=None, beta=None, g=None, C: int = 64, N: int = 3,
                            mask: bool = True, compute="bf16", t_dtype=torch.float32,
                            g_cumulative: bool = False, stats=None, out=None, stream=None):
    """Truncated (optionally band-masked) Neumann inverse per block -> T [n_blocks, C, C].

    Give either A ([.., C, C] fp32) or K/beta/g.  stats: optional CUDA int64 tensor of 4
    (fp8 diagnostics; zeroed then accumulated on the stream)."""
    d, nb, _ = _blocks(A, K, beta, g, C, g_cumulative)
    dev = (A if A is not None else K).device
    if out is None:
        out = torch.empty((nb, C, C), device=dev, dtype=t_dtype)
    _dev(out, "out", (torch.float32, torch.bfloat16))
    if stats is not None:
        _dev(stats, "stats", (torch.int64,))
        if stats.numel() < 4:
            raise ValueError("stats needs 4 elements")
    st = _lib.gdn_tri_inverse_neumann(ctypes.byref(d), int(N), int(bool(mask)),
                                      _compute_code(compute), _ptr(out), _TORCH_DTYPE[out.dtype],
                                      _ptr(stats), _stream(stream))
    _check(st, "gdn_tri_inverse_neumann")
    return out


def gdn_tri_inverse_exact(A=None, K=None, beta=None, g=None, C: int = 64, compute="bf16",
                          t_dtype=torch.float32, g_cumulative: bool = False, out=None, stream=None):
    """Exact doubling-product inverse per block -> T [n_blocks, C, C]."""
    d, nb, _ = _blocks(A, K, beta, g, C, g_cumulative)
    dev = (A if A is not None else K).device
    if out is None:
        out = torch.empty((nb, C, C), device=dev, dtype=t_dtype)
    _dev(out, "out", (torch.float32, torch.bfloat16))
    st = _lib.gdn_tri_inverse_exact(ctypes.byref(d), _compute_code(compute), _ptr(out),
                                    _TORCH_DTYPE[out.dtype], _stream(stream))
    _check(st, "gdn_tri_inverse_exact")
    return out


def gdn_tri_inverse_residual(A=None, K=None, beta=None, g=None, C: int = 64, N: int = 3,
                             mask: bool = True, S: int = 8, compute="f32", t_dtype=torch.float32,
                             g_cumulative: bool = False, out=None, stream=None):
    """Truncated (optionally band-masked) Neumann sum refined by the parallel residual
    correction T = T0 sum_{s<=S} E^s, E = I - (I - A) T0 -> T [n_blocks, C, C]."""
    d, nb, _ = _blocks(A, K, beta, g, C, g_cumulative)
    dev = (A if A is not None else K).device
    if out is None:
        out = torch.empty((nb, C, C), device=dev, dtype=t_dtype)
    _dev(out, "out", (torch.float32, torch.bfloat16))
    st = _lib.gdn_tri_inverse_residual(ctypes.byref(d), int(N), int(bool(mask)), int(S),
                                       _compute_code(compute), _ptr(out), _TORCH_DTYPE[out.dtype],
                                       _stream(stream))
    _check(st, "gdn_tri_inverse_residual")
    return out


def gdn_tri_inverse_fs(A=None, K=None, beta=None, g=None, C: int = 64, t_dtype=torch.float32,
                       g_cumulative: bool = False, out=None, stream=None):
    """Forward substitution (fp32), the sequential baseline -> T [n_blocks, C, C]."""
    d, nb, _ = _blocks(A, K, beta, g, C, g_cumulative)
    dev = (A if A is not None else K).device
    if out is None:
        out = torch.empty((nb, C, C), device=dev, dtype=t_dtype)
    _dev(out, "out", (torch.float32, torch.bfloat16))
    st = _lib.gdn_tri_inverse_fs(ctypes.byref(d), _ptr(out), _TORCH_DTYPE[out.dtype], _stream(stream))
    _check(st, "gdn_tri_inverse_fs")
    return out


def _inv_cfg(mode, N, mask, compute):
    c = gdn_inverse_cfg()
    if mode in ("exact", GDN_INV_EXACT):
        c.mode = GDN_INV_EXACT
    elif mode in ("neumann_products", GDN_INV_NEUMANN_PRODUCTS):
        c.mode = GDN_INV_NEUMANN_PRODUCTS
    else:
        c.mode = GDN_INV_NEUMANN
    c.N, c.mask, c.compute = int(N), int(bool(mask)), _compute_code(compute)
    return c


def gdn_wy(K, beta, g, V, C: int = 64, T=None, mode="neumann", N: int = 3, mask: bool = True,
           compute="bf16", gate_k: bool = False, out_dtype=torch.bfloat16,
           g_cumulative: bool = False, W_out=None, U_out=None, stream=None):
    """WY products per block: W = T diag(s) K, U = T diag(beta) V (s = beta, or beta*e^G
    with gate_k).  T given ([n_blocks, C, C] fp32/bf16) or formed on the fly."""
    d, nb, dk = _blocks(None, K, beta, g, C, g_cumulative)
    _dev(V, "V", (torch.bfloat16,))
    dv = V.shape[-1]
    if V.numel() != nb * C * dv:
        raise ValueError("V must hold n_blocks * C rows")
    if T is not None:
        _dev(T, "T", (torch.float32, torch.bfloat16))
        if T.numel() != nb * C * C:
            raise ValueError("T must be [n_blocks, C, C]")
    if W_out is None:
        W_out = torch.empty((nb, C, dk), device=K.device, dtype=out_dtype)
    if U_out is None:
        U_out = torch.empty((nb, C, dv), device=K.device, dtype=out_dtype)
    _dev(W_out, "W_out", (torch.float32, torch.bfloat16))
    _dev(U_out, "U_out", (W_out.dtype,))
    cfg = _inv_cfg(mode, N, mask, compute)
    st = _lib.gdn_wy(ctypes.byref(d), _ptr(T), _TORCH_DTYPE[T.dtype] if T is not None else 0,
                     ctypes.byref(cfg), _ptr(V), int(dv), int(bool(gate_k)), _ptr(W_out),
                     _ptr(U_out), _TORCH_DTYPE[W_out.dtype], _stream(stream))
    _check(st, "gdn_wy")
    return W_out, U_out


def gdn_chunk_fwd_workspace_bytes(B: int, H: int, T: int, d_k: int, d_v: int, C: int = 64,
                                  mode="neumann", N: int = 3, mask: bool = True, compute="bf16") -> int:
    """Device workspace (bytes) gdn_chunk_fwd needs for these arguments (0: none)."""
    cfg = _inv_cfg(mode, N, mask, compute)
    return int(_lib.gdn_chunk_fwd_workspace_bytes(int(B), int(H), int(T), int(d_k), int(d_v), int(C),
                                                  ctypes.byref(cfg)))


def gdn_chunk_fwd(Q, K, V, beta, g, C: int = 64, scale: float | None = None, S0=None,
                  mode="neumann", N: int = 3, mask: bool = True, compute="bf16",
                  o_dtype=torch.bfloat16, stats=None, O=None, S_out=None, workspace=None, stream=None):
    """Chunk-wise gated delta rule forward.  Q, K [B,H,T,d_k], V [B,H,T,d_v] bf16;
    beta, g [B,H,T] fp32 -> (O [B,H,T,d_v], S_out [B,H,d_k,d_v] fp32).

    workspace: a CUDA uint8 tensor of at least gdn_chunk_fwd_workspace_bytes(...) bytes,
    or None to have one allocated here (through torch) when the variant needs it."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _dev(t, n, (torch.bfloat16,))
    _dev(beta, "beta", (torch.float32,))
    _dev(g, "g", (torch.float32,))
    if K.dim() != 4 or Q.shape != K.shape:
        raise ValueError("Q and K must both be [B, H, T, d_k]")
    B, H, T, dk = K.shape
    dv = V.shape[-1]
    if V.shape[:3] != (B, H, T) or beta.shape != (B, H, T) or g.shape != (B, H, T):
        raise ValueError("V, beta, g must match Q/K in [B, H, T]")
    if S0 is not None:
        _dev(S0, "S0", (torch.float32,))
        if S0.shape != (B, H, dk, dv):
            raise ValueError("S0 must be [B, H, d_k, d_v]")
    if O is None:
        O = torch.empty((B, H, T, dv), device=K.device, dtype=o_dtype)
    if S_out is None:
        S_out = torch.empty((B, H, dk, dv), device=K.device, dtype=torch.float32)
    _dev(O, "O", (torch.float32, torch.bfloat16))
    _dev(S_out, "S_out", (torch.float32,))
    if stats is not None:
        _dev(stats, "stats", (torch.int64,))
        if stats.numel() < 4:
            raise ValueError("stats needs 4 elements")
    if scale is None:
        scale = dk ** -0.5
    cfg = _inv_cfg(mode, N, mask, compute)
    need = int(_lib.gdn_chunk_fwd_workspace_bytes(B, H, T, dk, dv, C, ctypes.byref(cfg)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=K.device, dtype=torch.uint8)
    if workspace is not None:
        _dev(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.gdn_chunk_fwd(_ptr(Q), _ptr(K), _ptr(V), GDN_BF16, _ptr(beta), _ptr(g), _ptr(S0),
                            _ptr(O), _TORCH_DTYPE[O.dtype], _ptr(S_out), B, H, T, dk, dv, C,
                            float(scale), ctypes.byref(cfg), _ptr(workspace), ws_bytes, _ptr(stats),
                            _stream(stream))
    _check(st, "gdn_chunk_fwd")
    return O, S_out


def gdn_chunk_fwd_noalloc(Q, K, V, beta, g, C: int = 64, scale: float | None = None, S0=None,
                          mode="neumann", N: int = 3, mask: bool = True, compute="bf16",
                          o_dtype=torch.bfloat16, stats=None, O=None, S_out=None, stream=None):
    """gdn_chunk_fwd with the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate).  Arguments and results as gdn_chunk_fwd; O and
    S_out are still the caller's (pass them to allocate nothing here either)."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _dev(t, n, (torch.bfloat16,))
    _dev(beta, "beta", (torch.float32,))
    _dev(g, "g", (torch.float32,))
    if K.dim() != 4 or Q.shape != K.shape:
        raise ValueError("Q and K must both be [B, H, T, d_k]")
    B, H, T, dk = K.shape
    dv = V.shape[-1]
    if V.shape[:3] != (B, H, T) or beta.shape != (B, H, T) or g.shape != (B, H, T):
        raise ValueError("V, beta, g must match Q/K in [B, H, T]")
    if S0 is not None:
        _dev(S0, "S0", (torch.float32,))
    if O is None:
        O = torch.empty((B, H, T, dv), device=K.device, dtype=o_dtype)
    if S_out is None:
        S_out = torch.empty((B, H, dk, dv), device=K.device, dtype=torch.float32)
    _dev(O, "O", (torch.float32, torch.bfloat16))
    _dev(S_out, "S_out", (torch.float32,))
    if stats is not None:
        _dev(stats, "stats", (torch.int64,))
    if scale is None:
        scale = dk ** -0.5
    cfg = _inv_cfg(mode, N, mask, compute)
    st = _lib.gdn_chunk_fwd_noalloc(_ptr(Q), _ptr(K), _ptr(V), GDN_BF16, _ptr(beta), _ptr(g), _ptr(S0),
                                    _ptr(O), _TORCH_DTYPE[O.dtype], _ptr(S_out), B, H, T, dk, dv, C,
                                    float(scale), ctypes.byref(cfg), _ptr(stats), _stream(stream))
    _check(st, "gdn_chunk_fwd_noalloc")
    return O, S_out


def gdn_decode(Q, K, V, beta, g, S=None, scale: float | None = None, S_out=None, O=None,
               o_dtype=torch.bfloat16, stream=None):
    """Gated delta rule token by token with the state kept on chip for all n tokens.
    Q, K [B,H,n,d_k], V [B,H,n,d_v] (bf16 or fp32, one dtype); beta, g [B,H,n] fp32;
    S [B,H,d_k,d_v] fp32 or None (zeros).  Pass S_out=S to update the state in place.
    Returns (O [B,H,n,d_v], S_out [B,H,d_k,d_v] fp32)."""
    for t, n_ in ((Q, "Q"), (K, "K"), (V, "V")):
        _dev(t, n_, (torch.bfloat16, torch.float32))
    if not (Q.dtype == K.dtype == V.dtype):
        raise ValueError("Q, K and V must share one dtype")
    _dev(beta, "beta", (torch.float32,))
    _dev(g, "g", (torch.float32,))
    if K.dim() != 4 or Q.shape != K.shape:
        raise ValueError("Q and K must both be [B, H, n, d_k]")
    B, H, n, dk = K.shape
    dv = V.shape[-1]
    if V.shape[:3] != (B, H, n) or beta.shape != (B, H, n) or g.shape != (B, H, n):
        raise ValueError("V, beta, g must match Q/K in [B, H, n]")
    if S is not None:
        _dev(S, "S", (torch.float32,))
        if S.shape != (B, H, dk, dv):
            raise ValueError("S must be [B, H, d_k, d_v]")
    if O is None:
        O = torch.empty((B, H, n, dv), device=K.device, dtype=o_dtype)
    if S_out is None:
        S_out = torch.empty((B, H, dk, dv), device=K.device, dtype=torch.float32)
    _dev(O, "O", (torch.float32, torch.bfloat16))
    _dev(S_out, "S_out", (torch.float32,))
    if scale is None:
        scale = dk ** -0.5
    st = _lib.gdn_decode(_ptr(Q), _ptr(K), _ptr(V), _TORCH_DTYPE[K.dtype], _ptr(beta), _ptr(g),
                         _ptr(S), _ptr(S_out), _ptr(O), _TORCH_DTYPE[O.dtype], B, H, n, dk, dv,
                         float(scale), _stream(stream))
    _check(st, "gdn_decode")
    return O, S_out


# ---- linear attention with a decay for each head, and the norms around it -------------------
# Launches run on the tensors' device, whichever device is current.  With an explicit stream
# everything allocated here belongs to that stream, so that no other stream's work can be
# given a workspace that is still in use.

_BF16, _FLOAT = (torch.bfloat16,), (torch.float32, torch.bfloat16)
_ACT = {"silu": GDN_GATE_SILU, "sigmoid": GDN_GATE_SIGMOID}


class _Here:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE_SCOPE = _Here()


def _scope(dev, stream):
    """Context in which dev is the current device and, if given, stream the current stream."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, dev))
        return torch.cuda.stream(stream)
    return _HERE_SCOPE if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _current(dev):
    """The current stream of dev as the library takes it (without building a Stream object: the
    calls of a decode step cost more on the host than their kernels take)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _at(t):
    return None if t is None else t.data_ptr()


def _arg(t, name, dtypes, shape, dev):
    """A required tensor: on dev (None: any GPU), contiguous, of one of dtypes, of this shape."""
    if (type(t) is torch.Tensor and t.shape == shape and t.dtype in dtypes and t.is_contiguous()
            and (t.is_cuda if dev is None else t.get_device() == dev.index)):
        return t
    _dev(t, name, dtypes)
    if t is None:
        raise TypeError("%s is required" % name)
    if dev is not None and t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _out(t, name, dtypes, shape, dev, dtype, like=None):
    """An output: the caller's tensor after its checks, or a new one (like: a contiguous tensor of
    this shape, which makes a new one of the same type cheaper)."""
    if t is None:
        if dtype not in dtypes:
            raise TypeError("%s has dtype %s, expected one of %s" % (name, dtype, dtypes))
        if like is not None and like.dtype is dtype:
            return torch.empty_like(like)
        return torch.empty(shape, device=dev, dtype=dtype)
    return _arg(t, name, dtypes, shape, dev)


def _scratch(workspace, need, dev):
    if workspace is None:
        return (torch.empty(need, device=dev, dtype=torch.uint8), need) if need else (None, 0)
    _dev(workspace, "workspace")
    if workspace.device != dev:
        raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
    return workspace, workspace.numel() * workspace.element_size()


def _lin_shape(Q, K, V, g, scale, offsets, dtypes):
    """The gdn_lin_shape of a call after the inputs' checks; returns (shape, the states' shape, device)."""
    if K is None or K.dim() != 4 or V is None or V.dim() != 4:
        raise ValueError("Q and K must be [B, H_qk, T, d_k], V [B, H, T, d_v]")
    B, Hk, T, dk = K.shape
    H, dv = V.shape[1], V.shape[3]
    dev = K.device
    _arg(K, "K", dtypes, (B, Hk, T, dk), None)
    _arg(Q, "Q", (K.dtype,), (B, Hk, T, dk), dev)
    _arg(V, "V", (K.dtype,), (B, H, T, dv), dev)
    if Hk == 0 or H % Hk != 0:
        raise ValueError("the %d heads of V cannot share the %d heads of Q and K" % (H, Hk))
    per_head = g is not None and g.dim() == 1
    _arg(g, "g", (torch.float32,), (H,) if per_head else (B, H, T), dev)
    n = B
    if offsets is not None:
        if B != 1:
            raise ValueError("packed sequences lie in one row: B must be 1, got %d" % B)
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("offsets must be [sequences + 1], of one sequence at least")
        n = offsets.numel() - 1
        _arg(offsets, "offsets", (torch.int32,), (n + 1,), dev)
    sh = gdn_lin_shape(T, _at(offsets), n, H, Hk, dk, dv, per_head, dk ** -0.5 if scale is None else float(scale))
    return sh, (n, H, dk, dv), dev


def _plain_shape(B, H, H_qk, T, d_k, d_v, packed):
    # of the offsets only their presence counts
    return gdn_lin_shape(int(T), 16 if packed else None, int(B), int(H), int(H_qk), int(d_k), int(d_v), 1, 1.0)


def gdn_lin_chunk_fwd_workspace_bytes(B: int, H: int, T: int, d_k: int, d_v: int, H_qk: int | None = None,
                                      packed: bool = False) -> int:
    """Device workspace (bytes) gdn_lin_chunk_fwd needs for B sequences (0: none)."""
    return int(_lib.gdn_lin_chunk_fwd_workspace_bytes(
        ctypes.byref(_plain_shape(B, H, H if H_qk is None else H_qk, T, d_k, d_v, packed))))


def gdn_lin_chunk_bwd_workspace_bytes(B: int, H: int, T: int, d_k: int, d_v: int, H_qk: int | None = None,
                                      packed: bool = False) -> int:
    """Device workspace (bytes) gdn_lin_chunk_bwd needs for B sequences."""
    return int(_lib.gdn_lin_chunk_bwd_workspace_bytes(
        ctypes.byref(_plain_shape(B, H, H if H_qk is None else H_qk, T, d_k, d_v, packed))))


def gdn_lin_chunk_fwd(Q, K, V, g, scale: float | None = None, S0=None, offsets=None, o_dtype=torch.bfloat16,
                      O=None, S_out=None, workspace=None, stream=None):
    """Linear attention with a decay for each head, whole sequences:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    Q, K [B,H_qk,T,d_k], V [B,H,T,d_v] bf16 (H_qk divides H); g fp32, [B,H,T] log-decays or
    [H] for one decay per head.  offsets: int32 [n+1] for n packed sequences in B = 1 rows of
    T tokens.  S0 [B or n,H,d_k,d_v] fp32 or None (zeros; not the same tensor as S_out).  Any T.  workspace: a uint8 tensor
    of gdn_lin_chunk_fwd_workspace_bytes(...) bytes, or None to have one allocated here.
    Returns (O [B,H,T,d_v], S_out [B or n,H,d_k,d_v] fp32)."""
    sh, state, dev = _lin_shape(Q, K, V, g, scale, offsets, _BF16)
    if S0 is not None:
        _arg(S0, "S0", (torch.float32,), state, dev)
    with _scope(dev, stream):
        O = _out(O, "O", _FLOAT, V.shape, dev, o_dtype, V)
        S_out = _out(S_out, "S_out", (torch.float32,), state, dev, torch.float32, S0)
        if S0 is not None and S_out.data_ptr() == S0.data_ptr() and S0.numel():
            raise ValueError("S_out must not be S0: a sequence's parts read the one while others write the other")
        ws, ws_bytes = _scratch(workspace, _lib.gdn_lin_chunk_fwd_workspace_bytes(ctypes.byref(sh)), dev)
        st = _lib.gdn_lin_chunk_fwd(ctypes.byref(sh), _at(Q), _at(K), _at(V), GDN_BF16, _at(g), _at(S0), _at(O),
                                    _TORCH_DTYPE[O.dtype], _at(S_out), _at(ws), ws_bytes, _current(dev))
    _check(st, "gdn_lin_chunk_fwd")
    return O, S_out


def gdn_lin_chunk_bwd(Q, K, V, g, dO, scale: float | None = None, S0=None, dS=None, offsets=None,
                      grad_dtype=torch.bfloat16, want_dg: bool = True, workspace=None, stream=None):
    """Backward pass of gdn_lin_chunk_fwd from dO [B,H,T,d_v] (bf16) and dS (gradient of
    S_out, or None).  Returns (dQ, dK, dV in grad_dtype, dg fp32 as g or None, dS0 fp32, or
    None without S0)."""
    sh, state, dev = _lin_shape(Q, K, V, g, scale, offsets, _BF16)
    _arg(dO, "dO", _BF16, V.shape, dev)
    for t, name in ((S0, "S0"), (dS, "dS")):
        if t is not None:
            _arg(t, name, (torch.float32,), state, dev)
    if grad_dtype not in _FLOAT:
        raise TypeError("grad_dtype is %s, expected one of %s" % (grad_dtype, _FLOAT))
    with _scope(dev, stream):
        dQ, dK, dV = (torch.empty(t.shape, device=dev, dtype=grad_dtype) for t in (Q, K, V))
        dg = torch.empty_like(g) if want_dg else None
        dS0 = None if S0 is None else torch.empty(state, device=dev, dtype=torch.float32)
        ws, ws_bytes = _scratch(workspace, _lib.gdn_lin_chunk_bwd_workspace_bytes(ctypes.byref(sh)), dev)
        st = _lib.gdn_lin_chunk_bwd(ctypes.byref(sh), _at(Q), _at(K), _at(V), GDN_BF16, _at(g), _at(S0), _at(dO),
                                    _at(dS), _at(dQ), _at(dK), _at(dV), _TORCH_DTYPE[grad_dtype], _at(dg),
                                    _at(dS0), _at(ws), ws_bytes, _current(dev))
    _check(st, "gdn_lin_chunk_bwd")
    return dQ, dK, dV, dg, dS0


def gdn_lin_decode(Q, K, V, g, S=None, scale: float | None = None, S_out=None, O=None, o_dtype=torch.bfloat16,
                   stream=None):
    """The recurrence of gdn_lin_chunk_fwd token by token with the state kept on chip.
    Q, K [B,H_qk,n,d_k], V [B,H,n,d_v] (bf16 or fp32, one dtype), g [B,H,n] or [H] fp32,
    S [B,H,d_k,d_v] fp32 or None (zeros).  Pass S_out=S to update the state in place.
    Returns (O [B,H,n,d_v], S_out)."""
    sh, state, dev = _lin_shape(Q, K, V, g, scale, None, _FLOAT)
    if S is not None:
        _arg(S, "S", (torch.float32,), state, dev)
    with _scope(dev, stream):
        O = _out(O, "O", _FLOAT, V.shape, dev, o_dtype, V)
        S_out = _out(S_out, "S_out", (torch.float32,), state, dev, torch.float32, S)
        st = _lib.gdn_lin_decode(ctypes.byref(sh), _at(Q), _at(K), _at(V), _TORCH_DTYPE[K.dtype], _at(g), _at(S),
                                 _at(S_out), _at(O), _TORCH_DTYPE[O.dtype], _current(dev))
    _check(st, "gdn_lin_decode")
    return O, S_out


def _gate_args(O, Z, w, act):
    """Checks of the gated norm's inputs; returns (B, H, T, d, Z's token stride, device)."""
    if O is None or O.dim() != 4:
        raise ValueError("O must be [B, H, T, d]")
    B, H, T, d = O.shape
    dev = O.device
    _arg(O, "O", _FLOAT, (B, H, T, d), None)
    if not isinstance(Z, torch.Tensor) or not Z.is_cuda or Z.dtype != O.dtype:
        raise TypeError("Z must be a CUDA (HIP) tensor of O's dtype")
    if Z.device != dev:
        raise ValueError("Z is on %s, expected %s" % (Z.device, dev))
    if tuple(Z.shape) != (B, T, H, d):
        raise ValueError("Z must be %s, got %s" % ((B, T, H, d), tuple(Z.shape)))
    # tokens at any stride (a part of a wider projection), the values of a token together
    step = Z.stride(1) if T > 1 else Z.stride(0) if B > 1 else H * d
    if Z.numel() and ((d > 1 and Z.stride(3) != 1) or (H > 1 and Z.stride(2) != d) or
                      (B > 1 and T > 1 and Z.stride(0) != T * step) or step < H * d):
        raise ValueError("Z's heads must be contiguous within a token and its tokens at one stride")
    if not Z.numel():
        step = H * d
    if w is not None:
        _arg(w, "w", (torch.float32,), (d,), dev)
    if act not in _ACT:
        raise ValueError("act must be one of %s" % (tuple(_ACT),))
    return B, H, T, d, step, dev


def gdn_gate_norm_fwd(O, Z, w=None, eps: float = 1e-6, act: str = "silu", Y=None, stream=None):
    """Gated norm of the head outputs: O [B,H,T,d] (as gdn_lin_chunk_fwd, gdn_chunk_fwd and the
    decode entry points return it), Z [B,T,H,d] (its tokens at any stride), w [d] fp32 or None
    -> Y [B,T,H,d] = O / rms(O) * w * act(Z), act "silu" or "sigmoid"; O, Z, Y bf16 or fp32."""
    B, H, T, d, step, dev = _gate_args(O, Z, w, act)
    with _scope(dev, stream):
        Y = _out(Y, "Y", (O.dtype,), (B, T, H, d), dev, O.dtype)
        st = _lib.gdn_gate_norm_fwd(_at(O), _at(Z), step, _at(w), _at(Y), _TORCH_DTYPE[O.dtype], B, H, T, d,
                                    _ACT[act], float(eps), _current(dev))
    _check(st, "gdn_gate_norm_fwd")
    return Y


def gdn_gate_norm_bwd(dY, O, Z, w=None, eps: float = 1e-6, act: str = "silu", workspace=None, stream=None):
    """Backward pass of gdn_gate_norm_fwd from dY [B,T,H,d].  Returns (dO [B,H,T,d],
    dZ [B,T,H,d], dw [d] fp32, or None without w)."""
    B, H, T, d, step, dev = _gate_args(O, Z, w, act)
    _arg(dY, "dY", (O.dtype,), (B, T, H, d), dev)
    with _scope(dev, stream):
        dO = torch.empty_like(O)
        dZ = torch.empty((B, T, H, d), device=dev, dtype=O.dtype)
        dw = None if w is None else torch.empty((d,), device=dev, dtype=torch.float32)
        ws, ws_bytes = (None, 0) if dw is None else _scratch(
            workspace, _lib.gdn_gate_norm_bwd_workspace_bytes(B, H, T, d), dev)
        st = _lib.gdn_gate_norm_bwd(_at(dY), _at(O), _at(Z), step, _at(w), _at(dO), _at(dZ), _at(dw),
                                    _TORCH_DTYPE[O.dtype], B, H, T, d, _ACT[act], float(eps), _at(ws), ws_bytes,
                                    _current(dev))
    _check(st, "gdn_gate_norm_bwd")
    return dO, dZ, dw


def _res_args(X, Y, w_post, s, w_pre, x_name):
    """Checks of the residual norm's inputs; returns (rows, D, device)."""
    if X is None or X.dim() < 1:
        raise ValueError("%s must be [.., D]" % x_name)
    dev, D = X.device, X.shape[-1]
    _arg(X, x_name, _FLOAT, X.shape, None)
    _arg(Y, "Y", _FLOAT, X.shape, dev)
    for t, name in ((w_post, "w_post"), (s, "s"), (w_pre, "w_pre")):
        if t is not None:
            _arg(t, name, (torch.float32,), (D,), dev)
    return (X.numel() // D if D else 0), D, dev


def gdn_residual_norm_fwd(X, Y, w_post=None, s=None, alpha: float = 1.0, w_pre=None, eps: float = 1e-6,
                          want_norm: bool = True, R=None, N=None, stream=None):
    """Residual sum with the norms around it: R = X + alpha s * (rms(Y) * w_post) and
    N = rms(R) * w_pre, over rows of D (X, Y [.., D], bf16 or fp32 each; R as X, N as Y).
    w_post None: Y is not normed; s, w_pre None: ones; want_norm=False: N is None.  R may be X.
    Returns (R, N)."""
    rows, D, dev = _res_args(X, Y, w_post, s, w_pre, "X")
    with _scope(dev, stream):
        R = _out(R, "R", (X.dtype,), X.shape, dev, X.dtype, X)
        N = _out(N, "N", (Y.dtype,), Y.shape, dev, Y.dtype, Y) if want_norm else None
        st = _lib.gdn_residual_norm_fwd(_at(X), _TORCH_DTYPE[X.dtype], _at(Y), _TORCH_DTYPE[Y.dtype], _at(w_post),
                                        _at(s), float(alpha), _at(w_pre), _at(R), _at(N), rows, D, float(eps),
                                        _current(dev))
    _check(st, "gdn_residual_norm_fwd")
    return R, N


def gdn_residual_norm_bwd(dN, dR, R, Y, w_post=None, s=None, alpha: float = 1.0, w_pre=None, eps: float = 1e-6,
                          workspace=None, stream=None):
    """Backward pass of gdn_residual_norm_fwd from dN (as Y) and dR (as R), either None for
    zeros, with the R that the forward pass returned.  Returns (dX, dY, dw_pre, dw_post, ds),
    the last three fp32 [D], each None without its factor (dw_pre also without dN)."""
    rows, D, dev = _res_args(R, Y, w_post, s, w_pre, "R")
    if dN is not None:
        _arg(dN, "dN", (Y.dtype,), Y.shape, dev)
    if dR is not None:
        _arg(dR, "dR", (R.dtype,), R.shape, dev)
    with _scope(dev, stream):
        dX, dY = torch.empty_like(R), torch.empty_like(Y)
        vec = lambda t: None if t is None else torch.empty((D,), device=dev, dtype=torch.float32)  # noqa: E731
        dw_pre, dw_post, ds = vec(w_pre if dN is not None else None), vec(w_post), vec(s)
        ws, ws_bytes = (None, 0) if dw_pre is dw_post is ds is None else _scratch(
            workspace, _lib.gdn_residual_norm_bwd_workspace_bytes(rows, D), dev)
        st = _lib.gdn_residual_norm_bwd(_at(dN), _at(dR), _at(R), _TORCH_DTYPE[R.dtype], _at(Y),
                                        _TORCH_DTYPE[Y.dtype], _at(w_post), _at(s), float(alpha), _at(w_pre),
                                        _at(dX), _at(dY), _at(dw_pre), _at(dw_post), _at(ds), rows, D, float(eps),
                                        _at(ws), ws_bytes, _current(dev))
    _check(st, "gdn_residual_norm_bwd")
    return dX, dY, dw_pre, dw_post, ds
