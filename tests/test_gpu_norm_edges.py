"""The norms' gradients where they can go wrong: eps = 0 with numbers of rows that leave part of a
workgroup without a row; gates far from 0; more rows than all workgroups take at a time; the delta
rule's outputs in front of them.

Tolerances: fp32 arithmetic on the values as given, a row's sums right to 2^-20 and exponentials
and divisions to 2^-21, so an element is right to 2^-18 of M, the same expression over absolute
values; gradients of weights, sums over rows in fp32 and fp64, to 2^-17 of the sum of absolute
values; outputs stored in bf16 add half a step, 2^-8 of the value."""
import pytest
import torch

import lin_reference as ref
from helpers import cuda, say

tri = pytest.importorskip("tri_inverse_amd")
pytestmark = pytest.mark.gpu
TOL, TOL_W = 2.0 ** -18, 2.0 ** -17
BF, F32 = torch.bfloat16, torch.float32


def close(got, want, mag, tol, what):
    got = got.detach().cpu()
    assert tuple(got.shape) == tuple(want.shape), what
    half = 2.0 ** -8 if got.dtype == BF else 0.0
    assert torch.isfinite(got).all(), what
    room = tol * mag + half * (want.abs() + tol * mag) + 1e-30
    worst = float(((got.double() - want).abs() / room).max()) if want.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g of its tolerance" % (what, worst)


def rms_bwd(dy, x, w, eps):
    """Gradient of rms(x) w with respect to x and w, and their magnitudes."""
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n, u = x * rstd, dy * w
    dx = rstd * (u - n * (u * n).mean(-1, keepdim=True))
    mx = rstd * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True))
    axes = tuple(range(x.dim() - 1))
    return dx, mx, (dy * n).sum(axes), (dy * n).abs().sum(axes)


def check_gate(O, Z, w, dY, eps):
    """Forward and backward of the gated norm with the SiLU gate against fp64."""
    Y = tri.gdn_gate_norm_fwd(cuda(O), cuda(Z), cuda(w), eps=eps)
    dO, dZ, dw = tri.gdn_gate_norm_bwd(cuda(dY), cuda(O), cuda(Z), cuda(w), eps=eps)
    torch.cuda.synchronize()
    want = ref.gate_norm(O, Z, w, eps, "silu")
    close(Y, want, want.abs(), TOL, "Y")
    z, o, dy, wd = Z.double(), O.double().transpose(1, 2), dY.double(), w.double()
    sg = torch.sigmoid(z)
    dx, mx, gw, mw = rms_bwd(dy * z * sg, o, wd, eps)
    n = o * (o.square().mean(-1, keepdim=True) + eps).rsqrt()
    close(dO.transpose(1, 2), dx, mx, TOL, "dO")
    rest = torch.sigmoid(-z)
    close(dZ, dy * n * wd * sg * (1 + z * rest), (dy * n * wd).abs() * sg * (1 + z.abs() * rest), TOL, "dZ")
    close(dw, gw, mw, TOL_W, "dw")


def check_residual(X, Y, dN, dR, wq, s, wp, eps):
    """Backward of the residual norm (X stands for the sum R) with every factor against fp64."""
    got = tri.gdn_residual_norm_bwd(cuda(dN), cuda(dR), cuda(X), cuda(Y), w_post=cuda(wq), s=cuda(s), alpha=0.6,
                                    w_pre=cuda(wp), eps=eps)
    torch.cuda.synchronize()
    x, y, A, B, Cw = X.double(), Y.double(), wq.double(), s.double(), wp.double()
    z = y * (y.square().mean(-1, keepdim=True) + eps).rsqrt() * A
    dr, m1, gp, mp = rms_bwd(dN.double(), x, Cw, eps)
    dr, m1 = dr + dR.double(), m1 + dR.double().abs()
    dy, _, gq, _ = rms_bwd(0.6 * dr * B, y, A, eps)
    _, my, _, mq = rms_bwd(0.6 * m1 * B.abs(), y.abs(), A.abs(), eps)
    close(got[0], dr, m1, TOL, "dX")
    close(got[1], dy, my, 2 * TOL, "dY")
    close(got[2], gp, mp, TOL_W, "dw_pre")
    close(got[3], gq, mq, TOL_W, "dw_post")
    close(got[4], (0.6 * dr * z).sum(0), (0.6 * m1 * z.abs()).sum(0), TOL_W, "ds")


def gate_inputs(seed, B, H, T, d, dtype):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    return r(B, H, T, d), 3 * r(B, T, H, d), 1 + 0.2 * torch.randn(d, generator=g), r(B, T, H, d)


def residual_inputs(seed, rows, D, xt, yt):
    g = torch.Generator().manual_seed(seed)
    r = lambda t: torch.randn((rows, D), generator=g).to(t)  # noqa: E731
    return (r(xt), 2 * r(yt), r(yt), r(xt)) + tuple(1 + 0.3 * torch.randn(D, generator=g) for _ in range(3))


@pytest.mark.parametrize("B,H,T,d", [(1, 1, 1, 32), (1, 1, 17, 128), (2, 3, 11, 96), (1, 1, 33, 256), (1, 3, 21, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gate_norm_without_eps(B, H, T, d, dtype):
    """Lanes past the last row hold zeros, whose norm would be infinite: they add nothing to dw."""
    say(f"gate norm eps=0 B={B} H={H} T={T} d={d} {dtype}")
    check_gate(*gate_inputs(T, B, H, T, d, dtype), eps=0.0)


@pytest.mark.parametrize("rows,D", [(1, 8), (2, 64), (3, 328), (5, 512), (7, 96), (1030, 64), (5, 1000)])
@pytest.mark.parametrize("xt,yt", [(F32, BF), (F32, F32)])
def test_residual_norm_without_eps(rows, D, xt, yt):
    say(f"residual norm eps=0 rows={rows} D={D} {xt} {yt}")
    check_residual(*residual_inputs(rows, rows, D, xt, yt), eps=0.0)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gate_derivative_far_from_zero(act):
    """dZ relative to itself: the derivative is e^-|z| in size for far gates of the sigmoid, for z > 0
    as for z < 0.  The exponential's argument in units of log 2 is rounded in the product (half a
    step, 2^-24 of it) and through log2 e (at most 2^-25): less than 2^-23 |z| of the derivative."""
    say(f"gate derivative {act}")
    z = torch.cat([torch.linspace(-30.0, 30.0, 241), torch.tensor([0.0, -1e-3, 1e-3, 10.0, 15.0, 17.0, 20.0])])
    T = z.numel()
    Z = z.view(1, T, 1, 1).expand(1, T, 1, 32).contiguous()
    O, dY = torch.ones((1, 1, T, 32)), torch.ones((1, T, 1, 32))
    _, dZ, _ = tri.gdn_gate_norm_bwd(cuda(dY), cuda(O), cuda(Z), eps=0.0, act=act)
    torch.cuda.synchronize()
    zd = Z.double()
    sg, rest = torch.sigmoid(zd), torch.sigmoid(-zd)
    want, mag = (sg * (1 + zd * rest), sg * (1 + zd.abs() * rest)) if act == "silu" else (sg * rest, sg * rest)
    close(dZ, want, mag, TOL + 2.0 ** -23 * zd.abs(), "dZ")


def test_gate_norm_rows_beyond_one_round():
    """More rows than all workgroups take at a time: each walks on, its column sums carried over."""
    say("gate norm, 22004 rows of 128")
    check_gate(*gate_inputs(3, 1, 4, 5501, 128, BF), eps=1e-5)


@pytest.mark.parametrize("rows,D", [(2100, 264), (1100, 520), (600, 2056), (1030, 4096)])
def test_residual_norm_rows_beyond_one_round(rows, D):
    say(f"residual norm backward, {rows} rows of {D}")
    check_residual(*residual_inputs(rows, rows, D, F32, BF), eps=1e-5)


@pytest.mark.parametrize("rows,D", [(8200, 264), (4100, 520), (2100, 2056)])
def test_residual_norm_forward_rows_beyond_one_round(rows, D):
    say(f"residual norm, {rows} rows of {D}")
    X, Y, _, _, wq, s, wp = residual_inputs(rows, rows, D, F32, BF)
    R, N = tri.gdn_residual_norm_fwd(cuda(X), cuda(Y), w_post=cuda(wq), s=cuda(s), alpha=0.6, w_pre=cuda(wp), eps=1e-5)
    torch.cuda.synchronize()
    r, n = ref.residual_norm(X, Y, wq, s, 0.6, wp, 1e-5)
    y = Y.double()
    z = y * (y.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * wq.double()
    mr = X.double().abs() + (0.6 * s.double() * z).abs()
    close(R, r, mr, TOL, "R")
    # N: the sum's own error, and the row's error through its norm
    rs = (r.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    close(N, n, mr * rs * wp.double().abs() + n.abs() * (mr.square().mean(-1, keepdim=True).sqrt() * rs), 2 * TOL, "N")


def test_gate_norm_behind_the_delta_rule():
    """The gated norm reads the gated delta rule's outputs as gdn_chunk_fwd and gdn_decode write them."""
    import synth

    say("gate norm behind gdn_chunk_fwd and gdn_decode")
    B, H, T, d = 2, 3, 192, 128
    x = {k: cuda(v) for k, v in synth.prefill(5, B, H, T, d, d).items() if isinstance(v, torch.Tensor)}
    g = torch.Generator().manual_seed(5)
    Z, w = torch.randn((B, T, H, d), generator=g).to(BF), 1 + 0.1 * torch.randn(d, generator=g)
    O, S = tri.gdn_chunk_fwd(x["Q"], x["K"], x["V"], x["beta"], x["g"], C=64, scale=d ** -0.5, N=3)
    Y = tri.gdn_gate_norm_fwd(O, cuda(Z), cuda(w))
    token = [x[k][:, :, :1].contiguous() for k in ("Q", "K", "V", "beta", "g")]
    o, _ = tri.gdn_decode(*token, S=S, scale=d ** -0.5)
    y = tri.gdn_gate_norm_fwd(o, cuda(Z[:, :1]), cuda(w))
    torch.cuda.synchronize()
    for out, got, z in ((O, Y, Z), (o, y, Z[:, :1])):
        assert out.dtype == BF and float(out.float().abs().max()) > 0
        want = ref.gate_norm(out.cpu(), z, w, 1e-6, "silu")
        close(got, want, want.abs(), TOL, "Y")
