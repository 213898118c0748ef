"""GPU parity of the gated norm and the residual norm (forward and backward) against fp64.

fp32 arithmetic on the values as given: a row's sum of squares (at most 16384 terms, added in
8 lanes' runs and trees) is right to 2^-20, exponentials and divisions to 2^-21, so an element
is right to TOL = 2^-18 of M, the same expression over absolute values; outputs stored in bf16
add half a step, 2^-8 of the value.  Gradients of weights are sums over rows in fp32 and fp64:
2^-17 of the sum of absolute values."""
import ctypes

import pytest
import torch

import lin_reference as ref
from helpers import cuda, say

tri = pytest.importorskip("tri_inverse_amd")
gpu = pytest.mark.gpu
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


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_reference_gradients(act):
    """The references against differences (gradcheck) in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64, requires_grad=True)  # noqa: E731
    O, Z, w = r(2, 3, 2, 4), r(2, 2, 3, 4), r(4)
    assert torch.autograd.gradcheck(lambda *a: ref.gate_norm(*a, 1e-6, act), (O, Z, w))
    X, Y, wp, s, wq = r(3, 4), r(3, 4), r(4), r(4), r(4)
    assert torch.autograd.gradcheck(lambda x, y, a, b, c: ref.residual_norm(x, y, a, b, 0.7, c, 1e-6), (X, Y, wp, s, wq))
    dy, x, v = r(3, 4), r(3, 4), r(4)
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    gx, gw = torch.autograd.grad((n * v * dy.detach()).sum(), (x, v))
    got = rms_bwd(dy.detach(), x.detach(), v.detach(), 1e-6)
    assert torch.allclose(gx, got[0]) and torch.allclose(gw, got[2])


def gate_inputs(seed, B, H, T, d, dtype, extra):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    Z = (r(B, T, H * d + extra) * 3)[..., :H * d].unflatten(-1, (H, d))
    return r(B, H, T, d), Z, 1 + 0.2 * torch.randn(d, generator=g), r(B, T, H, d)


def on_gpu(Z, extra):
    """Z on the GPU with its token stride kept."""
    B, T, H, d = Z.shape
    wide = torch.full((B, T, H * d + extra), float("nan"), device="cuda", dtype=Z.dtype)
    wide[..., :H * d] = Z.flatten(2).cuda()
    return wide[..., :H * d].unflatten(-1, (H, d))


GATES = [(1, 1, 1, 32, 0), (2, 3, 5, 64, 8), (1, 4, 77, 96, 0), (3, 2, 33, 128, 264), (1, 16, 130, 128, 0),
         (2, 5, 9, 160, 16), (1, 3, 300, 256, 0), (2, 1, 1, 224, 8)]


@gpu
@pytest.mark.parametrize("case", GATES, ids=[str(i) for i in range(len(GATES))])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gate_norm(case, dtype, act):
    B, H, T, d, extra = case
    say(f"gate norm {case} {dtype} {act}")
    O, Z, w, dY = gate_inputs(7, B, H, T, d, dtype, extra)
    O[0, 0, 0] = 0  # a row of zeros: the norm is eps alone
    for wt in (w, None):
        Zc = on_gpu(Z, extra)
        Y = tri.gdn_gate_norm_fwd(cuda(O), Zc, None if wt is None else cuda(wt), eps=1e-5, act=act)
        dO, dZ, dw = tri.gdn_gate_norm_bwd(cuda(dY), cuda(O), Zc, None if wt is None else cuda(wt), eps=1e-5, act=act)
        torch.cuda.synchronize()
        want = ref.gate_norm(O, Z, wt, 1e-5, act)
        close(Y, want, want.abs(), TOL, "Y")
        z, o, dy = Z.double(), O.double().transpose(1, 2), dY.double()
        sg = torch.sigmoid(z)
        f = z * sg if act == "silu" else sg
        df = sg * (1 + z * (1 - sg)) if act == "silu" else sg * (1 - sg)
        mdf = sg * (1 + z.abs() * (1 - sg)) + (sg if act == "silu" else 0) if act == "silu" else sg
        wd = torch.ones(d).double() if wt is None else wt.double()
        dx, mx, gw, mw = rms_bwd(dy * f, o, wd, 1e-5)
        n = o / torch.sqrt(o.square().mean(-1, keepdim=True) + 1e-5)
        close(dO.transpose(1, 2), dx, mx, TOL, "dO")
        close(dZ, dy * n * wd * df, (dy * n * wd * mdf).abs(), TOL, "dZ")
        if wt is None:
            assert dw is None
        else:
            close(dw, gw, mw, TOL_W, "dw")


@gpu
def test_gate_norm_far_gates():
    """Gates whose exponential overflows or vanishes."""
    say("gate norm far gates")
    O = torch.ones((1, 1, 4, 32))
    Z = torch.tensor([-200.0, -90.0, 90.0, 200.0]).view(1, 4, 1, 1).expand(1, 4, 1, 32).contiguous()
    for act in ("silu", "sigmoid"):
        Y = tri.gdn_gate_norm_fwd(cuda(O), cuda(Z), act=act, eps=0.0)
        dO, dZ, _ = tri.gdn_gate_norm_bwd(torch.ones((1, 4, 1, 32), device="cuda"), cuda(O), cuda(Z), act=act, eps=0.0)
        torch.cuda.synchronize()
        want = ref.gate_norm(O, Z, None, 0.0, act)
        assert torch.allclose(Y.cpu().double(), want, rtol=1e-5, atol=1e-30)
        assert torch.isfinite(dO).all() and torch.isfinite(dZ).all()


ROWS = [(1, 8), (5, 64), (64, 512), (7, 520), (33, 1000), (3, 2048), (130, 2056), (9, 4096), (600, 328), (2, 8192),
        (3, 8200), (2, 16384)]


@gpu
@pytest.mark.parametrize("rows,D", ROWS)
@pytest.mark.parametrize("xt,yt", [(F32, BF), (BF, BF), (F32, F32), (BF, F32)])
def test_residual_norm(rows, D, xt, yt):
    say(f"residual norm rows={rows} D={D} {xt} {yt}")
    g = torch.Generator().manual_seed(D + rows)
    X, Y = torch.randn((rows, D), generator=g).to(xt), (2 * torch.randn((rows, D), generator=g)).to(yt)
    dN, dR = torch.randn((rows, D), generator=g).to(yt), torch.randn((rows, D), generator=g).to(xt)
    Y[0] = 0
    vec = lambda: 1 + 0.3 * torch.randn(D, generator=g)  # noqa: E731
    wq, s, wp = vec(), vec(), vec()
    up = lambda t: None if t is None else cuda(t)  # noqa: E731
    for a, b, c in ((wq, s, wp), (None, None, wp), (wq, None, None), (None, s, wp)):
        R, N = tri.gdn_residual_norm_fwd(cuda(X), cuda(Y), w_post=up(a), s=up(b), alpha=0.6, w_pre=up(c), eps=1e-5)
        R1, N1 = tri.gdn_residual_norm_fwd(cuda(X), cuda(Y), w_post=up(a), s=up(b), alpha=0.6, w_pre=up(c), eps=1e-5,
                                           want_norm=False)
        got = tri.gdn_residual_norm_bwd(cuda(dN), cuda(dR), cuda(X), cuda(Y), w_post=up(a), s=up(b), alpha=0.6,
                                        w_pre=up(c), eps=1e-5)
        torch.cuda.synchronize()
        r, n = ref.residual_norm(X, Y, a, b, 0.6, c, 1e-5)
        x, y = X.double(), Y.double()
        A, B_, Cw = (torch.ones(D).double() if t is None else t.double() for t in (a, b, c))
        yn = y * (y.square().mean(-1, keepdim=True) + 1e-5).rsqrt() if a is not None else y
        z = yn * A
        mr = x.abs() + (0.6 * B_ * z).abs()
        close(R, r, mr, TOL, "R")
        # N: the sum's own error, and the row's error through its norm
        rs = (r.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
        close(N, n, (mr * rs * Cw.abs()) + n.abs() * (mr.square().mean(-1, keepdim=True).sqrt() * rs), 2 * TOL, "N")
        assert N1 is None and torch.equal(R1, R)
        dr, m1, gp, mp = rms_bwd(dN.double(), x, Cw, 1e-5)
        dr, m1 = dr + dR.double(), m1 + dR.double().abs()
        dz, mz = 0.6 * dr * B_, 0.6 * m1 * B_.abs()
        if a is not None:
            dy, my, gq, _ = rms_bwd(dz, y, A, 1e-5)
            _, my, _, mq = rms_bwd(mz, y.abs(), A.abs(), 1e-5)
        else:
            dy, my = dz, mz
        close(got[0], dr, m1, TOL, "dX")
        close(got[1], dy, my, 2 * TOL, "dY")
        if c is None:
            assert got[2] is None
        else:
            close(got[2], gp, mp, TOL_W, "dw_pre")
        if a is None:
            assert got[3] is None
        else:
            close(got[3], gq, mq, TOL_W, "dw_post")
        if b is None:
            assert got[4] is None
        else:
            close(got[4], (0.6 * dr * z).sum(0), (0.6 * m1 * z.abs()).sum(0), TOL_W, "ds")


@gpu
def test_residual_norm_partial_gradients_and_in_place():
    say("residual norm partial gradients, in place")
    g = torch.Generator().manual_seed(5)
    X, Y, dR = (torch.randn((6, 96), generator=g) for _ in range(3))
    w = 1 + 0.1 * torch.randn(96, generator=g)
    dX, dY, *rest = tri.gdn_residual_norm_bwd(None, cuda(dR), cuda(X), cuda(Y), alpha=2.0, w_pre=cuda(w))
    torch.cuda.synchronize()
    assert torch.equal(dX.cpu(), dR) and torch.equal(dY.cpu(), 2.0 * dR) and rest == [None, None, None]
    dX, dY, *_ = tri.gdn_residual_norm_bwd(None, None, cuda(X), cuda(Y))
    torch.cuda.synchronize()
    assert torch.count_nonzero(dX) == 0 and torch.count_nonzero(dY) == 0
    x = cuda(X)
    R, N = tri.gdn_residual_norm_fwd(x, cuda(Y), w_pre=cuda(w), R=x)
    R2, N2 = tri.gdn_residual_norm_fwd(cuda(X), cuda(Y), w_pre=cuda(w))
    torch.cuda.synchronize()
    assert R is x and torch.equal(R, R2) and torch.equal(N, N2)


@gpu
def test_no_rows():
    say("norms without rows")
    w = torch.ones(64, device="cuda")
    R, N = tri.gdn_residual_norm_fwd(torch.empty((0, 64), device="cuda"), torch.empty((0, 64), device="cuda"))
    out = tri.gdn_residual_norm_bwd(torch.empty((0, 64), device="cuda"), None, R, N, w_post=w, s=w, w_pre=w)
    O, Z = torch.empty((2, 3, 0, 64), device="cuda"), torch.empty((2, 0, 3, 64), device="cuda")
    Y = tri.gdn_gate_norm_fwd(O, Z, w)
    g = tri.gdn_gate_norm_bwd(Y, O, Z, w)
    torch.cuda.synchronize()
    assert all(torch.count_nonzero(t) == 0 and t.numel() == 64 for t in out[2:] + (g[2],))


@gpu
def test_norms_captured():
    say("norms captured")
    g = torch.Generator().manual_seed(8)
    X, Y, dN = (cuda(torch.randn((300, 512), generator=g)) for _ in range(3))
    w = cuda(1 + 0.1 * torch.randn(512, generator=g))
    O, Z = cuda(torch.randn((2, 3, 100, 64), generator=g)), cuda(torch.randn((2, 100, 3, 64), generator=g))

    def both():
        return (tri.gdn_residual_norm_fwd(X, Y, w_post=w, s=w, w_pre=w) +
                tri.gdn_residual_norm_bwd(dN, X, X, Y, w_post=w, s=w, w_pre=w) +
                tri.gdn_gate_norm_bwd(Z, O, Z, w[:64]) + (tri.gdn_gate_norm_fwd(O, Z, w[:64]),))

    eager = [t.clone() for t in both()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out)), i
        assert all(torch.equal(a, b) for a, b in zip(eager, both())), i


@gpu
def test_python_refusals():
    O, Z = torch.zeros((2, 3, 5, 64), device="cuda"), torch.zeros((2, 5, 3, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    X = torch.zeros((4, 64), device="cuda")
    gate, res = tri.gdn_gate_norm_fwd, tri.gdn_residual_norm_fwd
    for bad in (lambda: gate(O, Z.bfloat16()), lambda: gate(O, Z[:, :, :2]), lambda: gate(O, Z, w[:32]),
                lambda: gate(O, Z, act="relu"), lambda: gate(O, Z.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: gate(O.transpose(1, 2), Z), lambda: gate(O, Z.cpu()), lambda: gate(O, Z[:, :1].expand(2, 5, 3, 64)),
                lambda: tri.gdn_gate_norm_bwd(O, O, Z), lambda: res(X, X[:3]), lambda: res(X, X, s=w[:8]),
                lambda: res(X.half(), X), lambda: res(X, X, w_pre=w.double()),
                lambda: tri.gdn_residual_norm_bwd(X.bfloat16(), None, X, X)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(tri.GdnError):
        gate(torch.zeros((1, 1, 1, 48), device="cuda"), torch.zeros((1, 1, 1, 48), device="cuda"))
    with pytest.raises(tri.GdnError):
        res(torch.zeros((4, 12), device="cuda"), torch.zeros((4, 12), device="cuda"))


# ---- refusals of the C entry points, on the CPU ------------------------------------------------

FAKE = 0x10000


def test_c_refusals_gate():
    lib = tri._lib

    def fwd(O=FAKE, zs=256, w=None, dt=0, B=2, H=4, T=5, d=64, act=0, eps=1e-6):
        return lib.gdn_gate_norm_fwd(O, FAKE, zs, w, FAKE, dt, B, H, T, d, act, eps, None)

    def bwd(dO=FAKE, zs=256, dw=FAKE, dt=0, B=2, H=4, T=5, d=64, act=0, eps=1e-6, ws=FAKE, nb=1 << 30):
        return lib.gdn_gate_norm_bwd(FAKE, FAKE, FAKE, zs, FAKE, dO, FAKE, dw, dt, B, H, T, d, act, eps, ws, nb, None)

    for f in (fwd, bwd):
        assert f(B=-1) == 2 and f(d=0) == 2 and f(act=2) == 2 and f(eps=-1.0) == 2 and f(eps=float("nan")) == 2
        assert f(zs=248) == 2 and f(zs=260) == 4 and f(dt=2) == 3
        assert f(d=48) == 5 and f(d=288, zs=2048) == 5 and f(T=1 << 40) == 5
    assert fwd(T=0) == 0 and fwd(O=None) == 1 and fwd(w=FAKE + 4) == 4
    assert bwd(dO=None) == 1 and bwd(ws=None) == 6 and bwd(nb=8) == 6 and bwd(ws=FAKE + 8) == 4
    assert bwd(T=0, dw=None) == 0
    assert lib.gdn_gate_norm_bwd_workspace_bytes(2, 4, 5, 48) == 0
    assert lib.gdn_gate_norm_bwd_workspace_bytes(2, 4, 5, 64) > 0


def test_c_refusals_residual():
    lib = tri._lib

    def fwd(X=FAKE, xt=0, yt=1, w=None, rows=3, D=64, eps=1e-6):
        return lib.gdn_residual_norm_fwd(X, xt, FAKE, yt, w, None, 1.0, None, FAKE, FAKE, rows, D, eps, None)

    def bwd(R=FAKE, xt=0, yt=1, wq=FAKE, s=FAKE, dwq=FAKE, ds=FAKE, rows=3, D=64, eps=1e-6, ws=FAKE, nb=1 << 30):
        return lib.gdn_residual_norm_bwd(FAKE, FAKE, R, xt, FAKE, yt, wq, s, 1.0, None, FAKE, FAKE, FAKE, dwq, ds, rows,
                                         D, eps, ws, nb, None)

    for f in (fwd, bwd):
        assert f(rows=-1) == 2 and f(D=0) == 2 and f(eps=-1.0) == 2 and f(xt=2) == 3 and f(yt=4) == 3
        assert f(D=12) == 5 and f(D=16392) == 5
    assert fwd(rows=0) == 0 and fwd(X=None) == 1 and fwd(w=FAKE + 4) == 4
    assert bwd(R=None) == 1 and bwd(wq=None) == 1 and bwd(s=None) == 1
    assert bwd(ws=None) == 6 and bwd(nb=8) == 6 and bwd(ws=FAKE + 8) == 4
    assert lib.gdn_residual_norm_bwd_workspace_bytes(3, 12) == 0
    assert lib.gdn_residual_norm_bwd_workspace_bytes(3, 64) > 0
