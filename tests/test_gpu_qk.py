"""GPU parity of the norm and rotation of queries and keys (forward and backward) against fp64.

fp32 arithmetic on the values as given: a row's sum of squares (at most 256 terms) is right to 2^-20,
roots and divisions to 2^-22, cosines and sines to 2^-23 of 1, so an element is right to TOL = 2^-18 of
the same expression over absolute values, where either value of a turned pair counts as both;
outputs stored in bf16 add half a step, 2^-8 of the value.  Gradients of the weights are sums over
rows in fp32 and fp64: 2^-17 of the sum of absolute values."""
import ctypes
import math

import numpy as np
import pytest
import torch

import lin_reference
import rec_reference as ref
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


def up(t):
    return None if t is None else cuda(t)


def frequencies(r, base=10000.0):
    return torch.exp(-torch.arange(r // 2).double() * (2.0 / max(r, 1) * math.log(base)))


def inputs(seed, B, T, Hq, Hk, d, extra, dtype):
    """Queries and keys as parts of one projection's rows (CPU), and what they are called with."""
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn((B, T, (Hq + Hk) * d + extra), generator=g).to(dtype)
    rows[..., (Hq + Hk) * d:] = float("nan")
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return rows, 1 + 0.3 * r(d), 1 + 0.3 * r(d), r(B, Hq, T, d).to(dtype), r(B, Hk, T, d).to(dtype), g


def split(rows, Hq, Hk, d):
    return rows[..., :Hq * d].unflatten(-1, (Hq, d)), rows[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))


def check(rows, Hq, Hk, d, wq, wk, dQ, dK, freqs, pos, norm, eps, pairs, axis):
    """Forward and backward against the reference; pos None: the token's index."""
    gpu_rows = cuda(rows)
    Q, K = split(gpu_rows, Hq, Hk, d)
    how = dict(wq=up(wq), wk=up(wk), freqs=up(freqs), positions=up(pos), norm=norm, eps=eps, pairs=pairs, axis=axis)
    yq, yk = tri.gdn_qk_norm_fwd(Q, K, **how)
    got = tri.gdn_qk_norm_bwd(up(dQ), up(dK), Q, K, **how)
    torch.cuda.synchronize()
    B, T = rows.shape[:2]
    if pos is None:
        pos, axis = torch.arange(T).expand(B, T), None
    q, k = split(rows, Hq, Hk, d)
    for name, x, w, dy, y, dx, dw in (("Q", q, wq, dQ, yq, got[0], got[2]), ("K", k, wk, dK, yk, got[1], got[3])):
        want = ref.qk_forward(x, w, freqs, pos, norm, eps, pairs, axis)
        mag = want.abs()
        if freqs is not None:
            r = 2 * freqs.numel()
            at = (slice(0, r // 2), slice(r // 2, r)) if pairs == "halves" else (slice(0, r, 2), slice(1, r, 2))
            both = mag[..., at[0]] + mag[..., at[1]]
            mag[..., at[0]], mag[..., at[1]] = both, both
        close(y, want, mag, TOL, name)
        gx, mx, gw, mw = ref.qk_backward(dy, x, w, freqs, pos, norm, eps, pairs, axis)
        close(dx, gx, mx, TOL, "d" + name)
        if w is None:
            assert dw is None
        else:
            close(dw, gw, mw, TOL_W, "dw of " + name)


# B, T, Hq, Hk, d, rotated, extra values of a projection row
SHAPES = [(1, 1, 1, 1, 32, 32, 0), (2, 5, 3, 1, 64, 8, 8), (1, 77, 4, 4, 96, 64, 0), (3, 33, 2, 2, 128, 128, 264),
          (1, 130, 16, 4, 128, 0, 0), (2, 9, 5, 1, 160, 72, 16), (1, 300, 3, 3, 256, 256, 0), (2, 1, 1, 7, 224, 24, 8),
          (40, 1, 32, 16, 128, 64, 0), (1, 1000, 2, 1, 96, 96, 0)]


@gpu
@pytest.mark.parametrize("case", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_shapes(case, dtype, norm, pairs):
    B, T, Hq, Hk, d, r, extra = case
    say(f"queries and keys {case} {dtype} {norm} {pairs}")
    rows, wq, wk, dQ, dK, g = inputs(T + d, B, T, Hq, Hk, d, extra, dtype)
    rows[0, 0, :d] = 0  # a row of zeros: the norm is eps alone
    freqs = frequencies(r) if r else None
    pos = torch.randint(-5, 5000, (B, T), generator=g, dtype=torch.int32) if r and T % 2 else None
    check(rows, Hq, Hk, d, wq, wk, dQ, dK, freqs, pos, norm, 1e-5, pairs, None)


@gpu
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_axes(axes, pairs):
    """Runs of pairs for each axis, and axes that take turns; weights absent."""
    B, T, Hq, Hk, d, r = 2, 21, 3, 1, 96, 72
    say(f"queries and keys on {axes} axes, {pairs}")
    rows, _, _, dQ, dK, g = inputs(axes, B, T, Hq, Hk, d, 0, F32)
    pos = torch.randint(0, 400, (axes, B, T), generator=g, dtype=torch.int32)
    for axis in ([i * axes // (r // 2) for i in range(r // 2)], [i % axes for i in range(r // 2)]):
        check(rows, Hq, Hk, d, None, None, dQ, dK, frequencies(r), pos, "l2", 1e-6, pairs, axis)


@gpu
def test_far_positions():
    """Angles of positions up to 2^31 - 1 lose nothing: 2^-18 as of near ones."""
    say("queries and keys at far positions")
    T, d = 64, 128
    rows, wq, wk, dQ, dK, g = inputs(2, 1, T, 2, 2, d, 0, F32)
    pos = torch.randint(0, 2 ** 31 - 1, (1, T), generator=g, dtype=torch.int32)
    pos[0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 1_000_000, 0], dtype=torch.int32)
    # at 2^31 the angle of the reference and the kernel's are each right to 2^-21 radians, in fp64
    check(rows, 2, 2, d, wq, wk, dQ, dK, frequencies(d), pos, "rms", 1e-6, "halves", None)


@gpu
@pytest.mark.parametrize("T,d", [(1, 32), (17, 128), (11, 96), (9, 256)])
def test_without_eps(T, d):
    """Lanes past the last token hold zeros, whose norm would be infinite: they add nothing to dw."""
    say(f"queries and keys eps=0 T={T} d={d}")
    rows, wq, wk, dQ, dK, _ = inputs(T, 1, T, 3, 1, d, 0, F32)
    check(rows, 3, 1, d, wq, wk, dQ, dK, frequencies(32), None, "rms", 0.0, "halves", None)


@gpu
def test_one_tensor():
    """Queries alone and keys alone give what both together do."""
    say("queries alone, keys alone")
    rows, wq, wk, dQ, dK, _ = inputs(3, 2, 40, 4, 2, 64, 0, BF)
    Q, K = split(cuda(rows), 4, 2, 64)
    how = dict(freqs=cuda(frequencies(64)))
    q, k = tri.gdn_qk_norm_fwd(Q, K, cuda(wq), cuda(wk), **how)
    q1, none = tri.gdn_qk_norm_fwd(Q, None, cuda(wq), **how)
    none2, k1 = tri.gdn_qk_norm_fwd(None, K, None, cuda(wk), **how)
    g = tri.gdn_qk_norm_bwd(cuda(dQ), cuda(dK), Q, K, cuda(wq), cuda(wk), **how)
    gq = tri.gdn_qk_norm_bwd(cuda(dQ), None, Q, None, cuda(wq), **how)
    gk = tri.gdn_qk_norm_bwd(None, cuda(dK), None, K, None, cuda(wk), **how)
    torch.cuda.synchronize()
    assert none is none2 is gq[1] is gq[3] is gk[0] is gk[2] is None
    assert torch.equal(q, q1) and torch.equal(k, k1) and torch.equal(g[0], gq[0]) and torch.equal(g[1], gk[1])
    # other workgroups, so other partial sums of the weights' gradients
    assert torch.allclose(g[2], gq[2], rtol=1e-4, atol=1e-4) and torch.allclose(g[3], gk[3], rtol=1e-4, atol=1e-4)


@gpu
def test_tokens_beyond_one_round():
    """More pieces of work than the backward pass has workgroups: each walks on, its sums carried over."""
    say("queries and keys, 40003 tokens")
    rows, wq, wk, dQ, dK, _ = inputs(5, 1, 40003, 2, 1, 32, 0, BF)
    check(rows, 2, 1, 32, wq, wk, dQ, dK, frequencies(32), None, "rms", 1e-6, "neighbours", None)


@gpu
def test_no_rows():
    say("queries and keys without rows")
    w = torch.ones(64, device="cuda")
    E, G = torch.empty((2, 0, 3, 64), device="cuda"), torch.empty((2, 3, 0, 64), device="cuda")
    q, k = tri.gdn_qk_norm_fwd(E, E, w, w)
    g = tri.gdn_qk_norm_bwd(G, G, E, E, w, w)
    torch.cuda.synchronize()
    assert q.shape == k.shape == (2, 3, 0, 64) and g[0].shape == (2, 0, 3, 64)
    assert all(torch.count_nonzero(t) == 0 and t.numel() == 64 for t in g[2:])


@gpu
def test_captured_and_on_two_streams():
    say("queries and keys captured, two streams")
    rows, wq, wk, dQ, dK, _ = inputs(6, 2, 300, 8, 2, 128, 8, BF)
    Q, K = split(cuda(rows), 8, 2, 128)
    wq, wk, dQ, dK, freqs = (cuda(t) for t in (wq, wk, dQ, dK, frequencies(64)))

    def both(stream=None):
        return (tri.gdn_qk_norm_fwd(Q, K, wq, wk, freqs, stream=stream) +
                tri.gdn_qk_norm_bwd(dQ, dK, Q, K, wq, wk, freqs, stream=stream))

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
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    rounds = [[both(s) for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in rounds for o in r for a, b in zip(eager, o))


@gpu
def test_mixer_layer():
    """A mixer's layer as it is used: projection rows -> queries and keys -> linear attention (whole prompt,
    then one token) -> gated norm, each against fp64 on the inputs that it was given; and the delta rule
    on unit rows."""
    import synth

    say("queries and keys, linear attention, gated norm")
    B, T, Hq, H, d = 2, 130, 2, 4, 128
    rows, wq, wk, _, _, g = inputs(9, B, T + 1, Hq, Hq, d, 0, BF)
    V = torch.randn((B, H, T + 1, d), generator=g).to(BF)
    decay = -torch.exp2(-2.0 - 5.0 * torch.rand(H, generator=g))
    Z = torch.randn((B, T + 1, H, d), generator=g).to(BF)
    freqs, wo = frequencies(64), 1 + 0.1 * torch.randn(d, generator=g)
    S, state = None, None
    for s, e in ((0, T), (T, T + 1)):
        Q, K = split(cuda(rows[:, s:e]), Hq, Hq, d)
        pos = torch.arange(s, e, dtype=torch.int32).expand(B, e - s).contiguous()
        q, k = tri.gdn_qk_norm_fwd(Q, K, cuda(wq), cuda(wk), cuda(freqs), cuda(pos), norm="l2")
        v = cuda(V[:, :, s:e])
        if S is None:
            O, S = tri.gdn_lin_chunk_fwd(q, k, v, cuda(decay))
        else:
            O, S = tri.gdn_lin_decode(q, k, v, cuda(decay), S=S, S_out=S)
        Y = tri.gdn_gate_norm_fwd(O, cuda(Z[:, s:e]), cuda(wo))
        torch.cuda.synchronize()
        xq, xk = split(rows[:, s:e], Hq, Hq, d)
        for got, x, w in ((q, xq, wq), (k, xk, wk)):
            want = ref.qk_forward(x, w, freqs, pos, "l2", 1e-6, "halves", None)
            mag = want.abs()
            mag[..., :64] = (mag[..., :32] + mag[..., 32:64]).repeat(1, 1, 1, 2)
            close(got, want, mag, TOL, "q, k")
        x = {"Q": q.cpu(), "K": k.cpu(), "V": V[:, :, s:e], "g": decay}
        want, state2 = lin_reference.lin_forward(x, d ** -0.5, S0=state)
        mag, _ = lin_reference.lin_forward(x, d ** -0.5, S0=None if state is None else state.abs(), magnitude=True)
        close(O, want, mag, 2.0 ** -12, "O")
        want = lin_reference.gate_norm(O.cpu(), Z[:, s:e], wo, 1e-6, "silu")
        close(Y, want, want.abs(), TOL, "Y")
        state = S.cpu().double()
    y = synth.prefill(3, B, Hq, 128, d, d)
    Q, K = split(cuda(rows[:, :128]), Hq, Hq, d)
    q, k = tri.gdn_qk_norm_fwd(Q, K, norm="l2")
    O, _ = tri.gdn_chunk_fwd(q, k, cuda(y["V"]), cuda(y["beta"]), cuda(y["g"]))
    torch.cuda.synchronize()
    assert torch.isfinite(O).all() and float((k.float().square().sum(-1) - 1).abs().max()) < 2.0 ** -6


@gpu
def test_python_refusals():
    Q, K = torch.zeros((2, 5, 4, 64), device="cuda"), torch.zeros((2, 5, 2, 64), device="cuda")
    w, f = torch.ones(64, device="cuda"), torch.ones(32, device="cuda", dtype=torch.float64)
    pos = torch.zeros((2, 5), device="cuda", dtype=torch.int32)
    many = torch.zeros((2, 2, 5), device="cuda", dtype=torch.int32)
    go = tri.gdn_qk_norm_fwd
    for bad in (lambda: go(None), lambda: go(Q, K.bfloat16()), lambda: go(Q, K[:1]), lambda: go(Q.cpu()), lambda: go(Q.half()),
                lambda: go(Q, wk=w), lambda: go(Q, wq=w[:8]), lambda: go(Q, freqs=f.float()), lambda: go(Q, positions=pos),
                lambda: go(Q, freqs=torch.ones(40, device="cuda").double()), lambda: go(Q, freqs=f, positions=pos.long()),
                lambda: go(Q, freqs=f, positions=many), lambda: go(Q, freqs=f, axis=[0] * 32),
                lambda: go(Q, freqs=f, positions=many, axis=[0] * 8), lambda: go(Q, freqs=f, positions=many, axis=[2] * 32),
                lambda: go(Q, freqs=f, positions=many, axis=[-1] * 32), lambda: go(Q, norm="layer"), lambda: go(Q, pairs="all"),
                lambda: go(Q.transpose(1, 2)), lambda: go(Q[0]), lambda: go(Q, K[0]), lambda: go(Q[..., ::2]),
                lambda: go(Q, Q_out=Q), lambda: tri.gdn_qk_norm_bwd(Q, None, Q),
                lambda: tri.gdn_qk_norm_bwd(Q.transpose(1, 2).contiguous(), K, Q)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(tri.GdnError):
        go(torch.zeros((1, 1, 1, 48), device="cuda"))
    with pytest.raises(tri.GdnError):
        go(Q, freqs=f[:2])


@gpu
def test_more_pairs_than_a_row_has_axes_for():
    # as many axes as pairs, twice what the shape has room for
    Q, f = torch.zeros((1, 1, 1, 512), device="cuda"), torch.ones(256, device="cuda", dtype=torch.float64)
    pos = torch.zeros((1, 1, 1), device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError):
        tri.gdn_qk_norm_fwd(Q, freqs=f, positions=pos, axis=[0] * 256)
    with pytest.raises(ValueError):
        tri.gdn_qk_norm_fwd(Q[..., :256].contiguous(), freqs=f[:128], positions=[[[0]]], axis=[0] * 128)


@gpu
@pytest.mark.parametrize("kind", (tuple, bytes, np.array, torch.tensor))
def test_axis_of_any_sequence(kind):
    g = torch.Generator(device="cuda").manual_seed(3)
    Q = torch.randn((1, 7, 2, 64), device="cuda", generator=g)
    f = torch.rand(32, device="cuda", dtype=torch.float64, generator=g)
    pos = torch.randint(0, 99, (3, 1, 7), device="cuda", dtype=torch.int32, generator=g)
    axis = [(5 * i) % 3 for i in range(32)]
    want = tri.gdn_qk_norm_fwd(Q, freqs=f, positions=pos, axis=axis)[0]
    assert torch.equal(tri.gdn_qk_norm_fwd(Q, freqs=f, positions=pos, axis=kind(axis))[0], want)


# ---- refusals of the C entry points, on the CPU ------------------------------------------------

FAKE = 0x10000


def shape(axis=(), **kw):
    d = dict(T=5, q_stride=256, k_stride=128, B=2, H_q=4, H_k=2, d=64, dtype=0, norm=1, eps=1e-6, rot=64, pairs=0, axes=1)
    d.update(kw)
    s = tri.gdn_qk_shape(*(d[f] for f, _ in tri.gdn_qk_shape._fields_ if f != "axis"))
    for i, a in enumerate(axis):
        s.axis[i] = a
    return s


def test_c_refusals():
    lib = tri._lib
    by = ctypes.byref

    def fwd(Q=FAKE, K=FAKE, wq=None, freqs=FAKE, pos=None, out=FAKE, **kw):
        return lib.gdn_qk_norm_fwd(by(shape(**kw)), Q, K, wq, None, freqs, pos, out, FAKE, None)

    def bwd(Q=FAKE, K=FAKE, wq=None, freqs=FAKE, pos=None, out=FAKE, dw=FAKE, ws=FAKE, nb=1 << 30, **kw):
        return lib.gdn_qk_norm_bwd(by(shape(**kw)), FAKE, FAKE, Q, K, wq, None, freqs, pos, out, FAKE, dw, None, ws, nb, None)

    for f in (fwd, bwd):
        assert f(B=-1) == 2 and f(T=-1) == 2 and f(H_q=-1) == 2 and f(d=0) == 2 and f(eps=-1.0) == 2
        assert f(eps=float("nan")) == 2 and f(dtype=2) == 3 and f(norm=3) == 2 and f(pairs=2) == 2 and f(d=48, rot=0) == 5
        assert f(d=288, rot=0, q_stride=4096, k_stride=4096) == 5 and f(rot=72) == 2 and f(rot=12) == 2 and f(rot=-8) == 2
        assert f(axes=0) == 2 and f(axes=5) == 2 and f(axis=[0] * 31 + [1]) == 2 and f(q_stride=248) == 2
        assert f(q_stride=260) == 4 and f(k_stride=0) == 2 and f(T=1 << 40) == 5
        assert f(Q=None) == 1 and f(K=None) == 1 and f(freqs=None) == 1 and f(out=None) == 1
        assert f(Q=FAKE + 8) == 4 and f(wq=FAKE + 4) == 4 and f(pos=FAKE + 4) == 4
    assert lib.gdn_qk_norm_fwd(None, *[None] * 9) == 1
    assert fwd(T=0) == 0 and fwd(H_q=0, H_k=0) == 0 and bwd(B=0, dw=None) == 0
    assert bwd(ws=None) == 6 and bwd(nb=8) == 6 and bwd(ws=FAKE + 8) == 4
    assert lib.gdn_qk_norm_bwd_workspace_bytes(by(shape(d=48))) == 0
    assert lib.gdn_qk_norm_bwd_workspace_bytes(by(shape())) > 0
