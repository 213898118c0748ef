"""The fp64 references of the recurrence and of the queries' and keys' norm and rotation against torch's
gradients and against differences (CPU)."""
import math

import pytest
import torch

import rec_reference as ref


@pytest.mark.parametrize("decay", ["power", "sigmoid", "log"])
@pytest.mark.parametrize("norm", ["sqrt", "linear", "none"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("lens", [None, [3, 0, 1, 2]])
def test_recurrence_gradients(decay, norm, gate, lens):
    B, T, D = (2, 5, 3) if lens is None else (1, 8, 3)  # packed: one row before and one behind them
    x = ref.rec_inputs(1, B, T, D, decay, gate, torch.float64, n_state=None if lens is None else len(lens))
    names = [k for k in ("X", "A", "I", "w", "h0") if x[k] is not None]
    leaves = [x[k].double().requires_grad_() for k in names]

    def forward(*args):
        y = dict(x, **dict(zip(names, args)))
        g, a, b, _, i, _, _ = ref.gates(y, decay, norm)
        u, rows, last = b * i * y["X"], [], []
        for k, (row, s, e) in enumerate(ref.spans_of(B, T, lens, 1)):
            h = y["h0"][k]
            for t in range(s, e):
                h = a[row, t] * h + u[row, t]
                rows.append(h)
            last.append(h)
        return torch.stack(rows), torch.stack(last)

    assert torch.autograd.gradcheck(forward, leaves)
    H, h = forward(*leaves)
    Hr, hr, *_ = ref.rec_forward(x, decay, norm, x["h0"], lens, 1)
    rows = torch.cat([Hr[row, s:e] for row, s, e in ref.spans_of(B, T, lens, 1)])
    assert torch.allclose(H, rows) and torch.allclose(h, hr)
    dH = torch.cat([x["dH"][row, s:e] for row, s, e in ref.spans_of(B, T, lens, 1)])
    want = dict(zip(names, torch.autograd.grad((H * dH).sum() + (h * x["dh"].double()).sum(), leaves)))
    got, bounds = ref.rec_backward(x, decay, norm, x["h0"], x["dh"], lens, 1)
    for key, y, e in zip(("X", "A", "I", "w", "h0"), got, bounds):
        assert (y is None) == (key not in want)
        if y is not None:
            assert torch.allclose(y, want[key], rtol=1e-9, atol=1e-12), key
            assert (e >= 0).all() and float((e / (y.abs() + 1)).max()) < 1e-3


def test_slow_decays_bound():
    """Decays near 1: the bound stays far below what a rounding to bf16 takes."""
    x = ref.rec_inputs(2, 1, 400, 4, "power", True, slow=True)
    H, _, E, _, _ = ref.rec_forward(x, "power", "sqrt", x["h0"])
    assert float((E / H.abs().clamp(min=0.1)).max()) < 2.0 ** -9


@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("axis", [None, (0, 1, 1)])
def test_qk_gradients(norm, pairs, axis):
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn((2, 3, 2, 8), generator=g).double().requires_grad_(), torch.randn(8, generator=g).double().requires_grad_()
    freqs = torch.tensor([1.0, 0.3, 0.05], dtype=torch.float64)
    pos = torch.randint(0, 50, (2, 3) if axis is None else (2, 2, 3), generator=g)
    f = lambda x, w: ref.qk_forward(x, w, freqs, pos, norm, 1e-6, pairs, axis)  # noqa: E731
    assert torch.autograd.gradcheck(f, (x, w))
    dy = torch.randn((2, 2, 3, 8), generator=g).double()
    want = torch.autograd.grad((f(x, w) * dy).sum(), (x, w))
    got = ref.qk_backward(dy, x.detach(), w.detach(), freqs, pos, norm, 1e-6, pairs, axis)
    assert torch.allclose(got[0], want[0]) and torch.allclose(got[2], want[1])
    assert (got[1] >= got[0].abs() * (1 - 1e-12)).all() and (got[3] >= got[2].abs() * (1 - 1e-12)).all()


def test_rotation_keeps_distances():
    """The product of a turned query and a turned key depends on their distance alone."""
    g = torch.Generator().manual_seed(5)
    q, k = (torch.randn((1, 1, 1, 16), generator=g).double() for _ in range(2))
    freqs = torch.exp(-torch.arange(8).double() / 8 * math.log(10000.0))
    for pairs in ("halves", "neighbours"):
        at = lambda x, p: ref.qk_rotate(x, freqs, torch.tensor([[p]]), pairs, None)  # noqa: E731
        near, far = (at(q, 7) * at(k, 3)).sum(), (at(q, 1007) * at(k, 1003)).sum()
        assert abs(float(near - far)) < 1e-9
