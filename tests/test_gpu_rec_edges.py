"""GPU tests of the gated linear recurrence at the edges of its range, against fp64 (rec_reference.py), and refusals
of its C entry points."""
import ctypes

import pytest
import torch

import rec_reference as ref
from helpers import cuda, say
from test_gpu_rec import FAKE, check, close, offsets_of, shape, up

tri = pytest.importorskip("tri_inverse_amd")
gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@gpu
@pytest.mark.parametrize("decay", ["power", "sigmoid", "log"])
def test_gradients_of_nan_gates(decay):
    """A NaN in a gate makes the gradients that its own formula takes from it NaN, and leaves other channels."""
    say(f"recurrence, NaN gates, {decay}")
    x = {k: up(v) for k, v in ref.rec_inputs(4, 1, 70, 40, decay, True, F32).items()}

    def both(A, I):
        how = dict(I=I, w=x["w"], h0=x["h0"], decay=decay)
        _, _, st = tri.gdn_rec_fwd(x["X"], A, want_states=True, **how)
        return tri.gdn_rec_bwd(x["X"], A, x["dH"], dh=x["dh"], states=st, **how)

    A, I = x["A"].clone(), x["I"].clone()
    I[0, 30, ::4], A[0, 50, 1::4] = float("nan"), float("nan")
    dirty, clean = both(A, I), both(x["A"], x["I"])
    torch.cuda.synchronize()
    for name, g, y in zip(("dX", "dA", "dI"), dirty, clean):
        assert torch.isnan(g[0, 30, ::4]).all(), name + " of a NaN in I"
        assert torch.isnan(g[0, 50, 1::4]).all(), name + " of a NaN in A"
        for c in (2, 3):
            assert torch.equal(g[..., c::4], y[..., c::4]), name


@gpu
@pytest.mark.parametrize("decay,norm,far", [("log", "none", 80), ("power", "linear", 80), ("sigmoid", "linear", 80),
                                            ("power", "sqrt", 50), ("sigmoid", "sqrt", 50)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_gates_keep_their_digits(decay, norm, far, dtype):
    """Sequences of one token, whose state is its input's part alone: small sigmoids, and what large ones leave of 1,
    are right to the reference's bound, which does not grow with an fp32 gate.  X is scaled so that the outputs are large
    beside the tolerance's constant; with sqrt(1 - a^2) the gates end where the bound's floor would count.

    Of a bf16 gate z, rounded itself by 2^-9 |z| in e^-z, the product with log2 e is rounded to fp32: 2^-24 |z log2 e|, ln 2
    of it in e^-z, and log2 e as it is held is off by 2^-26.3 |z| more in it: together below 2^-23 |z| = EPS |z| / 8."""
    say(f"recurrence, gates up to {far}, {decay} {norm} {dtype}")
    B, D = 70, 136
    x = ref.rec_inputs(far, B, 1, D, decay, True, dtype)
    gate = (15 + (far - 15) * torch.rand((B, 1, D), generator=torch.Generator().manual_seed(7))).to(dtype)
    if decay == "log":
        x["A"][:], x["I"] = -float("inf"), -gate
    else:
        x["A"], x["I"] = gate if decay == "sigmoid" else -gate, None
    x["X"] = x["X"] * 2.0 ** 66
    if dtype == F32:
        check(x, decay, norm, h0=False, dh=False)
    how = dict(I=up(x["I"]), w=up(x["w"]), decay=decay, norm=norm)
    H, h, _ = tri.gdn_rec_fwd(up(x["X"]), up(x["A"]), **how)
    H1, h1 = tri.gdn_rec_step(up(x["X"]), up(x["A"]), **how)
    torch.cuda.synchronize()
    Hr, hr, EH, Eh, _ = ref.rec_forward(x, decay, norm)
    grow = 1 + gate.double() / 8 * (dtype == BF)
    for y, z in ((H, h), (H1, h1)):
        close(y, Hr, EH * grow, "H")
        close(z, hr, Eh * grow[:, 0], "h_out")


@gpu
def test_many_short_and_empty_sequences():
    """Sequences of none, one or two tokens: more of them than tokens."""
    say("recurrence, 3000 short sequences")
    lens = torch.randint(0, 3, (3000,), generator=torch.Generator().manual_seed(2))
    lens[1000:2000] = 0
    T = int(lens.sum()) + 30
    check(ref.rec_inputs(1, 1, T, 24, "power", True, F32, n_state=3000), "power", "sqrt", lens=lens.tolist(), first=10)


@gpu
def test_time_of_empty_sequences():
    """200000 sequences with 64 tokens among them: the states of the empty ones are copied by all waves of the call,
    not by one wave one after the other (which took 0.54 us each; 0.25 allowed)."""
    n, T, D = 200000, 64, 136
    say("recurrence, 200000 sequences of 64 tokens")
    some = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:T].sort().values
    lens = torch.zeros(n, dtype=torch.int64)
    lens[some] = 1
    off = cuda(torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32))
    x = {k: up(v) for k, v in ref.rec_inputs(3, 1, T, D, "power", True, F32).items()}
    h0, dh = torch.randn((n, D), device="cuda"), torch.randn((n, D), device="cuda")

    def both(h0, dh, off):
        how = dict(I=x["I"], w=x["w"], h0=h0, offsets=off)
        H, h, st = tri.gdn_rec_fwd(x["X"], x["A"], want_states=True, **how)
        return (H, h) + tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], dh=dh, states=st, **how)

    some = cuda(some)
    want = both(h0[some], dh[some], offsets_of([1] * T, 0))
    got = both(h0, dh, off)
    torch.cuda.synchronize()
    empty = torch.ones(n, dtype=torch.bool, device="cuda")
    empty[some] = False
    assert torch.equal(got[1][empty], h0[empty]) and torch.equal(got[6][empty], dh[empty])
    assert torch.equal(got[1][some], want[1]) and torch.equal(got[6][some], want[6])
    for i in (0, 2, 3, 4, 5):
        assert torch.equal(got[i], want[i]), i
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    both(h0, dh, off)
    end.record()
    torch.cuda.synchronize()
    print("forward and backward: %.1f ms" % start.elapsed_time(end), flush=True)
    assert start.elapsed_time(end) < 2 * n * 0.25e-3


def test_states_are_not_written_over():
    """A state that some workgroups read while others write its place is refused; the step may update in place."""
    lib, at = tri._lib, ctypes.byref(shape())
    S, R = FAKE + 4096, FAKE + 8192

    def fwd(h0, h_out):
        return lib.gdn_rec_fwd(at, FAKE, FAKE, None, FAKE, h0, FAKE, h_out, None, None, 0, None)

    def bwd(dh, dh0):
        return lib.gdn_rec_bwd(at, FAKE, FAKE, None, FAKE, None, None, FAKE, dh, FAKE, FAKE, None, None, dh0, None, 0, None)

    for f in (fwd, bwd):  # the workspace is looked at last
        assert f(S, S) == 5 and f(S, R) == 6 and f(None, None) == 6


@gpu
def test_states_of_no_sequence():
    """Packed rows that belong to no sequence: the states before every 64th token are zeros."""
    say("recurrence, no sequence")
    T, D = 130, 16
    x = torch.ones((1, T, D), device="cuda")
    off, states = torch.zeros(4, device="cuda", dtype=torch.int32), torch.full((1, 3, D), 7.0, device="cuda")
    H = torch.full_like(x, 7.0)
    sh = shape(T=T, D=D, B=0, decay=1, x_stride=D, a_stride=D, i_stride=D, offsets=off.data_ptr())
    p = lambda t: t.data_ptr()  # noqa: E731
    st = tri._lib.gdn_rec_fwd(ctypes.byref(sh), p(x), p(x), None, None, None, p(H), None, p(states), None, 0,
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and (states == 0).all() and (H == 7).all()
