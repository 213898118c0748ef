"""Outputs of linear attention in bf16 are those in fp32 rounded once: the type of an output
changes no product before it.  Compared bit by bit, so without a tolerance; against the fp64
recurrence an element is right to half a step of its value, 2^-8, beside the 2^-14 M of an
output in fp32 (three bf16 parts of every fp32 factor, exponentials to 2^-22, fp32 sums of a
chunk to about 2^-17, two such products; M is the same sum over absolute values)."""
import pytest
import torch

import lin_reference as ref
from helpers import cuda, say

tri = pytest.importorskip("tri_inverse_amd")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = 2.0 ** -14


def offsets_of(lens):
    return None if lens is None else cuda(torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32))


def close(got, want, mag, what):
    got = got.cpu()
    assert got.dtype == BF and torch.isfinite(got).all(), what
    room = TOL * mag + 2.0 ** -8 * (want.abs() + TOL * mag) + 1e-30
    worst = float(((got.double() - want).abs() / room).max())
    assert worst <= 1.0, "%s: %.3g of its tolerance" % (what, worst)


def slow(x):
    """Decays over thousands of tokens: the state carries the outputs."""
    x["g"] = -torch.exp2(-8.0 - 4.0 * torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(1)))
    return x


CASES = [  # H, Hk, T, dk, dv, decay, lengths of packed sequences, states given
    (2, 2, 1, 64, 64, "token", None, True), (4, 2, 77, 64, 64, "token", None, True),
    (3, 3, 200, 128, 128, "head", None, False), (2, 1, 150, 128, 256, "head", None, True),
    (2, 2, 150, 64, 96, "token", None, True), (2, 1, 1200, 128, 128, "token", None, True),
    (4, 2, 700, 64, 64, "head", [70, 0, 1, 500, 129], True), (2, 2, 400, 128, 64, "token", [300, 0, 100], False)]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_forward(case):
    H, Hk, T, dk, dv, decay, lens, state = case
    say(f"lin forward bf16 against fp32 {case}")
    x = slow(ref.lin_inputs(T, 1, H, Hk, T, dk, dv, decay, n_state=None if lens is None else len(lens)))
    S0 = x["S0"] if state else None
    call = lambda t: tri.gdn_lin_chunk_fwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g")), scale=0.2,  # noqa: E731
                                           S0=None if S0 is None else cuda(S0), offsets=offsets_of(lens), o_dtype=t)
    (O, S), (O32, S32) = call(BF), call(F32)
    torch.cuda.synchronize()
    assert torch.equal(O, O32.to(BF)) and torch.equal(S, S32)
    want, mag = ref.lin_forward(x, 0.2, S0, lens), ref.lin_forward(x, 0.2, S0, lens, magnitude=True)
    close(O, want[0], mag[0], "O")


@pytest.mark.parametrize("case", [c for c in CASES if c[4] in (64, 128)], ids=str)
def test_backward(case):
    H, Hk, T, dk, dv, decay, lens, state = case
    say(f"lin backward bf16 against fp32 {case}")
    x = slow(ref.lin_inputs(T, 1, H, Hk, T, dk, dv, decay, n_state=None if lens is None else len(lens)))
    S0, dS = (x["S0"], x["dS"]) if state else (None, None)
    up = lambda t: None if t is None else cuda(t)  # noqa: E731
    call = lambda t: tri.gdn_lin_chunk_bwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g", "dO")), scale=0.2,  # noqa: E731
                                           S0=up(S0), dS=up(dS), offsets=offsets_of(lens), grad_dtype=t)
    got, got32 = call(BF), call(F32)
    torch.cuda.synchronize()
    want, mag = (ref.lin_backward(x, 0.2, S0, dS, lens, magnitude=m) for m in (False, True))
    for i, name in enumerate(("dQ", "dK", "dV")):
        assert torch.equal(got[i], got32[i].to(BF)), name
        close(got[i], want[i], mag[i], name)
    assert torch.equal(got[3], got32[3])
    assert got[4] is None if S0 is None else torch.equal(got[4], got32[4])
