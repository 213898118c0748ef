"""Linear attention where a call is divided into segments whose states are formed apart and joined,
at the sizes of training and of wide values: d_k = 128 backwards (the states are read transposed by
the scans of dQ and dK, dg runs between them), d_v of 96 and 256 forwards.  Tolerances and their
derivation are those of test_gpu_lin.py: 2^-14 M for outputs, whose bf16 type adds half a step of
the value, 2^-17 M for states, 2e-4 in the norm for dg."""
import pytest
import torch

import lin_reference as ref
from helpers import cuda, relF, say
from test_gpu_lin import TOL_DG, TOL_O, TOL_S, check_backward, close, offsets_of, run_forward

tri = pytest.importorskip("tri_inverse_amd")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("H,Hk,T,dk,dv,decay", [(2, 1, 1200, 128, 128, "token"), (2, 2, 1200, 128, 64, "head"),
                                                (3, 3, 2050, 128, 128, "head")])
def test_backward(H, Hk, T, dk, dv, decay):
    say(f"lin backward divided H={H} Hk={Hk} T={T} dk={dk} dv={dv} {decay}")
    x = ref.lin_inputs(T, 1, H, Hk, T, dk, dv, decay)
    check_backward(x, 0.25, x["S0"], x["dS"])
    check_backward(x, 0.25, x["S0"], x["dS"], grad_dtype=BF)
    check_backward(x, 0.25, None, None)


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dv", [64, 128])
def test_backward_packed(decay, dv):
    lens, first, behind = [1100, 0, 2, 300, 64], 3, 5
    T = first + sum(lens) + behind
    say(f"lin backward packed divided dv={dv} {decay}")
    x = ref.lin_inputs(17, 1, 4, 2, T, 128, dv, decay, n_state=len(lens))
    for t in (F32, BF):
        got = check_backward(x, 0.25, x["S0"], x["dS"], lens, first, grad_dtype=t)
        for y in got[:3]:
            assert torch.count_nonzero(y[:, :, :first]) == 0 and torch.count_nonzero(y[:, :, T - behind:]) == 0


@pytest.mark.parametrize("lens", [None, [500, 0, 700]])
def test_backward_without_dg(lens):
    """Without dg the other gradients keep their bits, though fewer states are formed for them."""
    say(f"lin backward without dg {lens}")
    x = ref.lin_inputs(19, 1, 2, 1, 1200, 128, 64, n_state=None if lens is None else len(lens))
    off = None if lens is None else cuda(offsets_of(lens))
    call = lambda want: tri.gdn_lin_chunk_bwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g", "dO")),  # noqa: E731
                                              S0=cuda(x["S0"]), dS=cuda(x["dS"]), offsets=off, want_dg=want)
    a, b = call(True), call(False)
    torch.cuda.synchronize()
    assert b[3] is None and all(torch.equal(p, q) for i, (p, q) in enumerate(zip(a, b)) if i != 3)
    want = ref.lin_backward(x, 128 ** -0.5, x["S0"], x["dS"], lens)
    assert relF(a[3].cpu(), want[3]) <= TOL_DG


@pytest.mark.parametrize("dk,dv,decay", [(64, 96, "token"), (128, 256, "head"), (128, 96, "head"), (64, 256, "token")])
def test_forward(dk, dv, decay):
    T = 4200
    say(f"lin forward divided dk={dk} dv={dv} {decay}")
    assert tri.gdn_lin_chunk_fwd_workspace_bytes(1, 2, T, dk, dv, H_qk=1) > 0
    x = ref.lin_inputs(T, 1, 2, 1, T, dk, dv, decay)
    want, mag = (ref.lin_forward(x, 0.125, x["S0"], magnitude=m) for m in (False, True))
    for t in (F32, BF):
        O, S = run_forward(x, 0.125, x["S0"], o_dtype=t)
        torch.cuda.synchronize()
        assert O.dtype == t
        close(O, want[0], mag[0], TOL_O, "O")
        close(S, want[1], mag[1], TOL_S, "S")


def test_forward_packed_wide():
    """Packed, d_v = 256: sequences of some segments between short and empty ones."""
    lens = [1500, 0, 1, 2600, 65]
    say("lin forward packed divided dv=256")
    assert tri.gdn_lin_chunk_fwd_workspace_bytes(len(lens), 4, sum(lens), 128, 256, H_qk=2, packed=True) > 0
    x = ref.lin_inputs(23, 1, 4, 2, sum(lens), 128, 256, n_state=len(lens))
    want, mag = (ref.lin_forward(x, 0.2, x["S0"], lens, magnitude=m) for m in (False, True))
    O, S = run_forward(x, 0.2, x["S0"], lens)
    torch.cuda.synchronize()
    close(O, want[0], mag[0], TOL_O, "O")
    close(S, want[1], mag[1], TOL_S, "S")
