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
