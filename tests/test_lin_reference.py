"""The fp64 references of the linear-attention and norm tests: gradients against central
differences of the forward recurrence, the chunk-free definitions against autograd."""
import pytest
import torch

import lin_reference as ref


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("lens", [None, [3, 0, 1, 5]])
def test_gradients_are_the_differences(decay, lens):
    B, H, Hk, T, dk, dv = (2, 4, 2, 9, 3, 2) if lens is None else (1, 4, 2, 9, 3, 2)
    x = ref.lin_inputs(3, B, H, Hk, T, dk, dv, decay, n_state=None if lens is None else 4)
    x = {k: t.double() for k, t in x.items()}
    scale, S0, dS = 0.4, x["S0"], x["dS"]

    def loss(y, S):
        o, last = ref.lin_forward(y, scale, S, lens)
        return float((o * y["dO"]).sum() + (last * dS).sum())

    got = ref.lin_backward(x, scale, S0, dS, lens)
    gen = torch.Generator().manual_seed(5)
    for name, grad in zip(("Q", "K", "V", "g", "S0"), got):
        way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        plus, minus = ({**x, name: x[name] + s * e * way} for s in (1, -1))
        num = (loss(plus, plus["S0"]) - loss(minus, minus["S0"])) / (2 * e)
        ana = float((grad * way).sum())
        assert abs(num - ana) <= 1e-7 * max(1.0, abs(ana)), (name, num, ana)


def test_recurrence_equals_the_weighted_sum():
    """o_t = scale sum_{s<=t} e^{g_{s+1} + .. + g_t} (q_t . k_s) v_s + the decayed given state."""
    x = ref.lin_inputs(4, 1, 1, 1, 6, 4, 3)
    O, _ = ref.lin_forward(x, 0.5, x["S0"])
    q, k, v, g = (x[n].double()[0, 0] for n in ("Q", "K", "V", "g"))
    for t in range(6):
        want = sum(torch.exp(g[s + 1:t + 1].sum()) * (q[t] @ k[s]) * v[s] for s in range(t + 1))
        want = want + torch.exp(g[:t + 1].sum()) * (q[t] @ x["S0"].double()[0, 0])
        assert torch.allclose(O[0, 0, t], 0.5 * want, rtol=1e-12, atol=1e-12)
