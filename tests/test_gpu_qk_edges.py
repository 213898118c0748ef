"""GPU tests of the norm and rotation of queries and keys at the edges of their range."""
import decimal
import math

import pytest
import torch

from helpers import cuda, say
from test_gpu_qk import frequencies

tri = pytest.importorskip("tri_inverse_amd")
gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def whole_turns(digits=60):
    """2 pi by Machin's formula."""
    with decimal.localcontext() as c:
        c.prec = digits + 5

        def arctan_of_inverse(n):
            term = total = decimal.Decimal(1) / n
            k = 1
            while abs(term) > decimal.Decimal(10) ** -(digits + 3):
                term, k = -term / (n * n), k + 2
                total += term / k
            return total

        return 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))


def test_whole_turns():
    assert float(whole_turns()) == 2 * math.pi and str(whole_turns()).startswith("6.28318530717958647692528676655900576839433879875")


@gpu
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_angles_at_far_positions(pairs):
    """The cosine and sine themselves, against angles of 60 digits.  The kernel's angle is rounded to fp32 below an eighth
    of a turn (2^-25) and its series end in one or two roundings of a value below 1 (2^-25 each) and smaller ones: 1.8 x 2^-24
    together, 2^-23 allowed, at any position."""
    say(f"queries and keys, angles at far positions, {pairs}")
    r, T = 64, 96
    g = torch.Generator().manual_seed(8)
    pos = torch.randint(2 ** 30, 2 ** 31, (1, T), generator=g, dtype=torch.int64)
    pos[0, 32:64] = torch.randint(2 ** 28, 2 ** 29, (32,), generator=g)
    pos[0, 1::2] *= -1
    pos[0, :6] = torch.tensor([2 ** 31 - 1, -2 ** 31, 1_000_000, 0, 1, -7])
    freqs = frequencies(r)
    freqs[1], freqs[2] = 0.9999, 1e9  # beside 1, whose products with positions are exact; whole turns past 2^53
    one = torch.zeros((1, T, 1, r))
    first = slice(0, r // 2) if pairs == "halves" else slice(0, r, 2)
    second = slice(r // 2, r) if pairs == "halves" else slice(1, r, 2)
    one[..., first] = 1.0
    how = dict(freqs=cuda(freqs), positions=cuda(pos.to(torch.int32)), norm="none", pairs=pairs)
    Q = cuda(one)
    y = tri.gdn_qk_norm_fwd(Q, **how)[0][0, 0].cpu().double()
    dx = tri.gdn_qk_norm_bwd(Q.transpose(1, 2).contiguous(), None, Q, **how)[0][0, :, 0].cpu().double()
    torch.cuda.synchronize()
    turn = whole_turns()
    want = torch.empty((T, r // 2), dtype=torch.float64)
    with decimal.localcontext() as c:
        c.prec = 60
        for t in range(T):
            for i in range(r // 2):
                angle = decimal.Decimal(int(pos[0, t])) * decimal.Decimal(float(freqs[i]))
                want[t, i] = float(angle - turn * (angle / turn).to_integral_value())
    for name, got, exact in (("cos", y[:, first], want.cos()), ("sin", y[:, second], want.sin()),
                             ("cos backwards", dx[:, first], want.cos()), ("sin backwards", dx[:, second], -want.sin())):
        worst = float((got - exact).abs().max()) * 2 ** 24
        print("%s: %.2f x 2^-24" % (name, worst), flush=True)
        assert worst <= 2.0, name


@gpu
def test_weight_gradients_over_many_equal_rows():
    """2^26 equal rows: every addition to a sum of 32 bits rounds the same way, so a lane's own run of them has to be short.
    n = (1 + eps)^-1/2, 0.45 x 2^-14 below 1, is lost from each addition to a sum between 512 and 1024."""
    T, H, d, eps = 65536, 1024, 32, 0.9 * 2.0 ** -14
    say("queries and keys, 2^26 equal rows")
    Q = torch.ones((1, T, H, d), device="cuda", dtype=BF)
    g = tri.gdn_qk_norm_bwd(Q.view(1, H, T, d), None, Q, None, torch.ones(d, device="cuda"), norm="rms", eps=eps)
    torch.cuda.synchronize()
    want = T * H / math.sqrt(1.0 + float(torch.tensor(eps, dtype=F32)))
    worst = float((g[2].cpu().double() / want - 1).abs().max())
    print("off by %.2f x 2^-17" % (worst * 2 ** 17), flush=True)
    assert worst <= 2.0 ** -17


@gpu
def test_more_heads_than_a_piece_of_work_takes():
    """130 query heads of 32768 tokens: three runs of heads, each gradient as without the other heads."""
    say("queries and keys, 130 heads")
    T, H, d = 32768, 130, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    Q, dQ = (torch.randn(s, device="cuda", generator=g).to(BF) for s in ((1, T, H, d), (1, H, T, d)))
    w = torch.ones(d, device="cuda")
    how = dict(freqs=cuda(frequencies(16)), eps=1e-5)
    dx, _, dw, _ = tri.gdn_qk_norm_bwd(dQ, None, Q, None, w, **how)
    for s, e in ((0, 64), (60, 70), (128, 130)):
        part = tri.gdn_qk_norm_bwd(dQ[:, s:e].contiguous(), None, Q[:, :, s:e], None, w, **how)
        assert torch.equal(dx[:, :, s:e], part[0]), (s, e)
    # the weights' gradients, of the values that are not turned
    n = Q.double()
    n = (n * (n.square().mean(-1, True) + 1e-5).rsqrt()).transpose(1, 2)[..., 16:]
    n *= dQ[..., 16:].double()
    torch.cuda.synchronize()
    assert ((dw[16:].double() - n.sum((0, 1, 2))).abs() <= 2.0 ** -17 * n.abs().sum((0, 1, 2))).all()
