"""GPU parity of linear attention with a decay for each head (chunk-wise forward, backward,
single tokens) against the fp64 token recurrence on the same inputs.

Tolerances are elementwise, relative to M, the same sums over absolute values:
  * products with an fp32 factor split into two or more bf16 parts (three are used) lose at most
    2^-16 of a term (two roundings of half a step, 2^-8 each); an output is a sum of two such
    products, the exponentials add 2^-22 and the fp32 sums of a chunk at most about 2^-17: 2^-14 M;
  * O and dV stored in bf16 are these sums rounded once (test_gpu_lin_rounding.py compares them
    so).  Here they have 2^-8 M more, half a step of each term, and in the norm 2^-8, where that
    rounding is at most 2^-8 / sqrt(3) in the root mean square;
  * states: three parts (2^-24), exponentials, fp32 sums of 64 terms a chunk carried over at
    most 40 chunks: 2^-17 M;
  * outputs stored in bf16 add half a step, 2^-8 of the value;
  * dg: per token a difference of two dot products of outputs as above (rms error about 2^-17
    of their size), at most 1024 of them summed from one pair of states, so about 2^-12 of one
    term and less than 1e-4 of the whole, whose rms is several terms': 2e-4 in the norm."""
import ctypes

import pytest
import torch

import lin_reference as ref
from helpers import cuda, relF, say

tri = pytest.importorskip("tri_inverse_amd")

gpu = pytest.mark.gpu
TOL_O, TOL_S, TOL_DG = 2.0 ** -14, 2.0 ** -17, 2e-4
TOL_ONE = 2.0 ** -8 + TOL_O  # bf16 outputs formed with one part


def close(got, want, mag, tol, what):
    got = got.detach().cpu()
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    err = (got.double() - want).abs()
    room = tol * mag + half * (want.abs() + tol * mag) + 1e-30
    assert torch.isfinite(got).all(), what
    worst = float((err / room).max()) if err.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g of its tolerance" % (what, worst)


def offsets_of(lens, first=0):
    return (torch.tensor([0] + list(lens)).cumsum(0) + first).to(torch.int32)


def run_forward(x, scale, S0, lens=None, first=0, **kw):
    off = None if lens is None else cuda(offsets_of(lens, first))
    return tri.gdn_lin_chunk_fwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g")), scale=scale,
                                 S0=None if S0 is None else cuda(S0), offsets=off, **kw)


@gpu
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 200, 321])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_forward_lengths(T, dk, dv):
    say(f"lin forward T={T} dk={dk} dv={dv}")
    x = ref.lin_inputs(T, 2, 3, 3, T, dk, dv)
    for S0, odt in ((x["S0"], torch.float32), (None, torch.bfloat16)):
        O, S = run_forward(x, dk ** -0.5, S0, o_dtype=odt)
        torch.cuda.synchronize()
        want, mag = ref.lin_forward(x, dk ** -0.5, S0), ref.lin_forward(x, dk ** -0.5, S0, magnitude=True)
        assert O.dtype == odt
        close(O, want[0], mag[0], TOL_O if odt == torch.float32 else TOL_ONE, "O")
        assert relF(O.cpu().double(), want[0]) <= 2.0 ** -8
        close(S, want[1], mag[1], TOL_S, "S")


@gpu
@pytest.mark.parametrize("H,Hk,dk,dv,decay,strong", [
    (4, 1, 128, 256, "token", False), (6, 2, 64, 96, "head", False), (1, 1, 64, 32, "token", True),
    (3, 3, 128, 160, "token", True), (8, 4, 128, 128, "head", False), (5, 5, 64, 224, "token", False)])
def test_forward_heads_widths_decays(H, Hk, dk, dv, decay, strong):
    T = 150
    say(f"lin forward H={H} Hk={Hk} dk={dk} dv={dv} {decay} strong={strong}")
    x = ref.lin_inputs(7, 2, H, Hk, T, dk, dv, decay, strong=strong)
    O, S = run_forward(x, 0.3, x["S0"], o_dtype=torch.float32)
    torch.cuda.synchronize()
    want, mag = ref.lin_forward(x, 0.3, x["S0"]), ref.lin_forward(x, 0.3, x["S0"], magnitude=True)
    close(O, want[0], mag[0], TOL_O, "O")
    close(S, want[1], mag[1], TOL_S, "S")


@gpu
@pytest.mark.parametrize("T,decay", [(4100, "token"), (6500, "head"), (4159, "head")])
def test_forward_divided_tokens(T, decay):
    """Few heads and many tokens: segments are formed apart and joined."""
    say(f"lin forward divided T={T} {decay}")
    assert tri.gdn_lin_chunk_fwd_workspace_bytes(1, 2, T, 64, 64) > 0
    x = ref.lin_inputs(T, 1, 2, 1, T, 64, 64, decay)
    O, S = run_forward(x, 0.125, x["S0"], o_dtype=torch.float32)
    torch.cuda.synchronize()
    want, mag = ref.lin_forward(x, 0.125, x["S0"]), ref.lin_forward(x, 0.125, x["S0"], magnitude=True)
    close(O, want[0], mag[0], TOL_O, "O")
    close(S, want[1], mag[1], TOL_S, "S")


PACKS = [[1], [64, 64], [0, 70, 0, 1, 129, 63, 0], [5] * 70 + [0] * 3 + [200], [1300, 3, 600], [0, 0, 0],
         [4400, 3, 0, 700]]


@gpu
@pytest.mark.parametrize("lens", PACKS, ids=[str(i) for i in range(len(PACKS))])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_forward_packed(lens, decay):
    """Packed sequences behind some rows that belong to none and in front of others: those rows
    hold NaN and are neither read into a result nor written."""
    H, Hk, dk, dv, first, behind = 4, 2, 64, 64, 3, 5
    T = first + sum(lens) + behind
    say(f"lin forward packed {len(lens)} sequences, {T} tokens, {decay}")
    if max(lens) > 4000:  # divided: segments are formed apart and joined
        assert tri.gdn_lin_chunk_fwd_workspace_bytes(len(lens), H, T, dk, dv, H_qk=Hk, packed=True) > 0
    x = ref.lin_inputs(11, 1, H, Hk, T, dk, dv, decay, n_state=len(lens))
    bad = dict(x)
    inside = slice(first, T - behind)
    for n in ("Q", "K", "V") + (("g",) if decay == "token" else ()):
        bad[n] = torch.full_like(x[n], float("nan"))
        bad[n][:, :, inside] = x[n][:, :, inside]
    O = torch.full((1, H, T, dv), 7.0, device="cuda")
    O, S = run_forward(bad, 0.2, x["S0"], lens, first, O=O)
    torch.cuda.synchronize()
    want = ref.lin_forward(x, 0.2, x["S0"], lens, first)
    mag = ref.lin_forward(x, 0.2, x["S0"], lens, first, magnitude=True)
    close(O[:, :, inside], want[0][:, :, inside], mag[0][:, :, inside], TOL_O, "O")
    close(S, want[1], mag[1], TOL_S, "S")
    assert (O[:, :, :first] == 7).all() and (O[:, :, T - behind:] == 7).all()


@gpu
def test_forward_no_tokens():
    say("lin forward T=0")
    x = ref.lin_inputs(1, 2, 3, 3, 0, 64, 64)
    O, S = run_forward(x, 1.0, x["S0"])
    _, Z = run_forward(x, 1.0, None)
    torch.cuda.synchronize()
    assert O.numel() == 0 and torch.equal(S.cpu(), x["S0"]) and torch.count_nonzero(Z) == 0


BWD = [  # B, H, Hk, T, dk, dv, decay, strong
    (2, 2, 2, 1, 64, 64, "token", False), (1, 3, 3, 63, 128, 64, "token", False), (2, 2, 2, 65, 64, 128, "head", False),
    (1, 4, 2, 130, 128, 128, "token", False), (1, 6, 2, 200, 64, 64, "head", False),
    (1, 2, 2, 300, 64, 64, "token", True), (1, 2, 1, 1200, 64, 64, "token", False), (1, 2, 2, 1100, 64, 128, "head", False)]


def check_backward(x, scale, S0, dS, lens=None, first=0, grad_dtype=torch.float32):
    off = None if lens is None else cuda(offsets_of(lens, first))
    got = tri.gdn_lin_chunk_bwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g", "dO")), scale=scale,
                                S0=None if S0 is None else cuda(S0), dS=None if dS is None else cuda(dS), offsets=off,
                                grad_dtype=grad_dtype)
    torch.cuda.synchronize()
    want = ref.lin_backward(x, scale, S0, dS, lens, first)
    mag = ref.lin_backward(x, scale, S0, dS, lens, first, magnitude=True)
    for i, name in enumerate(("dQ", "dK", "dV")):
        assert got[i].dtype == grad_dtype
        close(got[i], want[i], mag[i], TOL_ONE if name == "dV" and grad_dtype == torch.bfloat16 else TOL_O, name)
        assert relF(got[i].cpu().double(), want[i]) <= 2.0 ** -8
    err = relF(got[3].cpu().double(), want[3])
    assert torch.isfinite(got[3]).all() and err <= TOL_DG, "dg: %.3g" % err
    if S0 is not None:
        close(got[4], want[4], mag[4], TOL_S, "dS0")
    else:
        assert got[4] is None
    return got


@gpu
@pytest.mark.parametrize("case", BWD, ids=[str(i) for i in range(len(BWD))])
def test_backward(case):
    B, H, Hk, T, dk, dv, decay, strong = case
    say(f"lin backward {case}")
    x = ref.lin_inputs(T, B, H, Hk, T, dk, dv, decay, strong=strong)
    check_backward(x, 0.25, x["S0"], x["dS"])
    check_backward(x, 0.25, None, None, grad_dtype=torch.bfloat16)
    check_backward(x, 0.25, x["S0"], None)


@gpu
@pytest.mark.parametrize("lens", [[0, 70, 0, 1, 129, 63, 0], [1100, 2, 300], [3] * 70 + [100]])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_backward_packed(lens, decay):
    first, behind = 2, 4
    T = first + sum(lens) + behind
    say(f"lin backward packed {len(lens)} sequences, {T} tokens, {decay}")
    x = ref.lin_inputs(13, 1, 4, 2, T, 64, 64, decay, n_state=len(lens))
    got = check_backward(x, 0.25, x["S0"], x["dS"], lens, first)
    for t in got[:3] + ((got[3],) if decay == "token" else ()):
        rows = torch.cat([t[:, :, :first].flatten(), t[:, :, T - behind:].flatten()])
        assert torch.count_nonzero(rows) == 0  # rows of no sequence get no gradient


@gpu
def test_backward_no_tokens():
    say("lin backward T=0")
    for decay in ("token", "head"):
        x = ref.lin_inputs(1, 2, 3, 3, 0, 64, 64, decay)
        out = tri.gdn_lin_chunk_bwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g", "dO")), S0=cuda(x["S0"]), dS=cuda(x["dS"]))
        torch.cuda.synchronize()
        assert torch.equal(out[4].cpu(), x["dS"]) and torch.count_nonzero(out[3]) == 0


@gpu
def test_backward_is_the_difference_of_the_forward():
    """O and S_out are linear in V, in Q (S_out not at all) and, given S0 = 0, in K: the
    gradients' products with other values equal the outputs' products with dO and dS there.
    In g: central differences."""
    B, H, Hk, T, dk, dv = 1, 4, 2, 190, 64, 64
    say("lin backward against differences")
    x = ref.lin_inputs(21, B, H, Hk, T, dk, dv)
    y = ref.lin_inputs(22, B, H, Hk, T, dk, dv)
    d = {n: cuda(t) for n, t in x.items()}
    args = lambda z: (z["Q"], z["K"], z["V"], z["g"])  # noqa: E731
    dQ, dK, dV, dg, _ = tri.gdn_lin_chunk_bwd(*args(d), d["dO"], dS=d["dS"], grad_dtype=torch.float32)

    def loss(z):
        O, S = tri.gdn_lin_chunk_fwd(*args(z), o_dtype=torch.float32)
        return float((O.double() * d["dO"].double()).sum()), float((S.double() * d["dS"].double()).sum())

    for name, grad in (("Q", dQ), ("K", dK), ("V", dV)):
        z = {**d, name: cuda(y[name])}
        lo, ls = loss(z)
        want = lo + (ls if name != "Q" else 0.0)
        got = float((grad.double() * z[name].double()).sum())
        # both sides are sums with relative errors of about 2^-16 a term, adding at random
        room = 2.0 ** -14 * float((grad.double() * z[name].double()).square().sum().sqrt()) * 8
        assert abs(got - want) <= room + 1e-4 * abs(want), (name, got, want)
    way = cuda(torch.randn(x["g"].shape, generator=torch.Generator().manual_seed(1)))
    e = 2.0 ** -7
    plus, minus = ({**d, "g": d["g"] + s * e * way} for s in (1, -1))
    num = (sum(loss(plus)) - sum(loss(minus))) / (2 * e)
    ana = float((dg.double() * way.double()).sum())
    # third derivative: e^2/6 of sums of up to 30 coupled log-decays; a percent of the norm
    assert abs(num - ana) <= 0.02 * float((dg.double() * way.double()).square().sum().sqrt()) * 8, (num, ana)


@gpu
def test_same_call_same_bits():
    say("lin forward and backward twice")
    x = {n: cuda(t) for n, t in ref.lin_inputs(31, 1, 4, 1, 1500, 64, 64, "head").items()}
    for _ in range(2):
        a = tri.gdn_lin_chunk_bwd(x["Q"], x["K"], x["V"], x["g"], x["dO"], S0=x["S0"], dS=x["dS"])
        b = tri.gdn_lin_chunk_bwd(x["Q"], x["K"], x["V"], x["g"], x["dO"], S0=x["S0"], dS=x["dS"])
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@gpu
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 96), (128, 256), (64, 32)])
@pytest.mark.parametrize("n", [1, 2, 7])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode(dk, dv, n, dtype):
    """fp32 arithmetic throughout: 1e-5 in the norm; O in bf16 adds its half step."""
    for H, Hk, decay in ((4, 2, "token"), (3, 3, "head")):
        say(f"lin decode dk={dk} dv={dv} n={n} {dtype} H={H} Hk={Hk} {decay}")
        x = ref.lin_inputs(n, 3, H, Hk, n, dk, dv, decay)
        if dtype == torch.float32:
            gen = torch.Generator().manual_seed(9)
            for k in ("Q", "K", "V"):
                x[k] = torch.randn(x[k].shape, generator=gen)
        a = [cuda(x[k].to(dtype)) for k in ("Q", "K", "V")] + [cuda(x["g"])]
        O, S = tri.gdn_lin_decode(*a, S=cuda(x["S0"]), o_dtype=torch.float32)
        O16, S16 = tri.gdn_lin_decode(*a)
        torch.cuda.synchronize()
        want = ref.lin_forward(x, dk ** -0.5, x["S0"])
        zero = ref.lin_forward(x, dk ** -0.5)
        assert relF(O.cpu(), want[0]) <= 1e-5 and relF(S.cpu(), want[1]) <= 1e-5
        assert O16.dtype == torch.bfloat16
        assert relF(O16.cpu().double(), zero[0]) <= 2.0 ** -8 and relF(S16.cpu(), zero[1]) <= 1e-5


@gpu
def test_decode_in_place_forgets_and_empty():
    say("lin decode in place, -inf, n=0")
    x = ref.lin_inputs(5, 2, 4, 2, 3, 128, 128)
    x["g"][0, 1, 1] = -float("inf")
    d = {n: cuda(t) for n, t in x.items()}
    S = d["S0"].clone()
    O, out = tri.gdn_lin_decode(d["Q"], d["K"], d["V"], d["g"], S=S, S_out=S, o_dtype=torch.float32)
    torch.cuda.synchronize()
    want = ref.lin_forward(x, 128 ** -0.5, x["S0"])
    assert out is S and relF(O.cpu(), want[0]) <= 1e-5 and relF(S.cpu(), want[1]) <= 1e-5
    e = {n: d[n][:, :, :0].contiguous() for n in ("Q", "K", "V", "g")}
    _, S2 = tri.gdn_lin_decode(e["Q"], e["K"], e["V"], e["g"], S=S)
    torch.cuda.synchronize()
    assert torch.equal(S, S2)


@gpu
def test_prompt_then_tokens():
    """A prompt chunk-wise, then single tokens from its state: the outputs of the whole
    sequence at once, and the gated norm and the residual sum behind them run on both."""
    B, H, Hk, T, n, d = 2, 4, 2, 131, 3, 64
    say("lin prompt then decode then norms")
    x = ref.lin_inputs(41, B, H, Hk, T + n, d, d)
    c = {k: cuda(t) for k, t in x.items()}
    cut = lambda k, a, b: c[k][:, :, a:b].contiguous()  # noqa: E731
    whole, S_all = tri.gdn_lin_chunk_fwd(c["Q"], c["K"], c["V"], c["g"], o_dtype=torch.float32)
    O, S = tri.gdn_lin_chunk_fwd(*(cut(k, 0, T) for k in ("Q", "K", "V", "g")), o_dtype=torch.float32)
    outs = [O]
    for t in range(T, T + n):
        o, S = tri.gdn_lin_decode(*(cut(k, t, t + 1) for k in ("Q", "K", "V", "g")), S=S, S_out=S,
                                  o_dtype=torch.float32)
        outs.append(o)
    got = torch.cat(outs, 2)
    want, mag = ref.lin_forward(x, d ** -0.5), ref.lin_forward(x, d ** -0.5, magnitude=True)
    close(got, want[0], mag[0], TOL_O, "O")
    close(whole, want[0], mag[0], TOL_O, "O at once")
    close(S, want[1], mag[1], TOL_S, "S")
    gen = torch.Generator().manual_seed(2)
    Z, w = torch.randn((B, T + n, H, d), generator=gen), 1 + 0.1 * torch.randn(d, generator=gen)
    X = torch.randn((B, T + n, H * d), generator=gen)
    Y = tri.gdn_gate_norm_fwd(got, cuda(Z), cuda(w))
    R, N = tri.gdn_residual_norm_fwd(cuda(X), Y.flatten(2), alpha=0.5)
    torch.cuda.synchronize()
    y = ref.gate_norm(want[0], Z, w, 1e-6, "silu")
    r, nn = ref.residual_norm(X, y.flatten(2), None, None, 0.5, None, 1e-6)
    # the norm divides by rows whose size the outputs' error (2^-14 M) may be a part of
    assert relF(Y.cpu(), y) <= 1e-4 and relF(R.cpu(), r) <= 1e-4 and relF(N.cpu(), nn) <= 1e-4


@gpu
def test_captured_and_on_another_stream():
    """A captured call replayed between eager ones, and a call on a stream of its own, give the
    eager call's bits."""
    say("lin captured and streamed")
    T = 5000
    c = {k: cuda(t) for k, t in ref.lin_inputs(51, 1, 4, 2, T, 64, 64).items()}
    args = (c["Q"], c["K"], c["V"], c["g"])

    def both():
        O, S = tri.gdn_lin_chunk_fwd(*args, S0=c["S0"])
        return (O, S) + tri.gdn_lin_chunk_bwd(*args, c["dO"], S0=c["S0"], dS=c["dS"])

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
        again = both()
        assert all(torch.equal(a, b) for a, b in zip(eager, again)), i
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O, S = tri.gdn_lin_chunk_fwd(*args, S0=c["S0"], stream=s)
    g = tri.gdn_lin_chunk_bwd(*args, c["dO"], S0=c["S0"], dS=c["dS"], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, (O, S) + g))


@gpu
def test_caller_tensors_and_workspace():
    say("lin caller workspace")
    x = {k: cuda(t) for k, t in ref.lin_inputs(61, 1, 2, 2, 5000, 64, 64).items()}
    need = tri.gdn_lin_chunk_fwd_workspace_bytes(1, 2, 5000, 64, 64)
    O = torch.empty((1, 2, 5000, 64), device="cuda", dtype=torch.bfloat16)
    S = torch.empty((1, 2, 64, 64), device="cuda")
    ws = torch.empty(need, device="cuda", dtype=torch.uint8)
    o, s = tri.gdn_lin_chunk_fwd(x["Q"], x["K"], x["V"], x["g"], O=O, S_out=S, workspace=ws)
    ref_o, ref_s = tri.gdn_lin_chunk_fwd(x["Q"], x["K"], x["V"], x["g"])
    torch.cuda.synchronize()
    assert o is O and s is S and torch.equal(O, ref_o) and torch.equal(S, ref_s)
    with pytest.raises(tri.GdnError) as e:
        tri.gdn_lin_chunk_fwd(x["Q"], x["K"], x["V"], x["g"], workspace=ws[:need - 16])
    assert e.value.status == tri.GDN_ERR_WORKSPACE


@gpu
def test_python_refusals():
    """Wrong shapes, types, layouts and devices raise before anything is launched."""
    x = {k: cuda(t) for k, t in ref.lin_inputs(1, 1, 4, 2, 8, 64, 64).items()}
    ok = (x["Q"], x["K"], x["V"], x["g"])
    fwd = tri.gdn_lin_chunk_fwd
    off = torch.tensor([0, 8], device="cuda", dtype=torch.int32)
    for bad in (lambda: fwd(x["Q"][:, :1], *ok[1:]), lambda: fwd(x["Q"].float(), *ok[1:]),
                lambda: fwd(x["Q"].cpu(), *ok[1:]), lambda: fwd(*ok[:3], x["g"].double()),
                lambda: fwd(*ok[:3], x["g"][:, :2]), lambda: fwd(*ok, S0=x["S0"][:, :2]),
                lambda: fwd(*ok, offsets=off.long()), lambda: fwd(*ok, offsets=off.cpu()),
                lambda: fwd(*ok, O=torch.empty(1, device="cuda")), lambda: fwd(x["Q"], x["K"], x["V"][:, :3], ok[3]),
                lambda: fwd(x["Q"].transpose(1, 2).contiguous().transpose(1, 2), *ok[1:]),
                lambda: fwd(None, *ok[1:]), lambda: tri.gdn_lin_chunk_bwd(*ok, x["dO"][..., :32]),
                lambda: tri.gdn_lin_chunk_bwd(*ok, x["dO"], grad_dtype=torch.float16)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(tri.GdnError):  # d_v
        fwd(x["Q"], x["K"], x["V"][..., :24].contiguous(), x["g"])
    with pytest.raises(tri.GdnError):  # backward: d_v
        tri.gdn_lin_chunk_bwd(x["Q"], x["K"], x["V"][..., :32].contiguous(), x["g"], x["dO"][..., :32].contiguous())


# ---- refusals of the C entry points, on the CPU: fake pointers, returned before any HIP call --

FAKE = 0x10000


def shape(**kw):
    s = tri.gdn_lin_shape()
    s.T, s.B, s.H, s.H_qk = kw.get("T", 100), kw.get("B", 2), kw.get("H", 4), kw.get("H_qk", 2)
    s.d_k, s.d_v, s.g_per_head, s.scale = kw.get("d_k", 64), kw.get("d_v", 64), kw.get("per_head", 0), 1.0
    s.offsets = kw.get("offsets", None)
    return s


def c_fwd(s, Q=FAKE, g=FAKE, S0=None, O=FAKE, dt=tri.GDN_BF16, odt=tri.GDN_BF16, ws=FAKE, nb=1 << 40):
    return tri._lib.gdn_lin_chunk_fwd(ctypes.byref(s) if s is not None else None, Q, FAKE, FAKE, dt, g, S0, O, odt, FAKE,
                                      ws, nb, None)


def c_bwd(s, dO=FAKE, gdt=tri.GDN_BF16, ws=FAKE, nb=1 << 40):
    return tri._lib.gdn_lin_chunk_bwd(ctypes.byref(s) if s is not None else None, FAKE, FAKE, FAKE, tri.GDN_BF16, FAKE,
                                      None, dO, None, FAKE, FAKE, FAKE, gdt, FAKE, None, ws, nb, None)


def c_dec(s, S_out=FAKE, dt=tri.GDN_BF16):
    return tri._lib.gdn_lin_decode(ctypes.byref(s) if s is not None else None, FAKE, FAKE, FAKE, dt, FAKE, None, S_out,
                                   FAKE, tri.GDN_BF16, None)


def test_c_refusals():
    for call in (c_fwd, c_bwd, c_dec):
        assert call(None) == 1
        assert call(shape(B=-1)) == 2 and call(shape(T=-1)) == 2 and call(shape(d_k=0)) == 2
        assert call(shape(H=4, H_qk=3)) == 2 and call(shape(H=4, H_qk=0)) == 2 and call(shape(per_head=2)) == 2
        assert call(shape(d_k=96)) == 5 and call(shape(d_v=48)) == 5 and call(shape(d_v=288)) == 5
        assert call(shape(T=2 ** 31 - 64)) == 5 and call(shape(B=2 ** 16, H=2 ** 16, H_qk=1)) == 5
        assert call(shape(B=0)) == 0 and call(shape(H=0, H_qk=0)) == 0
    assert c_bwd(shape(d_v=32)) == 5 and c_bwd(shape(), gdt=4) == 3 and c_bwd(shape(), dO=None) == 1
    assert c_bwd(shape(), ws=None) == 6 and c_bwd(shape(), nb=16) == 6 and c_bwd(shape(), ws=FAKE + 4) == 4
    assert c_fwd(shape(), Q=None) == 1 and c_fwd(shape(), g=None) == 1 and c_fwd(shape(), O=None) == 1
    assert c_fwd(shape(), dt=tri.GDN_F32) == 5 and c_fwd(shape(), dt=9) == 3 and c_fwd(shape(), odt=2) == 3
    assert c_fwd(shape(), S0=FAKE + 4) == 4 and c_fwd(shape(), Q=FAKE + 8) == 4 and c_fwd(shape(offsets=FAKE + 4)) == 4
    long = shape(B=1, H=2, H_qk=2, T=100000)
    assert c_fwd(long, ws=None) == 6 and c_fwd(long, nb=64) == 6
    assert c_dec(shape(offsets=FAKE)) == 5 and c_dec(shape(), S_out=None) == 1 and c_dec(shape(), dt=3) == 3


def test_workspace_queries():
    fwd, bwd = tri.gdn_lin_chunk_fwd_workspace_bytes, tri.gdn_lin_chunk_bwd_workspace_bytes
    assert fwd(32, 16, 8192, 128, 128) == 0         # heads and sequences fill the GPU
    assert fwd(1, 2, 64, 64, 64) == 0               # nothing to divide
    assert fwd(1, 2, 100000, 64, 64) >= 2 * 64 * 64 * 4
    assert fwd(1, 3, 100, 96, 64) == 0 and bwd(1, 3, 100, 64, 32) == 0  # refused arguments
    assert bwd(0, 4, 100, 64, 64) == 0 and bwd(2, 4, 100, 64, 64) > 0
    assert bwd(2, 4, 100, 64, 64, H_qk=2) > bwd(2, 4, 100, 64, 64)


@gpu
def test_rows_beyond_32_bits():
    """16 heads of 1.1 million tokens: 2.25e9 values a tensor.  Every head forgets at one token
    near the end, so the rest equals a call on that rest alone."""
    H, T, t0, d = 16, 1_100_000, 1_099_000, 128
    say("lin forward beyond 2^31 values")
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((1, H, T, d), generator=gen, device="cuda", dtype=torch.bfloat16) * 0.1 for _ in range(3))
    g = torch.full((1, H, T), -0.05, device="cuda")
    g[:, :, t0] = -float("inf")
    O, S = tri.gdn_lin_chunk_fwd(q, k, v, g)
    cut = lambda x: x[:, :, t0:].contiguous()  # noqa: E731
    O2, S2 = tri.gdn_lin_chunk_fwd(cut(q), cut(k), cut(v), cut(g))
    torch.cuda.synchronize()
    # the chunks' borders differ: fp32 sums in another order, and the one part's roundings
    assert relF(S.cpu(), S2.cpu()) <= 2.0 ** -17
    assert relF(O[:, :, t0:].cpu().double(), O2.cpu().double()) <= 2.0 ** -7


@gpu
def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, give the bits of one after the other."""
    say("lin on two streams")
    xs = [{k: cuda(t) for k, t in ref.lin_inputs(71 + i, 1, 4, 2, 5000, 64, 64).items()} for i in range(2)]
    call = lambda x, s=None: (tri.gdn_lin_chunk_fwd(x["Q"], x["K"], x["V"], x["g"], S0=x["S0"], stream=s) +  # noqa: E731
                              tri.gdn_lin_chunk_bwd(x["Q"], x["K"], x["V"], x["g"], x["dO"], dS=x["dS"], stream=s)[:4])
    one = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        both = [call(x, s) for x, s in zip(xs, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(one, both):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@gpu
def test_backward_leaves_nothing_unwritten():
    """Every gradient is written in full, rows of no sequence as zeros: a call into memory that
    held NaN (the allocator hands freed blocks out again) shows none."""
    say("lin backward outputs whole")
    lens, first, behind = [70, 0, 64, 1], 3, 6
    T = first + sum(lens) + behind
    x = {k: cuda(t) for k, t in ref.lin_inputs(81, 1, 4, 2, T, 64, 64, n_state=len(lens)).items()}
    off = cuda(offsets_of(lens, first))
    for _ in range(3):
        out = tri.gdn_lin_chunk_bwd(x["Q"], x["K"], x["V"], x["g"], x["dO"], S0=x["S0"], offsets=off)
        assert all(torch.isfinite(t).all() for t in out)
        for t in out:
            t.fill_(float("nan"))
        del out, t


@gpu
@pytest.mark.parametrize("T,n,dk,dv,odt", [
    (64, 1, 128, 128, torch.bfloat16), (100, 37, 64, 64, torch.float32), (130, 66, 128, 256, torch.bfloat16),
    (200, 160, 64, 32, torch.bfloat16), (4500, 4301, 128, 128, torch.float32), (300, 255, 128, 128, torch.float32)])
def test_what_pads_a_sequence_reaches_no_earlier_row(T, n, dk, dv, odt):
    """The rows behind the first n hold NaN, infinities and the largest values: the first n rows
    of O are those of the n tokens alone (fp32 sums in another order, one rounding of the type).
    Infinities in single columns of V leave the other columns of later rows finite."""
    say(f"lin forward, {T - n} bad rows behind {n}")
    x = ref.lin_inputs(T + n, 2, 2, 1, T, dk, dv)
    bad = {k: x[k].clone() for k in ("Q", "K", "V", "g")}
    for i, k in enumerate(("Q", "K", "V", "g")):
        bad[k][:, :, n:] = float("nan")
        bad[k][:, :, n + 1::3] = (-1) ** i * float("inf")
        bad[k][:, :, n + 2::3] = torch.finfo(bad[k].dtype).max
    O, _ = run_forward(bad, 0.2, x["S0"], o_dtype=odt)
    some = dict(x, V=x["V"].clone())
    some["V"][:, :, n, 5::7] = float("inf")
    P, _ = run_forward(some, 0.2, x["S0"], o_dtype=odt)
    torch.cuda.synchronize()
    want, mag = ref.lin_forward(x, 0.2, x["S0"]), ref.lin_forward(x, 0.2, x["S0"], magnitude=True)
    tol = TOL_O if odt == torch.float32 else TOL_ONE
    close(O[:, :, :n], want[0][:, :, :n], mag[0][:, :, :n], tol, "O before the padding")
    close(P[:, :, :n], want[0][:, :, :n], mag[0][:, :, :n], tol, "O before infinities in V")
    fine = [c for c in range(dv) if c % 7 != 5]
    close(P[..., fine], want[0][..., fine], mag[0][..., fine], tol, "the other columns")
    assert not torch.isfinite(P[:, :, n, 5::7]).any()


@gpu
def test_backward_of_no_sequence():
    """No sequence at all: the heads' decays get zeros, and so do packed rows (from C, where offsets
    of one entry are valid)."""
    say("lin backward without sequences")
    x = ref.lin_inputs(3, 0, 4, 2, 70, 64, 64, "head")
    dQ, dK, dV, dg, _ = tri.gdn_lin_chunk_bwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g", "dO")))
    assert dQ.numel() == 0 and dV.numel() == 0 and dg.shape == (4,)
    y = ref.lin_inputs(3, 1, 4, 2, 70, 64, 64, "head")
    t = {n: cuda(y[n]) for n in ("Q", "K", "V", "g", "dO")}
    out = [torch.full_like(t[n], 7.0) for n in ("Q", "K", "V", "g")]
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    sh = tri.gdn_lin_shape(70, off.data_ptr(), 0, 4, 2, 64, 64, 1, 1.0)
    at = lambda n: t[n].data_ptr()  # noqa: E731
    st = tri._lib.gdn_lin_chunk_bwd(ctypes.byref(sh), at("Q"), at("K"), at("V"), tri.GDN_BF16, at("g"), None, at("dO"), None,
                                    out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), tri.GDN_BF16,
                                    out[3].data_ptr(), None, None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.count_nonzero(dg) == 0
    assert all(torch.count_nonzero(o) == 0 for o in out)


@gpu
def test_the_given_state_is_not_the_returned_one():
    x = ref.lin_inputs(3, 1, 2, 2, 70, 64, 64)
    S = cuda(x["S0"])
    with pytest.raises(ValueError, match="S_out must not be S0"):
        tri.gdn_lin_chunk_fwd(*(cuda(x[n]) for n in ("Q", "K", "V", "g")), S0=S, S_out=S)


def test_c_refusals_of_launches_too_large():
    """Sizes whose launches would have more than 2^32 threads are refused before anything runs."""
    for call in (c_fwd, c_bwd):
        assert call(shape(B=2 ** 23, H=2, H_qk=2, T=64)) == 5
        assert call(shape(B=2 ** 30, H=1, H_qk=1, T=2 ** 30)) == 5
    assert tri.gdn_lin_chunk_fwd_workspace_bytes(2 ** 30, 1, 2 ** 30, 64, 64) == 0
    assert tri.gdn_lin_chunk_bwd_workspace_bytes(2 ** 30, 1, 2 ** 30, 64, 64) == 0
    assert tri._lib.gdn_gate_norm_fwd(FAKE, FAKE, 4 * 128, None, FAKE, 1, 2, 4, 2 ** 24, 128, 0, 1e-6, None) == 5


@gpu
def test_no_tokens_without_tensors():
    """T = 0 from C with every tensor of rows NULL, a decay per head among them: the states pass."""
    say("lin C calls, T=0, no tensors")
    S0 = torch.randn((2, 3, 64, 64), device="cuda")
    S, D = torch.full_like(S0, 7.0), torch.full_like(S0, 7.0)
    for per_head in (0, 1):
        sh = tri.gdn_lin_shape(0, None, 2, 3, 3, 64, 64, per_head, 1.0)
        stream = torch.cuda.current_stream().cuda_stream
        assert tri._lib.gdn_lin_chunk_fwd(ctypes.byref(sh), None, None, None, tri.GDN_BF16, None, S0.data_ptr(), None,
                                          tri.GDN_BF16, S.data_ptr(), None, 0, stream) == 0
        need = tri._lib.gdn_lin_chunk_bwd_workspace_bytes(ctypes.byref(sh))
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        assert tri._lib.gdn_lin_chunk_bwd(ctypes.byref(sh), None, None, None, tri.GDN_BF16, None, S0.data_ptr(), None,
                                          S0.data_ptr(), None, None, None, tri.GDN_BF16, None, D.data_ptr(),
                                          ws.data_ptr(), need, stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(S, S0) and torch.equal(D, S0)
