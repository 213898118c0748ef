"""GPU parity of the gated linear recurrence (whole sequences, gradients, single tokens) against fp64.

Tolerances: the bound that the reference carries through the recurrence (rec_reference.py); outputs
stored in bf16 add half a step, 2^-8 of the value."""
import ctypes

import pytest
import torch

import rec_reference as ref
from helpers import cuda, say

tri = pytest.importorskip("tri_inverse_amd")
gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
KINDS = [(d, n, g) for d in ("power", "sigmoid", "log") for n in ("sqrt", "linear", "none") for g in (True, False)]


def close(got, want, bound, what):
    got = got.detach().cpu()
    assert tuple(got.shape) == tuple(want.shape), what
    half = 2.0 ** -8 if got.dtype == BF else 0.0
    assert torch.isfinite(got).all(), what
    room = bound + half * (want.abs() + bound) + 1e-30
    worst = float(((got.double() - want).abs() / room).max()) if want.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g of its tolerance" % (what, worst)


def up(t):
    return None if t is None else cuda(t)


def offsets_of(lens, first):
    return cuda(torch.tensor([first] + lens).cumsum(0).to(torch.int32))


def check(x, decay, norm, h0=True, dh=True, lens=None, first=0, give_states=True):
    """Forward and backward of one call against the reference."""
    h0, dh = (x["h0"] if h0 else None), (x["dh"] if dh else None)
    how = dict(I=up(x["I"]), w=up(x["w"]), h0=up(h0), decay=decay, norm=norm,
               offsets=None if lens is None else offsets_of(lens, first))
    X, A, dH = up(x["X"]), up(x["A"]), up(x["dH"])
    H = torch.full_like(X, 7.0)
    H, h, states = tri.gdn_rec_fwd(X, A, want_states=True, H=H, **how)
    got = tri.gdn_rec_bwd(X, A, dH, dh=up(dh), states=states if give_states else None, **how)
    torch.cuda.synchronize()
    Hr, hr, EH, Eh, (before, _, Eb) = ref.rec_forward(x, decay, norm, h0, lens, first)
    B, T, _ = X.shape
    inside = torch.zeros((B, T), dtype=torch.bool)
    starts = set()
    for row, s, e in ref.spans_of(B, T, lens, first):
        inside[row, s:e] = True
        starts.add((row, s))
    assert (H.cpu()[~inside] == 7.0).all(), "rows of no sequence were written"
    close(H.cpu()[inside], Hr[inside], EH[inside], "H")
    close(h, hr, Eh, "h_out")
    assert tuple(states.shape) == (B, (T + 63) // 64, X.shape[2])
    for b in range(B):
        for j in range(states.shape[1]):
            inner = inside[b, 64 * j] and (b, 64 * j) not in starts
            close(states[b, j], before[b, 64 * j] * inner, Eb[b, 64 * j] * inner, "states")
    want, bound = ref.rec_backward(x, decay, norm, h0, dh, lens, first)
    for name, g, y, e in zip(("dX", "dA", "dI", "dw", "dh0"), got, want, bound):
        if y is None or (name == "dh0" and h0 is None):
            assert g is None, name
        else:
            close(g, y, e, name)
            if name in ("dX", "dA", "dI"):
                assert (g.cpu()[~inside] == 0).all(), name


@gpu
@pytest.mark.parametrize("decay,norm,gate", KINDS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_kinds(decay, norm, gate, dtype):
    say(f"recurrence {decay} {norm} gate={gate} {dtype}")
    check(ref.rec_inputs(3, 2, 150, 136, decay, gate, dtype), decay, norm)


SHAPES = [(1, 1, 8), (3, 2, 128), (1, 7, 264), (2, 8, 72), (1, 9, 16), (2, 63, 136), (1, 64, 128), (2, 65, 8), (1, 127, 40),
          (1, 128, 256), (1, 129, 120), (3, 321, 24), (1, 1100, 8)]


@gpu
@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("states", [True, False])
def test_shapes(B, T, D, states):
    say(f"recurrence B={B} T={T} D={D} states={states}")
    x = ref.rec_inputs(T + D, B, T, D, "power", True, BF if T % 2 else F32)
    check(x, "power", "sqrt", give_states=states)
    check(x, "power", "sqrt", h0=False, dh=False, give_states=states)


@gpu
@pytest.mark.parametrize("decay", ["power", "sigmoid", "log"])
def test_slow_decays(decay):
    """Decays within 1e-2 to 1e-5 of 1: the input's factor is a small difference from 1."""
    say(f"recurrence slow {decay}")
    check(ref.rec_inputs(9, 1, 500, 40, decay, True, F32, slow=True), decay, "sqrt")


PACKED = [([5], 0, 0), ([1, 1, 1, 0, 2], 0, 3), ([0, 70, 0, 0, 64, 3, 0], 2, 5), ([64, 64, 128], 0, 0), ([63, 66, 200, 1], 1, 62),
          ([0, 0], 4, 60), ([8, 8, 16, 32, 1, 7], 56, 0), ([300, 2, 150], 130, 200)]


@gpu
@pytest.mark.parametrize("lens,first,tail", PACKED, ids=[str(i) for i in range(len(PACKED))])
@pytest.mark.parametrize("decay,norm,gate,dtype", [("power", "sqrt", True, F32), ("log", "none", False, BF)])
def test_packed(lens, first, tail, decay, norm, gate, dtype):
    """Packed sequences, some empty; rows before and behind them hold NaN and reach nothing."""
    say(f"recurrence packed {lens} from {first}, {tail} behind, {decay} {dtype}")
    T = first + sum(lens) + tail
    x = ref.rec_inputs(T, 1, T, 136, decay, gate, dtype, n_state=len(lens))
    for t in ("X", "A", "I", "dH"):
        if x[t] is not None:
            x[t][:, :first] = float("nan")
            x[t][:, T - tail:] = float("nan")
    x = dict(x)
    clean = {k: (torch.nan_to_num(v, nan=0.0) if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    # the reference reads no such row either; zeros keep its sums over all rows defined
    how = dict(I=up(x["I"]), w=up(x["w"]), h0=up(x["h0"]), decay=decay, norm=norm, offsets=offsets_of(lens, first))
    H, h, states = tri.gdn_rec_fwd(up(x["X"]), up(x["A"]), want_states=True, **how)
    dirty = tri.gdn_rec_bwd(up(x["X"]), up(x["A"]), up(x["dH"]), dh=up(x["dh"]), states=states, **how)
    how["I"] = up(clean["I"])
    H2, h2, s2 = tri.gdn_rec_fwd(up(clean["X"]), up(clean["A"]), want_states=True, **how)
    pure = tri.gdn_rec_bwd(up(clean["X"]), up(clean["A"]), up(clean["dH"]), dh=up(clean["dh"]), states=s2, **how)
    torch.cuda.synchronize()
    assert torch.equal(H[:, first:T - tail], H2[:, first:T - tail]) and torch.equal(h, h2) and torch.equal(states, s2)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(dirty, pure))
    check(clean, decay, norm, lens=lens, first=first)
    check(clean, decay, norm, h0=False, dh=False, lens=lens, first=first, give_states=False)


@gpu
def test_sequence_behind_an_overflow():
    """A sequence whose state becomes infinite or NaN leaves the ones beside it as they are."""
    say("recurrence beside infinities")
    lens, D = [70, 5, 130, 64], 136
    T = sum(lens)
    x = ref.rec_inputs(6, 1, T, D, "log", False, F32, n_state=4)
    how = dict(decay="log", norm="none", offsets=offsets_of(lens, 0))
    H, h, st = tri.gdn_rec_fwd(up(x["X"]), up(x["A"]), h0=up(x["h0"]), want_states=True, **how)
    g = tri.gdn_rec_bwd(up(x["X"]), up(x["A"]), up(x["dH"]), h0=up(x["h0"]), dh=up(x["dh"]), states=st, **how)
    X, dH = x["X"].clone(), x["dH"].clone()
    X[0, 3], X[0, 80], dH[0, 71], dH[0, 100] = float("inf"), float("nan"), float("nan"), float("inf")
    H2, h2, st2 = tri.gdn_rec_fwd(up(X), up(x["A"]), h0=up(x["h0"]), want_states=True, **how)
    g2 = tri.gdn_rec_bwd(up(X), up(x["A"]), up(dH), h0=up(x["h0"]), dh=up(x["dh"]), states=st2, **how)
    torch.cuda.synchronize()
    for s, e in ((0, 3), (70, 75), (75, 80), (205, 269)):
        assert torch.equal(H[:, s:e], H2[:, s:e]), (s, e)
    assert not torch.isfinite(H2[:, 3:70]).any() and not torch.isfinite(H2[:, 80:205]).any()
    assert torch.equal(h[[1, 3]], h2[[1, 3]])
    assert torch.equal(g[0][:, 205:], g2[0][:, 205:]) and torch.equal(g[1][:, 205:], g2[1][:, 205:])
    assert torch.equal(g[4][[0, 3]], g2[4][[0, 3]])


@gpu
def test_forgotten_states():
    """Log-decays of -inf forget the state; a = 1 keeps it and takes no input through sqrt(1 - a^2)."""
    say("recurrence with decays of 0 and 1")
    x = ref.rec_inputs(8, 1, 200, 72, "log", True, F32)
    x["A"][0, [5, 64, 130]] = -float("inf")
    x["A"][0, [6, 63, 128]] = 0.0
    for norm in ("sqrt", "linear", "none"):
        how = dict(I=up(x["I"]), h0=up(x["h0"]), decay="log", norm=norm)
        H, h, st = tri.gdn_rec_fwd(up(x["X"]), up(x["A"]), want_states=True, **how)
        got = tri.gdn_rec_bwd(up(x["X"]), up(x["A"]), up(x["dH"]), dh=up(x["dh"]), states=st, **how)
        torch.cuda.synchronize()
        Hr, hr, EH, Eh, _ = ref.rec_forward(x, "log", norm, x["h0"])
        close(H, Hr, EH, "H")
        close(h, hr, Eh, "h_out")
        want, bound = ref.rec_backward(x, "log", norm, x["h0"], x["dh"])
        for g, y, e in zip(got, want, bound):
            if y is not None:
                close(g, y, e, norm)


@gpu
@pytest.mark.parametrize("decay", ["power", "sigmoid"])
def test_far_gates(decay):
    """Gates whose exponential overflows or vanishes."""
    say(f"recurrence far gates {decay}")
    x = ref.rec_inputs(5, 1, 66, 40, decay, True, F32)
    x["A"][0, ::3], x["A"][0, 1::5] = 120.0, -120.0
    x["I"][0, ::4], x["I"][0, 2::7] = -110.0, 90.0
    if decay == "sigmoid":
        x["A"][0, 7], x["A"][0, 8] = -float("inf"), float("inf")
    check(x, decay, "sqrt")


@gpu
def test_rows_depend_on_no_later_token():
    say("recurrence causal")
    x = ref.rec_inputs(7, 1, 200, 40, "power", True, BF)
    how = dict(w=up(x["w"]), h0=up(x["h0"]))
    H, _, _ = tri.gdn_rec_fwd(up(x["X"]), up(x["A"]), I=up(x["I"]), **how)
    for t in (3, 64, 100, 199):
        y = {k: x[k].clone() for k in ("X", "A", "I")}
        for k in y:
            y[k][:, t:] = float("nan")
        H2, _, _ = tri.gdn_rec_fwd(up(y["X"]), up(y["A"]), I=up(y["I"]), **how)
        torch.cuda.synchronize()
        assert torch.equal(H[:, :t], H2[:, :t]), t


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_parts_of_a_projection(dtype):
    """X, A and I as parts of one row, gaps of NaN between them."""
    say(f"recurrence strided {dtype}")
    B, T, D = 2, 70, 72
    x = ref.rec_inputs(12, B, T, D, "power", True, dtype)
    wide = torch.full((B, T, 3 * D + 40), float("nan"), dtype=dtype, device="cuda")
    parts = []
    for k, at in (("X", 0), ("A", D + 16), ("I", 2 * D + 32)):
        wide[..., at:at + D] = up(x[k])
        parts.append(wide[..., at:at + D])
    how = dict(w=up(x["w"]), h0=up(x["h0"]))
    X, A, I = parts
    H, h, st = tri.gdn_rec_fwd(X, A, I, want_states=True, **how)
    g = tri.gdn_rec_bwd(X, A, up(x["dH"]), I, states=st, **how)
    H2, h2, st2 = tri.gdn_rec_fwd(up(x["X"]), up(x["A"]), up(x["I"]), want_states=True, **how)
    g2 = tri.gdn_rec_bwd(up(x["X"]), up(x["A"]), up(x["dH"]), up(x["I"]), states=st2, **how)
    y, hs = tri.gdn_rec_step(X, A, I, w=up(x["w"]), h=up(x["h0"]))
    y2, hs2 = tri.gdn_rec_step(up(x["X"]), up(x["A"]), up(x["I"]), w=up(x["w"]), h=up(x["h0"]))
    torch.cuda.synchronize()
    for a, b in zip((H, h, st) + g + (y, hs), (H2, h2, st2) + g2 + (y2, hs2)):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("decay,norm,gate", KINDS)
@pytest.mark.parametrize("B,n,D,dtype", [(3, 1, 136, BF), (1, 5, 8, F32), (70, 2, 264, BF)])
def test_step(decay, norm, gate, B, n, D, dtype):
    say(f"recurrence step {decay} {norm} gate={gate} B={B} n={n} D={D} {dtype}")
    x = ref.rec_inputs(n + D, B, n, D, decay, gate, dtype)
    Hr, hr, EH, Eh, _ = ref.rec_forward(x, decay, norm, x["h0"])
    how = dict(I=up(x["I"]), w=up(x["w"]), decay=decay, norm=norm)
    H, h = tri.gdn_rec_step(up(x["X"]), up(x["A"]), h=up(x["h0"]), **how)
    S = up(x["h0"])
    H2, h2 = tri.gdn_rec_step(up(x["X"]), up(x["A"]), h=S, h_out=S, **how)
    torch.cuda.synchronize()
    close(H, Hr, EH, "H")
    close(h, hr, Eh, "h_out")
    assert h2 is S and torch.equal(H, H2) and torch.equal(h, h2)
    Hz, hz = tri.gdn_rec_step(up(x["X"]), up(x["A"]), **how)
    torch.cuda.synchronize()
    Hr, hr, EH, Eh, _ = ref.rec_forward(x, decay, norm)
    close(Hz, Hr, EH, "H from zeros")
    close(hz, hr, Eh, "h_out from zeros")


@gpu
def test_prefill_then_steps():
    """A prompt of uneven packed sequences, then one token at a time: the states join the two."""
    say("recurrence prefill, then steps")
    lens, n, D = [130, 1, 67], 3, 136
    x = ref.rec_inputs(21, 1, sum(lens), D, "power", True, BF, n_state=3)
    y = ref.rec_inputs(22, 3, n, D, "power", True, BF)
    y["w"] = x["w"]
    _, h, _ = tri.gdn_rec_fwd(up(x["X"]), up(x["A"]), up(x["I"]), w=up(x["w"]), offsets=offsets_of(lens, 0))
    out = []
    for t in range(n):
        token = [up(y[k][:, t:t + 1]) for k in ("X", "A", "I")]
        H, h = tri.gdn_rec_step(*token, w=up(x["w"]), h=h, h_out=h)
        out.append(H)
    torch.cuda.synchronize()
    _, hr, _, Eh, _ = ref.rec_forward(x, "power", "sqrt", None, lens, 0)
    Hr, hl, EH, El, _ = ref.rec_forward(y, "power", "sqrt", hr)
    # what the prompt's states are off by decays like them: at most its bound
    close(torch.cat(out, 1), Hr, EH + Eh[:, None], "H")
    close(h, hl, El + Eh, "h_out")


@gpu
def test_no_tokens():
    say("recurrence without tokens")
    D = 16
    w, h0 = torch.ones(D, device="cuda"), torch.randn((3, D), device="cuda")
    E = torch.empty((3, 0, D), device="cuda")
    H, h, st = tri.gdn_rec_fwd(E, E, w=w, h0=h0, want_states=True)
    g = tri.gdn_rec_bwd(E, E, E, w=w, h0=h0, dh=2 * h0, states=st)
    _, z, _ = tri.gdn_rec_fwd(E, E, w=w)
    P = torch.empty((1, 0, D), device="cuda")
    off = torch.zeros(4, device="cuda", dtype=torch.int32)
    _, hp, _ = tri.gdn_rec_fwd(P, P, w=w, h0=h0, offsets=off)
    _, hs = tri.gdn_rec_step(E, E, w=w, h=h0)
    none = torch.empty((0, 5, D), device="cuda")
    Hn, hn, _ = tri.gdn_rec_fwd(none, none, w=w)
    gn = tri.gdn_rec_bwd(none, none, none, w=w)
    torch.cuda.synchronize()
    assert H.numel() == 0 and torch.equal(h, h0) and torch.equal(hp, h0) and torch.equal(hs, h0)
    assert torch.count_nonzero(z) == 0 and torch.equal(g[4], 2 * h0) and torch.count_nonzero(g[3]) == 0
    assert Hn.numel() == 0 and hn.numel() == 0 and torch.count_nonzero(gn[3]) == 0


@gpu
def test_captured_and_on_two_streams():
    """The same bits eagerly, from a graph replayed between eager calls, and from two streams at once."""
    say("recurrence captured, two streams")
    x = {k: up(v) for k, v in ref.rec_inputs(31, 2, 700, 264, "power", True, BF).items()}

    def both(stream=None):
        H, h, st = tri.gdn_rec_fwd(x["X"], x["A"], x["I"], w=x["w"], h0=x["h0"], want_states=True, stream=stream)
        g = tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], x["I"], w=x["w"], h0=x["h0"], dh=x["dh"], states=st, stream=stream)
        return (H, h, st) + g

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
def test_many_tiles():
    """More workgroups than the GPU holds at once, and a sequence of many tiles."""
    say("recurrence of many tiles")
    for B, T, D, kind in ((1, 20011, 520, "power"), (3, 4100, 1032, "sigmoid")):
        print(B, T, D, flush=True)
        x = {k: up(v) for k, v in ref.rec_inputs(T, B, T, D, kind, True, BF).items()}
        how = dict(w=x["w"], h0=x["h0"], decay=kind)
        H, h, st = tri.gdn_rec_fwd(x["X"], x["A"], x["I"], want_states=True, **how)
        g = tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], x["I"], dh=x["dh"], states=st, **how)
        g2 = tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], x["I"], dh=x["dh"], **how)
        torch.cuda.synchronize()
        Hr, hr, EH, Eh, _ = ref.rec_forward(x, kind, "sqrt", x["h0"])
        close(H, Hr.cpu(), EH.cpu(), "H")
        close(h, hr.cpu(), Eh.cpu(), "h_out")
        want, bound = ref.rec_backward(x, kind, "sqrt", x["h0"], x["dh"])
        for name, a, y, e in zip(("dX", "dA", "dI", "dw", "dh0"), g, want, bound):
            if y is not None:
                close(a, y.cpu(), e.cpu(), name)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(g, g2))


@gpu
@pytest.mark.parametrize("lens,first,tail", [([9000, 1, 0, 300, 8193, 5000, 64, 4096], 70, 40), ([1] * 700 + [0, 9001], 0, 0),
                                             ([127, 8192, 1025, 63, 7777], 1, 0), ([20000], 500, 9000)],
                         ids=["mixed", "ones", "odd", "one"])
def test_packed_over_many_tiles(lens, first, tail):
    """Sequences that start and end in any of the tiles that join by eights and by 64."""
    say(f"recurrence packed over many tiles, {len(lens)} sequences")
    T = first + sum(lens) + tail
    x = {k: up(v) for k, v in ref.rec_inputs(T, 1, T, 24, "power", True, F32, n_state=len(lens), slow=True).items()}
    how = dict(I=x["I"], w=x["w"], h0=x["h0"], offsets=offsets_of(lens, first))
    H, h, st = tri.gdn_rec_fwd(x["X"], x["A"], want_states=True, **how)
    g = tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], dh=x["dh"], states=st, **how)
    torch.cuda.synchronize()
    inside = slice(first, first + sum(lens))
    Hr, hr, EH, Eh, _ = ref.rec_forward(x, "power", "sqrt", x["h0"], lens, first)
    close(H[:, inside], Hr[:, inside].cpu(), EH[:, inside].cpu(), "H")
    close(h, hr.cpu(), Eh.cpu(), "h_out")
    want, bound = ref.rec_backward(x, "power", "sqrt", x["h0"], x["dh"], lens, first)
    for name, a, y, e in zip(("dX", "dA", "dI", "dw", "dh0"), g, want, bound):
        close(a, y.cpu(), e.cpu(), name)


@gpu
def test_one_row_of_any_stride():
    """One sequence of one token: its strides say nothing."""
    say("recurrence, one row")
    x = ref.rec_inputs(3, 1, 1, 24, "sigmoid", False, F32)
    X, A = (torch.as_strided(up(x[k]), (1, 1, 24), (3, 5, 1)) for k in ("X", "A"))
    H, h, _ = tri.gdn_rec_fwd(X, A, decay="sigmoid")
    torch.cuda.synchronize()
    Hr, hr, EH, Eh, _ = ref.rec_forward(x, "sigmoid", "sqrt")
    close(H, Hr, EH, "H")
    close(h, hr, Eh, "h_out")


@gpu
def test_one_workspace_for_calls_in_a_row():
    """A workspace left by another call, of other sizes, changes nothing."""
    say("recurrence, one workspace")
    ws = torch.full((1 << 22,), 0xAB, device="cuda", dtype=torch.uint8)
    for seed, (B, T, D, kind) in enumerate([(1, 2000, 264, "power"), (3, 500, 40, "log"), (2, 1300, 136, "sigmoid")]):
        assert max(tri.gdn_rec_fwd_workspace_bytes(B, T, D), tri.gdn_rec_bwd_workspace_bytes(B, T, D, kind)) <= ws.numel()
        x = {k: up(v) for k, v in ref.rec_inputs(seed, B, T, D, kind, True, BF).items()}
        how = dict(I=x["I"], w=x["w"], h0=x["h0"], decay=kind)
        one = tri.gdn_rec_fwd(x["X"], x["A"], want_states=True, workspace=ws, **how)
        one += tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], states=one[2], workspace=ws, **how)
        one += tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], workspace=ws, **how)
        own = tri.gdn_rec_fwd(x["X"], x["A"], want_states=True, **how)
        own += tri.gdn_rec_bwd(x["X"], x["A"], x["dH"], states=own[2], **how) * 2
        torch.cuda.synchronize()
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(one, own))


@gpu
def test_python_refusals():
    X = torch.zeros((2, 5, 16), device="cuda")
    w, h = torch.ones(16, device="cuda"), torch.zeros((2, 16), device="cuda")
    f = tri.gdn_rec_fwd
    off = torch.tensor([0, 5], device="cuda", dtype=torch.int32)
    for bad in (lambda: f(X, X), lambda: f(X, X, w=w, decay="log"), lambda: f(X, X, w=w, decay="exp"),
                lambda: f(X, X, w=w, norm="rms"), lambda: f(X, X.bfloat16(), w=w), lambda: f(X, X[:, :4], w=w),
                lambda: f(X, X.cpu(), w=w), lambda: f(X.half(), X.half(), w=w), lambda: f(X, X, w=w[:8]),
                lambda: f(X, X, w=w.double()), lambda: f(X, X, w=w, h0=h[:1]), lambda: f(X, X, w=w, h0=h, h_out=h),
                lambda: f(X, X, w=w, offsets=off), lambda: f(X[:1], X[:1], w=w, offsets=off.long()),
                lambda: f(X.transpose(0, 1), X, w=w), lambda: f(X[:, ::2], X[:, ::2], X[:, :3].transpose(1, 2), w=w),
                lambda: f(X, X[:, :1].expand(2, 5, 16), w=w), lambda: f(X[0], X[0], w=w),
                lambda: f(X, X, w=w, H=X[:, :, :8]), lambda: f(X, X, w=w, workspace=torch.zeros(8)),
                lambda: tri.gdn_rec_bwd(X, X, X[:1], w=w), lambda: tri.gdn_rec_bwd(X, X, X, w=w, dh=h[:, :8]),
                lambda: tri.gdn_rec_bwd(X, X, X, w=w, states=h), lambda: tri.gdn_rec_step(X, X, w=w, h=h[:1])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    odd = torch.zeros((2, 5, 12), device="cuda")
    with pytest.raises(tri.GdnError):
        f(odd, odd, decay="sigmoid")
    long = torch.zeros((2, 200, 16), device="cuda")
    with pytest.raises(tri.GdnError):
        f(long, long, decay="sigmoid", workspace=torch.zeros(16, device="cuda"))


# ---- refusals of the C entry points, on the CPU ------------------------------------------------

FAKE = 0x10000


def shape(**kw):
    d = dict(T=200, offsets=None, x_stride=64, a_stride=64, i_stride=64, B=2, D=64, decay=0, norm=0, dtype=0)
    d.update(kw)
    return tri.gdn_rec_shape(*(d[f] for f, _ in tri.gdn_rec_shape._fields_))


def test_c_refusals():
    lib = tri._lib
    by = ctypes.byref

    def fwd(X=FAKE, I=None, w=FAKE, h0=None, H=FAKE, ws=FAKE, nb=1 << 30, **kw):
        return lib.gdn_rec_fwd(by(shape(**kw)), X, FAKE, I, w, h0, H, None, None, ws, nb, None)

    def bwd(X=FAKE, I=None, w=FAKE, dH=FAKE, dI=None, dw=None, ws=FAKE, nb=1 << 30, **kw):
        return lib.gdn_rec_bwd(by(shape(**kw)), X, FAKE, I, w, None, None, dH, None, FAKE, FAKE, dI, dw, None, ws, nb, None)

    def step(X=FAKE, h_out=FAKE, w=FAKE, **kw):
        return lib.gdn_rec_step(by(shape(**kw)), X, FAKE, None, w, None, h_out, FAKE, None)

    for f in (fwd, bwd, step):
        assert f(B=-1) == 2 and f(T=-1) == 2 and f(D=0) == 2 and f(decay=3) == 2 and f(norm=-1) == 2
        assert f(dtype=2) == 3 and f(D=60) == 5 and f(x_stride=56) == 2 and f(a_stride=68) == 4 and f(i_stride=0) == 2
        assert f(X=None) == 1 and f(w=None) == 1 and f(X=FAKE + 4) == 4 and f(T=1 << 31) == 5
    assert lib.gdn_rec_fwd(None, *[None] * 9, 0, None) == 1
    assert fwd(B=0) == 0 and step(B=0) == 0 and step(offsets=FAKE) == 5 and step(h_out=None) == 1
    assert fwd(H=None) == 1 and fwd(h0=FAKE + 8) == 4 and fwd(I=FAKE + 2) == 4 and fwd(offsets=FAKE + 4) == 4
    assert fwd(ws=None) == 6 and fwd(nb=8) == 6 and fwd(ws=FAKE + 8) == 4
    assert bwd(ws=None) == 6 and bwd(nb=8) == 6 and bwd(ws=FAKE + 8) == 4
    assert bwd(dH=None) == 1 and bwd(I=FAKE) == 1 and bwd(dw=FAKE, decay=1) == 5
    assert fwd(T=(1 << 31) - 65, B=1 << 20) == 5 and bwd(T=(1 << 31) - 65, B=1 << 20) == 5
    q = lambda f, **kw: f(by(shape(**kw)))  # noqa: E731
    assert q(lib.gdn_rec_fwd_workspace_bytes, T=64) == 0 and q(lib.gdn_rec_fwd_workspace_bytes) > 0
    assert q(lib.gdn_rec_fwd_workspace_bytes, D=60) == 0 and q(lib.gdn_rec_bwd_workspace_bytes, B=0) == 0
    assert q(lib.gdn_rec_bwd_workspace_bytes) > q(lib.gdn_rec_fwd_workspace_bytes)
    assert tri.gdn_rec_fwd_workspace_bytes(2, 200, 64) > 0 and tri.gdn_rec_bwd_workspace_bytes(2, 200, 64, packed=True) > 0


def test_counts_past_32_bits():
    for f in (tri.gdn_rec_fwd_workspace_bytes, tri.gdn_rec_bwd_workspace_bytes):
        assert f((1 << 31) - 1, 1, 8) >= 0
        for B in (1 << 31, (1 << 32) + 1):
            with pytest.raises(ValueError):
                f(B, 200, 64)
