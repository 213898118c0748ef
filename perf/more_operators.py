"""The operators that stand beside linear attention in a mixed model and in front of it, timed and
compared: the gated linear recurrence of every channel (whole sequences, a training step, single
tokens), and the norm of queries and keys for each head with the position rotation, on one axis or
several (forward and backward).

``run`` computes them either in plain torch operations (``own`` false) or by the calls a user
makes of tri_inverse_amd (``own`` true), on the inputs that ``prepare`` makes.

Recurrence, per sequence and channel, s = sigmoid:

    log a_t = -w s(A_t) ("power"),  log s(A_t) ("sigmoid"),  A_t ("log")
    u_t = b_t s(I_t) X_t,  b_t = sqrt(1 - a_t^2) ("sqrt"),  1 - a_t ("linear"),  1 ("none")
    h_t = a_t h_{t-1} + u_t

X, A, I, H [B, T, D]; A and I may be parts of one wider projection; s(I) may be absent.  Packed
sequences lie one after another in T, with their offsets.  Backwards the gradients of X, A, I, w and
h_0 come from those of all h_t and of the last ones.

Queries and keys, from projection rows [B, T, heads, d] to [B, heads, T, d]: y = R(p) (x / n(x) * w)
with n(x) = sqrt(mean(x^2) + eps) ("rms") or sqrt(sum(x^2) + eps) ("l2"), and R the rotation of pair
i by p f_i, p the token's position on the pair's axis; pairs are (i, i + r/2) ("halves") or
(2i, 2i + 1) ("neighbours") of the first r values.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases -------------------------------------------------------------------------

def _rec(name, op, B, T, D, decay="power", norm="sqrt", gate=True, seqs=0, state=False, dtype="bf16"):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "decay": decay, "norm": norm, "gate": gate, "seqs": seqs,
            "state": state, "dtype": dtype}


def _qk(name, op, B, T, Hq, Hk, d, rot, norm="rms", pairs="halves", axes=1, far=0, extra=0, dtype="bf16"):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "norm": norm,
            "pairs": pairs, "axes": axes, "far": far, "extra": extra, "dtype": dtype}


def listed():
    return [
        # the prompt of four sequences, as wide as 16 heads of 128
        _rec("rec_fwd_prefill", "rec_fwd", 4, 8192, 2048),
        # one long document, few channels, the forget gate's own form: the work has to be split over the tokens
        _rec("rec_fwd_long", "rec_fwd", 1, 65536, 1024, decay="sigmoid", norm="linear", gate=False),
        # a serving step's prompts of very different lengths, packed, with the states they continue from
        _rec("rec_fwd_packed", "rec_fwd", 1, 11171, 1544, seqs=13, state=True, dtype="f32"),
        # short prompts: latency
        _rec("rec_fwd_short", "rec_fwd", 2, 77, 520, state=True),
        # a training step: forward and backward
        _rec("rec_train", "rec_train", 4, 4096, 2048),
        # the same for packed documents, log-decays as given, states carried
        _rec("rec_train_packed", "rec_train", 1, 5003, 776, decay="log", norm="none", gate=False, seqs=7, state=True,
             dtype="f32"),
        # one token of a batch of sequences
        _rec("rec_step_batch", "rec_step", 64, 1, 2048, state=True),
        # queries and keys of the prefill workload
        _qk("qk_fwd_prefill", "qk_fwd", 4, 8192, 16, 16, 128, 128),
        # one token of a batch of sequences, at far positions, shared keys
        _qk("qk_fwd_decode", "qk_fwd", 64, 1, 32, 16, 128, 64, far=1_000_000, extra=2048),
        # pictures and text in one row: positions in time, height and width, unit rows, odd length
        _qk("qk_fwd_axes", "qk_fwd", 3, 4099, 12, 4, 96, 64, norm="l2", pairs="neighbours", axes=3, dtype="f32"),
        # a training step's backward pass
        _qk("qk_bwd_train", "qk_bwd", 4, 4096, 16, 16, 128, 128),
        # the same for pictures, part of each head rotated, gates behind the keys in the projection
        _qk("qk_bwd_axes", "qk_bwd", 1, 1023, 8, 2, 256, 64, axes=2, extra=264),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rec_fwd", "rec_fwd", "rec_fwd", "rec_train", "rec_train", "rec_step", "qk_fwd", "qk_fwd", "qk_fwd",
                     "qk_bwd", "qk_bwd"])
    if op.startswith("rec"):
        D, dtype = 8 * _log(rng, 1, 512), rng.choice(["bf16", "bf16", "f32"])
        decay = rng.choice(["power", "power", "sigmoid", "log"])
        case = {"op": op, "decay": decay, "norm": rng.choice(["sqrt", "sqrt", "linear", "none"]),
                "gate": rng.random() < 0.6, "state": rng.random() < 0.5, "dtype": dtype, "seqs": 0, "D": D}
        if op == "rec_step":
            return {**case, "B": _log(rng, 1, 64), "T": rng.choice([1, 1, 1, 2, 5]), "state": True}
        values = (60_000_000 if op == "rec_fwd" else 30_000_000) // (2 if dtype == "f32" else 1)
        T = _log(rng, 1, min(65536, max(2, values // D)))
        seqs = rng.choice([0, 0, min(T, _log(rng, 2, 24))])
        B = 1 if seqs else max(1, min(_log(rng, 1, 16), values // (T * D)))
        return {**case, "B": B, "T": T, "seqs": seqs}
    d, dtype = rng.choice([32, 64, 96, 128, 128, 256]), rng.choice(["bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 4])
    values = (60_000_000 if op == "qk_fwd" else 30_000_000) // (2 if dtype == "f32" else 1)
    T = _log(rng, 1, values // ((Hq + Hk) * d))
    return {"op": op, "B": max(1, min(_log(rng, 1, 64), values // ((Hq + Hk) * d * T))), "T": T, "Hq": Hq, "Hk": Hk,
            "d": d, "rot": 8 * rng.randint(1, d // 8), "norm": rng.choice(["rms", "rms", "l2"]),
            "pairs": rng.choice(["halves", "neighbours"]), "axes": rng.choice([1, 1, 2, 3]),
            "far": rng.choice([0, 0, 30_000, 1_000_000]), "extra": rng.choice([0, 8, 264]), "dtype": dtype}


def _lengths(case):
    """The packed sequences' lengths: skewed, some of one token, some empty; the same for every seed."""
    rng = random.Random(case["T"] * 131 + case["seqs"])
    weight = [0.0 if i % 5 == 3 else math.exp(rng.uniform(0, 5)) for i in range(case["seqs"])]
    weight[0] = max(weight[0], 1.0)
    lens = [int(case["T"] * w / sum(weight)) for w in weight]
    lens[0] += case["T"] - sum(lens)
    return lens


# ---- inputs ----------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = dict(case)
    dt = DTYPE[case["dtype"]]

    def randn(*shape, dtype=torch.float32, by=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * by).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    B, T = case["B"], case["T"]
    if case["op"].startswith("rec"):
        D, n = case["D"], case["seqs"] or B
        st["X"] = randn(B, T, D, dtype=dt)
        # both gates are halves of one projection, where there are two
        gates = randn(B, T, 2 * D if case["gate"] else D)
        if case["decay"] == "log":  # horizons from some tokens to some hundreds
            gates[..., :D] = torch.nn.functional.logsigmoid(gates[..., :D] + 3.0)
        elif case["decay"] == "sigmoid":
            gates[..., :D] += 3.0
        gates = gates.to(dt)
        st["A"], st["I"] = gates[..., :D], gates[..., D:] if case["gate"] else None
        # a between 0.9 and 0.999 where the gate is fully open
        st["w"] = -torch.log(0.9 + 0.099 * rand(D)) if case["decay"] == "power" else None
        st["h0"] = randn(n, D) if case["state"] else None
        if case["op"] == "rec_train":
            st["dH"] = randn(B, T, D, dtype=dt)
            st["dh"] = randn(n, D) if case["state"] else None
        st["offsets"] = None
        st["spans"] = [(0, T)]
        if case["seqs"]:
            ends = torch.tensor([0] + _lengths(case)).cumsum(0)
            st["spans"] = list(zip(ends[:-1].tolist(), ends[1:].tolist()))
            st["offsets"] = ends.to(torch.int32).cuda()
        return st
    Hq, Hk, d, r = case["Hq"], case["Hk"], case["d"], case["rot"]
    rows = randn(B, T, (Hq + Hk) * d + case["extra"], dtype=dt)
    st["Q"], st["K"] = rows[..., :Hq * d].unflatten(-1, (Hq, d)), rows[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    st["wq"], st["wk"] = (1.0 + randn(d, by=0.1) for _ in range(2))
    st["freqs"] = torch.exp(torch.arange(r // 2, device="cuda", dtype=torch.float64) * (-2.0 / r * math.log(10000.0)))
    st["axis"] = None
    if case["axes"] > 1:  # a run of pairs for each axis
        st["axis"] = tuple(min(i * case["axes"] // (r // 2), case["axes"] - 1) for i in range(r // 2))
        size = 1 + max(1, int(T ** 0.5))
        t = torch.arange(T, device="cuda")
        grid = torch.stack([t // (size * size) if case["axes"] == 3 else t // size, t // size % size, t % size])
        st["positions"] = (grid[:case["axes"]] if case["axes"] == 3 else grid[::2])[:, None, :].expand(-1, B, -1)
    else:
        st["positions"] = torch.arange(T, device="cuda").expand(1, B, T)
    if case["far"]:  # each sequence has its own number of tokens behind it
        st["positions"] = st["positions"] + (rand(1, B, 1) * case["far"]).long()
    st["positions"] = st["positions"].to(torch.int32).contiguous()
    if case["axes"] == 1:
        st["positions"] = st["positions"][0]
    if case["op"] == "qk_bwd":
        st["dQ"], st["dK"] = randn(B, Hq, T, d, dtype=dt), randn(B, Hk, T, d, dtype=dt)
    return st


# ---- one pass --------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"rec_fwd": _plain_rec, "rec_step": _plain_rec, "rec_train": _plain_rec_train, "qk_fwd": _plain_qk,
            "qk_bwd": _plain_qk_bwd}[st["op"]](st)


def _run_own(st):
    import tri_inverse_amd as tri

    op = st["op"]
    if op.startswith("rec"):
        how = {"I": st["I"], "w": st["w"], "decay": st["decay"], "norm": st["norm"]}
        if op == "rec_step":
            return tri.gdn_rec_step(st["X"], st["A"], h=st["h0"], **how)
        how.update(h0=st["h0"], offsets=st["offsets"])
        H, h, states = tri.gdn_rec_fwd(st["X"], st["A"], want_states=op == "rec_train", **how)
        if op == "rec_fwd":
            return H, h
        return (H, h) + tri.gdn_rec_bwd(st["X"], st["A"], st["dH"], dh=st["dh"], states=states, **how)
    how = {"wq": st["wq"], "wk": st["wk"], "freqs": st["freqs"], "positions": st["positions"], "norm": st["norm"],
           "eps": EPS, "pairs": st["pairs"], "axis": st["axis"]}
    if op == "qk_fwd":
        return tri.gdn_qk_norm_fwd(st["Q"], st["K"], **how)
    return tri.gdn_qk_norm_bwd(st["dQ"], st["dK"], st["Q"], st["K"], **how)


# ---- the plain forms: the recurrence -----------------------------------------------------

def _gates(st):
    """log a, the input's factor and gate, in 32 bits."""
    A = st["A"].float()
    if st["decay"] == "power":
        g = -st["w"] * torch.sigmoid(A)
    else:
        g = torch.nn.functional.logsigmoid(A) if st["decay"] == "sigmoid" else A
    if st["norm"] == "sqrt":
        b = torch.sqrt(-torch.expm1(2 * g))
    else:
        b = -torch.expm1(g) if st["norm"] == "linear" else None
    return g, b, None if st["I"] is None else torch.sigmoid(st["I"].float())


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t over axis 1, h before the first zero: blocks of tokens side by side, token by
    token, then the blocks' ends one after another, then every block from its start."""
    B, T, D = a.shape
    C = max(1, int(T ** 0.5))
    N = (T + C - 1) // C
    pad = (0, 0, 0, N * C - T)
    a, u = (torch.nn.functional.pad(x, pad).view(B, N, C, D) for x in (a, u))
    P, h = torch.empty_like(a), torch.empty_like(a)
    P[:, :, 0], h[:, :, 0] = a[:, :, 0], u[:, :, 0]
    for c in range(1, C):
        P[:, :, c] = a[:, :, c] * P[:, :, c - 1]
        h[:, :, c] = a[:, :, c] * h[:, :, c - 1] + u[:, :, c]
    start = torch.zeros_like(h[:, :, 0])
    for n in range(1, N):
        start[:, n] = P[:, n - 1, -1] * start[:, n - 1] + h[:, n - 1, -1]
    return (h + P * start[:, :, None]).view(B, N * C, D)[:, :T]


def _ends(st):
    """Per sequence (row, first token, last token), and the sequences without tokens."""
    spans = [(0, s, e) for s, e in st["spans"]] if st["seqs"] else [(b, 0, st["T"]) for b in range(st["B"])]
    full = [i for i, (_, s, e) in enumerate(spans) if e > s]
    return (full, [spans[i][0] for i in full], [spans[i][1] for i in full], [spans[i][2] - 1 for i in full])


def _plain_states(st, g, b, s):
    """a (0 where a sequence starts), all states and the last ones, in 32 bits."""
    full, row, first, last = _ends(st)
    x = st["X"].float()
    u = x if s is None else s * x
    u = u if b is None else b * u
    a = torch.exp(g)
    if st["h0"] is not None:
        u = u.clone()
        u[row, first] += a[row, first] * st["h0"][full]
    a[row, first] = 0
    H = _scan(a, u)
    h = torch.zeros((st["seqs"] or st["B"], st["D"]), device="cuda") if st["h0"] is None else st["h0"].clone()
    h[full] = H[row, last]
    return a, H, h


def _plain_rec(st):
    _, H, h = _plain_states(st, *_gates(st))
    return H.to(st["X"].dtype), h


def _plain_rec_train(st):
    g, b, s = _gates(st)
    full, row, first, last = _ends(st)
    a, H, h = _plain_states(st, g, b, s)
    dH = st["dH"].float()
    if st["dh"] is not None:
        dH = dH.clone()
        dH[row, last] += st["dh"][full]
    later = torch.zeros_like(a)
    later[:, :-1] = a[:, 1:]
    G = _scan(later.flip(1), dH.flip(1)).flip(1)
    dh0 = None
    if st["h0"] is not None:
        dh0 = torch.zeros_like(st["h0"]) if st["dh"] is None else st["dh"].clone()
        dh0[full] = torch.exp(g[row, first]) * G[row, first]
    before = torch.zeros_like(H)
    before[:, 1:] = H[:, :-1]
    before[row, first] = 0 if st["h0"] is None else st["h0"][full]
    a = torch.exp(g)
    dg = G * a * before
    x = st["X"].float()
    z = x if s is None else s * x
    if b is not None:
        dg = dg - G * z * (a * a / b if st["norm"] == "sqrt" else a)
        G = G * b
    dI = None if s is None else (G * x * s * (1 - s)).to(st["X"].dtype)
    dX = (G if s is None else G * s).to(st["X"].dtype)
    dw = None
    if st["decay"] != "log":
        r = torch.sigmoid(st["A"].float())
        if st["decay"] == "power":
            dw = -(r * dg).sum((0, 1), dtype=torch.float64).float()
            dg = -st["w"] * dg * r * (1 - r)
        else:
            dg = dg * (1 - r)
    return H.to(st["X"].dtype), h, dX, dg.to(st["X"].dtype), dI, dw, dh0


# ---- the plain forms: queries and keys ---------------------------------------------------

def _angles(st):
    """cos and sin [B, T, 1, r / 2]: in 64 bits, where far positions need them."""
    p = st["positions"].double()
    p = p[..., None] if st["axis"] is None else p[list(st["axis"])].permute(1, 2, 0)
    phase = (p * st["freqs"])[:, :, None]
    return phase.cos().float(), phase.sin().float()


def _turn(x, cos, sin, st):
    r = st["rot"]
    y = x.clone()
    at = (slice(0, r // 2), slice(r // 2, r)) if st["pairs"] == "halves" else (slice(0, r, 2), slice(1, r, 2))
    y[..., at[0]] = x[..., at[0]] * cos - x[..., at[1]] * sin
    y[..., at[1]] = x[..., at[1]] * cos + x[..., at[0]] * sin
    return y


def _rstd(x, st):
    sq = x.square()
    return torch.rsqrt((sq.mean(-1, keepdim=True) if st["norm"] == "rms" else sq.sum(-1, keepdim=True)) + EPS)


def _plain_qk(st):
    cos, sin = _angles(st)
    out = []
    for x, w in ((st["Q"], st["wq"]), (st["K"], st["wk"])):
        y = x.float()
        y = _turn(y * _rstd(y, st) * w, cos, sin, st)
        out.append(y.to(x.dtype).transpose(1, 2).contiguous())
    return tuple(out)


def _plain_qk_bwd(st):
    cos, sin = _angles(st)
    grads, weights = [], []
    for x, w, dy in ((st["Q"], st["wq"], st["dQ"]), (st["K"], st["wk"], st["dK"])):
        y = x.float()
        rstd = _rstd(y, st)
        n = y * rstd
        dn = _turn(dy.float().transpose(1, 2), cos, -sin, st)
        weights.append((dn * n).sum((0, 1, 2), dtype=torch.float64).float())
        dn = dn * w
        along = (dn * n).mean(-1, keepdim=True) if st["norm"] == "rms" else (dn * n).sum(-1, keepdim=True)
        grads.append((rstd * (dn - n * along)).to(x.dtype))
    return tuple(grads + weights)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("rec"):
        n = case["B"] * case["T"] * case["D"]
        state = 4 * (case["seqs"] or case["B"]) * case["D"]
        fwd = (3 + case["gate"]) * n * size + state * (1 + case["state"])
        if case["op"] != "rec_train":
            return {"bytes": fwd, "flops": 20.0 * n}
        return {"bytes": fwd + (5 + 2 * case["gate"]) * n * size + 3 * state * case["state"], "flops": 70.0 * n}
    n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
    back = case["op"] == "qk_bwd"
    return {"bytes": (3 if back else 2) * n * size + 4 * case["axes"] * case["B"] * case["T"],
            "flops": (20.0 if back else 10.0) * n}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("rec"):
        return _exact_rec(st)
    return _exact_qk(st)


def _exact_rec(st):
    X, A = st["X"].double(), st["A"].double()
    sg = lambda t: 1 / (1 + torch.exp(-t))  # noqa: E731
    if st["decay"] == "power":
        a = torch.exp(-st["w"].double() * sg(A))
    else:
        a = sg(A) if st["decay"] == "sigmoid" else torch.exp(A)
    i = torch.ones_like(X) if st["I"] is None else sg(st["I"].double())
    b = {"sqrt": lambda: ((1 - a) * (1 + a)).sqrt(), "linear": lambda: 1 - a, "none": lambda: torch.ones_like(a)}[st["norm"]]()
    u = b * i * X
    H = torch.empty_like(X)
    before = torch.empty_like(X) if st["op"] == "rec_train" else None
    n = st["seqs"] or st["B"]
    given = torch.zeros((n, st["D"]), device="cuda", dtype=torch.float64) if st["h0"] is None else st["h0"].double()
    last = []
    for k, (s, e) in enumerate(st["spans"]):
        h = given[k:k + 1] if st["seqs"] else given
        for t in range(s, e):
            if before is not None:
                before[:, t] = h
            h = torch.addcmul(u[:, t], a[:, t], h)
            H[:, t] = h
        last.append(h)
    last = torch.cat(last)
    if st["op"] != "rec_train":
        return H, last
    dH = st["dH"].double()
    G = torch.empty_like(X)
    dgiven = torch.zeros_like(given) if st["dh"] is None else st["dh"].double()
    first = []
    for k, (s, e) in enumerate(st["spans"]):
        d = dgiven[k:k + 1] if st["seqs"] else dgiven
        for t in reversed(range(s, e)):
            d = d + dH[:, t]
            G[:, t] = d
            d = d * a[:, t]
        first.append(d)
    # by the chain rule: a enters through the state and through b
    db = {"sqrt": lambda: -a / b, "linear": lambda: -torch.ones_like(a), "none": lambda: torch.zeros_like(a)}[st["norm"]]()
    da = G * (before + i * X * db)
    dw = None
    if st["decay"] == "power":
        r = sg(A)
        dA = da * a * -st["w"].double() * r * (1 - r)
        dw = (da * a * -r).sum((0, 1))
    else:
        dA = da * a * (1 - a) if st["decay"] == "sigmoid" else da * a
    dI = None if st["I"] is None else G * b * X * i * (1 - i)
    return H, last, G * b * i, dA, dI, dw, None if st["h0"] is None else torch.cat(first)


def _exact_qk(st):
    p, r = st["positions"].double(), st["rot"]
    p = p[None] if st["axis"] is None else p
    axis = [0] * (r // 2) if st["axis"] is None else st["axis"]
    phase = torch.stack([p[axis[i]] * st["freqs"][i] for i in range(r // 2)], -1)[:, :, None]
    unit = torch.polar(torch.ones_like(phase), phase)

    def spin(x, by):
        z = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if st["pairs"] == "halves" else x[..., :r].unflatten(-1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
        z = z.transpose(-1, -2).flatten(-2) if st["pairs"] == "halves" else z.flatten(-2)
        return torch.cat([z, x[..., r:]], -1)

    out, sums = [], []
    for name in ("Q", "K"):
        x, w = st[name].double(), st["w" + name.lower()].double()
        of = x.shape[-1] if st["norm"] == "rms" else 1
        size = ((x * x).sum(-1, keepdim=True) / of + EPS).sqrt()
        if st["op"] == "qk_fwd":
            out.append(spin(x / size * w, unit).transpose(1, 2))
            continue
        dn = spin(st["d" + name].double().transpose(1, 2), unit.conj())
        sums.append((dn * x / size).sum((0, 1, 2)))
        dn = dn * w
        out.append(dn / size - x * (dn * x).sum(-1, keepdim=True) / (of * size ** 3))
    return tuple(out + sums)
