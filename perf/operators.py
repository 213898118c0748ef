"""The operators beside the gated delta rule that are timed and compared: linear attention
with a decay for each head (chunk-wise forward and backward, single tokens) and the norms
of the block around it (the gated norm of the head outputs, the residual sum with its norms).

``run`` computes them either in plain torch operations (``own`` false) or by the calls a
user makes of tri_inverse_amd (``own`` true), on the inputs that ``prepare`` makes.

Linear attention, per sequence and value head, g the log-decays (<= 0), tokens in order:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t

Q, K [B, H_qk, T, d_k] are shared by H / H_qk value heads each; V [B, H, T, d_v]; g is
[B, H, T] (a decay for each token) or [H] (one for each head).  Packed sequences lie one
after another in T, with their offsets.

Norms, rms(x) = x / sqrt(mean(x^2) + eps) over the last axis:

    gated norm      Y[b, t, h] = rms(O[b, h, t]) * w * silu(Z[b, t, h])
    residual norm   R = X + alpha * s * (rms(Y) * w_post),   N = rms(R) * w_pre
"""
import math
import random

import torch

own = False

C = 64  # tokens of a chunk in the plain chunk-wise form
EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases -------------------------------------------------------------------------

def _lin(name, op, B, H, Hk, T, dk, dv, decay="token", seqs=0, state=False):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "T": T, "dk": dk, "dv": dv, "decay": decay,
            "seqs": seqs, "state": state}


def listed():
    return [
        # the prompt of four sequences: the prefill workload of the repository's benchmark
        _lin("lin_fwd_prefill", "lin_fwd", 4, 16, 16, 8192, 128, 128),
        # one long prompt, few heads, one decay for each head: the work has to be split over the tokens
        _lin("lin_fwd_long", "lin_fwd", 1, 8, 4, 32768, 128, 128, decay="head"),
        # a serving step's prompts of very different lengths, packed, with the states they continue from
        _lin("lin_fwd_packed", "lin_fwd", 1, 16, 4, 11171, 128, 256, seqs=13, state=True),
        # short prompts: latency
        _lin("lin_fwd_short", "lin_fwd", 2, 4, 4, 77, 64, 64, state=True),
        # a training step's backward pass
        _lin("lin_bwd_train", "lin_bwd", 4, 16, 16, 4096, 128, 128),
        # the same for packed documents, grouped heads and one decay for each head, states carried
        _lin("lin_bwd_packed", "lin_bwd", 1, 12, 4, 5003, 64, 128, decay="head", seqs=7, state=True),
        # one decode step of a batch of sequences, and of a single one
        {"name": "lin_decode_batch", "op": "lin_decode", "B": 64, "H": 32, "Hk": 16, "n": 1, "dk": 128, "dv": 128,
         "dtype": "bf16", "decay": "token"},
        {"name": "lin_decode_one", "op": "lin_decode", "B": 1, "H": 32, "Hk": 32, "n": 1, "dk": 128, "dv": 128,
         "dtype": "f32", "decay": "head"},
        # the gated norm after the prefill workload, its gate a part of a wider projection
        {"name": "gate_norm_prefill", "op": "gate_fwd", "B": 4, "H": 16, "T": 8192, "d": 128, "extra": 512,
         "dtype": "bf16"},
        # its backward pass in training, at an odd length
        {"name": "gate_norm_train", "op": "gate_bwd", "B": 3, "H": 16, "T": 4099, "d": 128, "extra": 0, "dtype": "bf16"},
        # the residual stream of a decode step
        {"name": "residual_norm_decode", "op": "res_fwd", "rows": 64, "D": 2048, "x": "f32", "y": "bf16", "post": True,
         "scale": True},
        # its backward pass in training
        {"name": "residual_norm_train", "op": "res_bwd", "rows": 16384, "D": 4096, "x": "f32", "y": "bf16", "post": True,
         "scale": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_fwd", "lin_fwd", "lin_bwd", "lin_bwd", "lin_decode", "lin_decode", "gate_fwd",
                     "gate_bwd", "res_fwd", "res_bwd"])
    if op in ("lin_fwd", "lin_bwd"):
        Hk, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4])
        H = Hk * group
        dk = rng.choice([64, 128])
        dv = rng.choice([64, 128]) if op == "lin_bwd" else rng.choice([32, 64, 96, 128, 128, 256])
        most, values = (32768, 32_000_000) if op == "lin_fwd" else (16384, 12_000_000)
        tokens = max(2, min(most, values // (H * max(dk, dv))))
        T = _log(rng, 1, tokens)
        seqs = rng.choice([0, 0, min(T, _log(rng, 2, 24))])
        B = 1 if seqs else max(1, min(_log(rng, 1, 16), tokens // T))
        return {"op": op, "B": B, "H": H, "Hk": Hk, "T": T, "dk": dk, "dv": dv, "decay": rng.choice(["token", "head"]),
                "seqs": seqs, "state": rng.random() < 0.5}
    if op == "lin_decode":
        Hk, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2])
        return {"op": op, "B": _log(rng, 1, 64), "H": Hk * group, "Hk": Hk, "n": rng.choice([1, 1, 1, 2, 5]),
                "dk": rng.choice([64, 128]), "dv": rng.choice([32, 64, 96, 128, 128]),
                "dtype": rng.choice(["bf16", "f32"]), "decay": rng.choice(["token", "head"])}
    if op in ("gate_fwd", "gate_bwd"):
        H, d = rng.choice([1, 3, 4, 8, 16]), rng.choice([32, 64, 96, 128, 128, 256])
        tokens = (30_000_000 if op == "gate_fwd" else 12_000_000) // (H * d)
        T = _log(rng, 1, tokens)
        return {"op": op, "B": max(1, min(_log(rng, 1, 8), tokens // T)), "H": H, "T": T, "d": d,
                "extra": rng.choice([0, 8, 264]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    D = 8 * _log(rng, 8, 1024)
    return {"op": op, "rows": _log(rng, 1, 40_000_000 // D), "D": D, "x": rng.choice(["f32", "bf16"]), "y": "bf16",
            "post": rng.random() < 0.5, "scale": rng.random() < 0.5}


def _lengths(case):
    """The packed sequences' lengths: skewed, some of one token, some empty; the same for every seed."""
    rng = random.Random(case["T"] * 131 + case["seqs"])
    weight = [0.0 if i % 5 == 3 else math.exp(rng.uniform(0, 5)) for i in range(case["seqs"])]
    weight[0] = max(weight[0], 1.0)
    lens = [int(case["T"] * w / sum(weight)) for w in weight]
    lens[0] += case["T"] - sum(lens)
    return lens


# ---- inputs ----------------------------------------------------------------------------

def _unit(shape, gen, dtype):
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _decay(case, T, gen):
    if case["decay"] == "head":  # horizons spread over the heads, from about 30 tokens to some thousands
        h = torch.arange(case["H"], device="cuda", dtype=torch.float64)
        u = torch.rand(case["H"], generator=gen, device="cuda", dtype=torch.float64)
        return torch.log1p(-torch.exp2(-5.0 - 7.0 * (h + u) / case["H"])).float()
    x = torch.randn((case["B"], case["H"], T), generator=gen, device="cuda") + 2.0
    return torch.nn.functional.logsigmoid(x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = dict(case)

    def randn(*shape, dtype=torch.float32, by=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * by).to(dtype)

    op = case["op"]
    if op in ("lin_fwd", "lin_bwd"):
        B, H, T, dk, dv = case["B"], case["H"], case["T"], case["dk"], case["dv"]
        bf = torch.bfloat16
        st["Q"], st["K"] = _unit((B, case["Hk"], T, dk), gen, bf), _unit((B, case["Hk"], T, dk), gen, bf)
        st["V"] = randn(B, H, T, dv, dtype=bf)
        st["g"] = _decay(case, T, gen)
        n = case["seqs"] or B
        st["S0"] = randn(n, H, dk, dv, by=0.5) if case["state"] else None
        if op == "lin_bwd":
            st["dO"] = randn(B, H, T, dv, dtype=bf)
            st["dS"] = randn(n, H, dk, dv, by=0.5) if case["state"] else None
        lens = _lengths(case) if case["seqs"] else None
        st["offsets"] = None
        if lens:
            ends = torch.tensor(lens).cumsum(0)
            st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).cuda()
        st["plan"] = _plan(lens or [T])
    elif op == "lin_decode":
        B, H, n, dk, dv, dt = case["B"], case["H"], case["n"], case["dk"], case["dv"], DTYPE[case["dtype"]]
        st["Q"], st["K"] = _unit((B, case["Hk"], n, dk), gen, dt), _unit((B, case["Hk"], n, dk), gen, dt)
        st["V"] = randn(B, H, n, dv, dtype=dt)
        st["g"] = _decay(case, n, gen)
        st["S0"] = randn(B, H, dk, dv, by=0.5)
    elif op in ("gate_fwd", "gate_bwd"):
        B, H, T, d, dt = case["B"], case["H"], case["T"], case["d"], DTYPE[case["dtype"]]
        st["O"] = randn(B, H, T, d, dtype=dt, by=0.3)
        st["Z"] = randn(B, T, H * d + case["extra"], dtype=dt)[..., :H * d].unflatten(-1, (H, d))
        st["w"] = 1.0 + randn(d, by=0.1)
        if op == "gate_bwd":
            st["dY"] = randn(B, T, H, d, dtype=dt)
    else:
        rows, D, xt, yt = case["rows"], case["D"], DTYPE[case["x"]], DTYPE[case["y"]]
        st["X"], st["Y"] = randn(rows, D, dtype=xt, by=2.0), randn(rows, D, dtype=yt, by=0.7)
        st["w_post"] = 1.0 + randn(D, by=0.1) if case["post"] else None
        st["s"] = 0.5 + randn(D, by=0.1) if case["scale"] else None
        st["w_pre"] = 1.0 + randn(D, by=0.1)
        st["alpha"] = 0.75
        if op == "res_bwd":  # X stands for the sum R that the forward pass wrote
            st["dN"], st["dR"] = randn(rows, D, dtype=yt), randn(rows, D, dtype=xt)
    return st


def _plan(lens):
    """Where each chunk's tokens lie: rows [NC, C] (len(all) for a row past a sequence's end), the chunks' sequences."""
    rows, seq, at = [], [], 0
    total = sum(lens)
    for i, n in enumerate(lens):
        for c in range(0, n, C):
            rows.append([at + c + r if c + r < n else total for r in range(C)])
            seq.append(i)
        at += n
    if not rows:
        rows, seq = [[total] * C], [0]
    return {"rows": torch.tensor(rows).cuda(), "seq": torch.tensor(seq).cuda(), "n": len(lens)}


# ---- one pass --------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "lin_fwd":
        return _plain_fwd(st)
    if op == "lin_bwd":
        return _plain_bwd(st)
    if op == "lin_decode":
        return _plain_decode(st)
    if op == "gate_fwd":
        return _plain_gate(st)
    if op == "gate_bwd":
        return _plain_gate_bwd(st)
    if op == "res_fwd":
        return _plain_residual(st)
    return _plain_residual_bwd(st)


def _run_own(st):
    import tri_inverse_amd as tri

    op = st["op"]
    if op == "lin_fwd":
        return tri.gdn_lin_chunk_fwd(st["Q"], st["K"], st["V"], st["g"], S0=st["S0"], offsets=st["offsets"])
    if op == "lin_bwd":
        return tri.gdn_lin_chunk_bwd(st["Q"], st["K"], st["V"], st["g"], st["dO"], S0=st["S0"], dS=st["dS"],
                                     offsets=st["offsets"])
    if op == "lin_decode":
        return tri.gdn_lin_decode(st["Q"], st["K"], st["V"], st["g"], S=st["S0"], o_dtype=st["Q"].dtype)
    if op == "gate_fwd":
        return tri.gdn_gate_norm_fwd(st["O"], st["Z"], st["w"], eps=EPS)
    if op == "gate_bwd":
        return tri.gdn_gate_norm_bwd(st["dY"], st["O"], st["Z"], st["w"], eps=EPS)
    if op == "res_fwd":
        return tri.gdn_residual_norm_fwd(st["X"], st["Y"], w_post=st["w_post"], s=st["s"], alpha=st["alpha"],
                                         w_pre=st["w_pre"], eps=EPS)
    return tri.gdn_residual_norm_bwd(st["dN"], st["dR"], st["X"], st["Y"], w_post=st["w_post"], s=st["s"],
                                     alpha=st["alpha"], w_pre=st["w_pre"], eps=EPS)


# ---- the plain forms: linear attention ---------------------------------------------------

def _chunks(x, plan, H):
    """[B, h, T, d] as [B H, NC, C, d] in 32 bits, zero rows past a sequence's end."""
    x = x.float().repeat_interleave(H // x.shape[1], dim=1).flatten(0, 1)
    return torch.nn.functional.pad(x, (0, 0, 0, 1))[:, plan["rows"]]


def _decays(st):
    """In-chunk sums G and the chunks' decays, in 64 bits: E[c, c'] from the end of chunk c' to the start of
    chunk c, and per sequence from its start to each chunk's start and from each chunk's end to its end."""
    B, H, T, plan = st["B"], st["H"], st["T"], st["plan"]
    g = st["g"].double()
    g = (g.view(1, H, 1).expand(B, H, T) if g.dim() == 1 else g).flatten(0, 1)
    g = torch.nn.functional.pad(g, (0, 1))[:, plan["rows"]]
    G = g.cumsum(-1)
    total = G[..., -1]
    A = total.cumsum(-1)
    Ax = A - total
    seq, c = plan["seq"], torch.arange(plan["seq"].numel(), device="cuda")
    before = (c[:, None] > c[None, :]) & (seq[:, None] == seq[None, :])
    E = torch.exp(torch.where(before, Ax[:, :, None] - A[:, None, :], -math.inf)).float()
    inside = torch.arange(plan["n"], device="cuda")[:, None] == seq[None, :]
    sums = torch.where(inside, total[:, None, :], 0.0)
    start = torch.exp(torch.where(inside, sums.cumsum(-1) - sums, -math.inf)).float()
    rest = sums.flip(-1).cumsum(-1).flip(-1) - sums
    end = torch.exp(torch.where(inside, rest, -math.inf)).float()
    w = G[..., :, None] - G[..., None, :]
    tri = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    w = torch.exp(torch.where(tri, w, -math.inf)).float()
    return {"eG": G.exp().float()[..., None], "eR": (total[..., None] - G).exp().float()[..., None], "w": w, "E": E,
            "start": start, "end": end, "whole": sums.sum(-1).exp().float(), "total": total.exp().float()}


def _states(E, X, weight, first):
    """sum over c' of E[c, c'] X[c'], and the states given per sequence brought to each chunk."""
    S = (E @ X.flatten(2)).view_as(X)
    if first is not None:
        S = S + (weight.transpose(1, 2) @ first.flatten(2)).view_as(X)
    return S


def _carried(weight, X, whole, first):
    S = (weight @ X.flatten(2)).unflatten(-1, X.shape[2:])
    return S if first is None else S + whole[..., None, None] * first


def _rows_back(x, st, d):
    """[B H, NC, C, d] back to [B, H, T, d]."""
    out = torch.zeros((x.shape[0], st["T"] + 1, d), device="cuda", dtype=x.dtype)
    out[:, st["plan"]["rows"].flatten()] = x.reshape(x.shape[0], -1, d)
    return out[:, :st["T"]].reshape(st["B"], st["H"], st["T"], d)


def _by_head(S, st):
    """[sequences, H, dk, dv] as [B H, sequences of a row, dk, dv]."""
    if S is None:
        return None
    return S.transpose(0, 1) if st["seqs"] else S.flatten(0, 1)[:, None]


def _by_seq(S, st):
    return (S.transpose(0, 1) if st["seqs"] else S[:, 0].unflatten(0, (st["B"], st["H"]))).contiguous()


def _plain_fwd(st):
    H, plan, scale = st["H"], st["plan"], st["dk"] ** -0.5
    q, k, v = (_chunks(st[n], plan, H) for n in ("Q", "K", "V"))
    d = _decays(st)
    S0 = _by_head(st["S0"], st)
    KV = (k * d["eR"]).transpose(-1, -2) @ v
    S = _states(d["E"], KV, d["start"], S0)
    o = scale * (((q @ k.transpose(-1, -2)) * d["w"]) @ v + (q * d["eG"]) @ S)
    S_out = _carried(d["end"], KV, d["whole"], S0)
    return _rows_back(o, st, st["dv"]).to(torch.bfloat16), _by_seq(S_out, st)


def _plain_bwd(st):
    H, Hk, plan, scale = st["H"], st["Hk"], st["plan"], st["dk"] ** -0.5
    q, k, v, do = (_chunks(st[n], plan, H) for n in ("Q", "K", "V", "dO"))
    d = _decays(st)
    S0, dS = _by_head(st["S0"], st), _by_head(st["dS"], st)
    KV = (k * d["eR"]).transpose(-1, -2) @ v
    QD = scale * ((q * d["eG"]).transpose(-1, -2) @ do)
    S = _states(d["E"], KV, d["start"], S0)
    D = _states(d["E"].transpose(1, 2), QD, d["end"], dS)
    P = scale * (q @ k.transpose(-1, -2)) * d["w"]
    dP = scale * (do @ v.transpose(-1, -2)) * d["w"]
    dq = dP @ k + scale * d["eG"] * (do @ S.transpose(-1, -2))
    dk = dP.transpose(-1, -2) @ q + d["eR"] * (v @ D.transpose(-1, -2))
    dv = P.transpose(-1, -2) @ do + d["eR"] * (k @ D)
    r = ((q * dq).sum(-1) - (k * dk).sum(-1)).double()
    at_end = (D * (d["total"][..., None, None] * S + KV)).flatten(2).double().sum(-1)
    dg = r.flip(-1).cumsum(-1).flip(-1) + at_end[..., None]
    dg = _rows_back(dg[..., None], st, 1)[..., 0]
    dg = dg.sum((0, 2)) if st["g"].dim() == 1 else dg
    shared = lambda x: _rows_back(x, st, st["dk"]).unflatten(1, (Hk, H // Hk)).sum(2).to(torch.bfloat16)  # noqa: E731
    dS0 = None if S0 is None else _by_seq(_carried(d["start"], QD, d["whole"], dS), st)
    return shared(dq), shared(dk), _rows_back(dv, st, st["dv"]).to(torch.bfloat16), dg.float(), dS0


def _plain_decode(st):
    H, n, scale = st["H"], st["n"], st["dk"] ** -0.5
    q, k = (st[x].float().repeat_interleave(H // st["Hk"], dim=1) for x in ("Q", "K"))
    v, g = st["V"].float(), st["g"].double()
    G = (g.view(1, H, 1).expand(st["B"], H, n) if g.dim() == 1 else g).cumsum(-1)
    tri = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    w = torch.exp(torch.where(tri, G[..., :, None] - G[..., None, :], -math.inf)).float()
    eG, eR = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    o = scale * (((q @ k.transpose(-1, -2)) * w) @ v + (q * eG) @ st["S0"])
    S = eG[..., -1:, :] * st["S0"] + (k * eR).transpose(-1, -2) @ v
    return o.to(st["Q"].dtype), S


# ---- the plain forms: norms --------------------------------------------------------------

def _plain_gate(st):
    o, z = st["O"].float().transpose(1, 2), st["Z"].float()
    n = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
    return (n * st["w"] * (z * torch.sigmoid(z))).to(st["O"].dtype)


def _plain_gate_bwd(st):
    o, z, dy, w = st["O"].float().transpose(1, 2), st["Z"].float(), st["dY"].float(), st["w"]
    rstd = torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
    n, sg = o * rstd, torch.sigmoid(z)
    dz = dy * n * w * (sg * (1 + z * (1 - sg)))
    dn = dy * (z * sg)
    dw = (dn * n).sum((0, 1, 2), dtype=torch.float64).float()
    dn = dn * w
    do = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    return do.to(st["O"].dtype).transpose(1, 2).contiguous(), dz.to(st["Z"].dtype), dw


def _plain_residual(st):
    y = st["Y"].float()
    if st["w_post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * st["w_post"]
    if st["s"] is not None:
        y = y * st["s"]
    r = st["X"].float() + st["alpha"] * y
    n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * st["w_pre"]
    return r.to(st["X"].dtype), n.to(st["Y"].dtype)


def _norm_bwd(dy, x, w):
    """Gradients of rms(x) * w: with respect to x, and to w."""
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * rstd
    dw = (dy * n).sum(0, dtype=torch.float64).float()
    dy = dy * w
    return rstd * (dy - n * (dy * n).mean(-1, keepdim=True)), dw


def _plain_residual_bwd(st):
    r, y = st["X"].float(), st["Y"].float()
    dr, dw_pre = _norm_bwd(st["dN"].float(), r, st["w_pre"])
    dr = dr + st["dR"].float()
    dy, dw_post, ds = st["alpha"] * dr, None, None
    if st["s"] is not None:
        z = y
        if st["w_post"] is not None:
            z = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * st["w_post"]
        ds = (dy * z).sum(0, dtype=torch.float64).float()
        dy = dy * st["s"]
    if st["w_post"] is not None:
        dy, dw_post = _norm_bwd(dy, y, st["w_post"])
    return dr.to(st["X"].dtype), dy.to(st["Y"].dtype), dw_pre, dw_post, ds


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("lin_fwd", "lin_bwd", "lin_decode"):
        B, H, Hk, T, dk, dv = case["B"], case["H"], case["Hk"], case.get("T") or case.get("n"), case["dk"], case["dv"]
        size = 4 if case.get("dtype") == "f32" else 2
        qk, v, state = B * Hk * T * dk * size, B * H * T * dv * size, (case.get("seqs") or B) * H * dk * dv * 4
        g = 4 * (H if case["decay"] == "head" else B * H * T)
        if op == "lin_fwd":  # S in where it continues, S out; the products of the recurrence
            return {"bytes": 2 * qk + 2 * v + g + state * (1 + case["state"]), "flops": 4.0 * B * H * T * dk * dv}
        if op == "lin_decode":
            return {"bytes": 2 * qk + 2 * v + g + 2 * state, "flops": 4.0 * B * H * T * dk * dv}
        return {"bytes": 4 * qk + 3 * v + 2 * g + (3 * state if case["state"] else 0),
                "flops": 10.0 * B * H * T * dk * dv}
    if op in ("gate_fwd", "gate_bwd"):
        n, size = case["B"] * case["H"] * case["T"] * case["d"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": (3 if op == "gate_fwd" else 5) * n * size, "flops": (8.0 if op == "gate_fwd" else 20.0) * n}
    n, xs, ys = case["rows"] * case["D"], 4 if case["x"] == "f32" else 2, 4 if case["y"] == "f32" else 2
    if op == "res_fwd":
        return {"bytes": n * (2 * xs + 2 * ys), "flops": 10.0 * n}
    return {"bytes": n * (3 * xs + 3 * ys), "flops": 25.0 * n}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("lin_fwd", "lin_bwd"):
        return _exact_lin(st)
    if op == "lin_decode":
        o, S, _ = _recurrence(st, st["S0"].double(), slice(0, st["n"]), st["S0"].double())
        return o, S
    if op in ("gate_fwd", "gate_bwd"):
        return _exact_gate(st)
    return _exact_residual(st)


def _token(st, name, t):
    x = st[name][:, :, t].double()
    return x.repeat_interleave(st["H"] // x.shape[1], dim=1)


def _a(st, t):
    g = st["g"].double()
    return torch.exp(g.view(1, -1) if g.dim() == 1 else g[:, :, t])[..., None, None]


def _recurrence(st, S, tokens, like, keep=False):
    """The recurrence token by token: outputs, the last state, with `keep` the states before each token."""
    out, states = [], []
    for t in range(tokens.start, tokens.stop):
        if keep:
            states.append(S)
        S = _a(st, t) * S + _token(st, "K", t)[..., :, None] * _token(st, "V", t)[..., None, :]
        if not keep:
            out.append(st["dk"] ** -0.5 * (_token(st, "Q", t)[..., None, :] @ S)[..., 0, :])
    o = torch.stack(out, 2) if out else like.new_zeros((S.shape[0], S.shape[1], 0, S.shape[3]))
    return o, S, states


def _exact_lin(st):
    H, dk, dv, T = st["H"], st["dk"], st["dv"], st["T"]
    lens = _lengths(st) if st["seqs"] else [T]
    zeros = torch.zeros((st["B"], H, dk, dv), device="cuda", dtype=torch.float64)

    def given(name, i):
        S = st[name]
        return zeros if S is None else (S[i:i + 1] if st["seqs"] else S).double()

    at, parts, last = 0, [], []
    for i, n in enumerate(lens):
        if st["op"] == "lin_fwd":
            o, S, _ = _recurrence(st, given("S0", i), slice(at, at + n), zeros)
            parts.append((o,))
            last.append(S)
        else:
            p, D = _exact_grads(st, given("S0", i), given("dS", i), at, n, zeros)
            parts.append(p)
            last.append(D)
        at += n
    whole = [torch.cat(x, 2) for x in zip(*parts)]
    if st["op"] == "lin_fwd":
        return whole[0], torch.cat(last)
    dq, dk_, dv_, dg = whole
    shared = lambda x: x.unflatten(1, (st["Hk"], H // st["Hk"])).sum(2)  # noqa: E731
    dg = dg.sum((0, 2)) if st["g"].dim() == 1 else dg
    return shared(dq), shared(dk_), dv_, dg, None if st["S0"] is None else torch.cat(last)


def _exact_grads(st, S0, D, at, n, zeros):
    """Gradients of one sequence, from its last token to its first: D the gradient of the state after the token."""
    scale, block = st["dk"] ** -0.5, 64
    starts, S = [], S0
    for c in range(0, n, block):
        starts.append(S)
        S = _recurrence(st, S, slice(at + c, at + min(c + block, n)), zeros, keep=True)[1]
    out = []
    for c in reversed(range(0, n, block)):
        stop = min(c + block, n)
        _, _, before = _recurrence(st, starts[c // block], slice(at + c, at + stop), zeros, keep=True)
        for t in reversed(range(c, stop)):
            q, k, v, do, a = (*(_token(st, x, at + t) for x in ("Q", "K", "V", "dO")), _a(st, at + t))
            old = a * before[t - c]
            D = D + scale * q[..., :, None] * do[..., None, :]
            dq = scale * ((old + k[..., :, None] * v[..., None, :]) @ do[..., :, None])[..., 0]
            out.append((dq, (D @ v[..., :, None])[..., 0], (k[..., None, :] @ D)[..., 0, :], (D * old).sum((-1, -2))))
            D = a * D
    if not out:
        e = lambda d: zeros.new_zeros((zeros.shape[0], zeros.shape[1], 0, d))  # noqa: E731
        return (e(st["dk"]), e(st["dk"]), e(st["dv"]), e(1)[..., 0]), D
    return tuple(torch.stack(x[::-1], 2) for x in zip(*out)), D


def _exact_gate(st):
    o, z, w = st["O"].double().permute(0, 2, 1, 3), st["Z"].double(), st["w"].double()
    ms = (o * o).sum(-1, keepdim=True) / o.shape[-1] + EPS
    e = torch.exp(-z)
    if st["op"] == "gate_fwd":
        return o / ms.sqrt() * w * z / (1 + e)
    dy = st["dY"].double()
    dz = dy * w * o / ms.sqrt() * ((1 + e + z * e) / (1 + e) ** 2)
    u = dy * z / (1 + e)
    dw = (u * o / ms.sqrt()).sum((0, 1, 2))
    u = u * w
    do = u / ms.sqrt() - o * (u * o).sum(-1, keepdim=True) / (o.shape[-1] * ms ** 1.5)
    return do.permute(0, 2, 1, 3), dz, dw


def _exact_residual(st):
    x, y = st["X"].double(), st["Y"].double()
    D = x.shape[-1]
    wy = st["alpha"] * (1.0 if st["s"] is None else st["s"].double())
    wp = None if st["w_post"] is None else st["w_post"].double()
    my = (y * y).sum(-1, keepdim=True) / D + EPS
    z = y if wp is None else y / my.sqrt() * wp
    w = st["w_pre"].double()
    if st["op"] == "res_fwd":
        r = x + wy * z
        return r, r / ((r * r).sum(-1, keepdim=True) / D + EPS).sqrt() * w
    dn, mr = st["dN"].double(), (x * x).sum(-1, keepdim=True) / D + EPS
    dr = st["dR"].double() + dn * w / mr.sqrt() - x * (dn * w * x).sum(-1, keepdim=True) / (D * mr ** 1.5)
    ds = None if st["s"] is None else st["alpha"] * (dr * z).sum(0)
    dz = dr * wy
    if wp is None:
        return dr, dz, (dn * x / mr.sqrt()).sum(0), None, ds
    dy = dz * wp / my.sqrt() - y * (dz * wp * y).sum(-1, keepdim=True) / (D * my ** 1.5)
    return dr, dy, (dn * x / mr.sqrt()).sum(0), (dz * y / my.sqrt()).sum(0), ds
