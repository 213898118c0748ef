"""Plain fp64 implementations of linear attention with a decay for each head (the token
recurrence and its reverse) and of the norms around it, for the GPU tests.  Every function
also returns, where asked (``magnitude``), the same sums over absolute values: the scale a
rounding error of the kernel's products is relative to."""
import torch


def lin_inputs(seed, B, H, Hk, T, dk, dv, decay="token", n_state=None, strong=False):
    """Unit-row Q, K, normal V and dO in bf16, log-decays in fp32, states in fp32 (CPU)."""
    g = torch.Generator().manual_seed(seed)
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(s, generator=g), dim=-1).bfloat16()  # noqa: E731
    x = {"Q": unit(B, Hk, T, dk), "K": unit(B, Hk, T, dk), "V": torch.randn((B, H, T, dv), generator=g).bfloat16(),
         "dO": torch.randn((B, H, T, dv), generator=g).bfloat16()}
    if decay == "head":
        x["g"] = -torch.exp2(-2.0 - 8.0 * torch.rand(H, generator=g))
    else:
        x["g"] = torch.nn.functional.logsigmoid(torch.randn((B, H, T), generator=g) + 2.0)
        if strong and T > 0:  # some tokens forget nearly everything, some everything
            x["g"][torch.rand((B, H, T), generator=g) < 0.05] = -60.0
            x["g"][torch.rand((B, H, T), generator=g) < 0.03] = -float("inf")
    n = B if n_state is None else n_state
    x["S0"] = 0.5 * torch.randn((n, H, dk, dv), generator=g)
    x["dS"] = 0.5 * torch.randn((n, H, dk, dv), generator=g)
    return x


def _heads(x, H):
    return x.double().repeat_interleave(H // x.shape[1], dim=1)


def _decay(g, B, H, T):
    g = g.double()
    return torch.exp(g.view(1, H, 1).expand(B, H, T) if g.dim() == 1 else g)


def _spans(B, T, lens):
    if lens is None:
        return None
    at, out = 0, []
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def lin_forward(x, scale, S0=None, lens=None, first=0, magnitude=False):
    """O [B,H,T,dv] (zeros outside the sequences) and the final states; lens: packed lengths
    starting at token ``first`` of the one row."""
    f = (lambda t: t.double().abs()) if magnitude else (lambda t: t.double())
    H = x["V"].shape[1]
    q, k, v = _heads(f(x["Q"]), H), _heads(f(x["K"]), H), f(x["V"])
    B, _, T, dv = v.shape
    dk = q.shape[-1]
    a = _decay(x["g"], B, H, T)
    O = torch.zeros_like(v)
    spans = [(0, T)] if lens is None else [(first + s, first + e) for s, e in _spans(B, T, lens)]
    last = []
    for i, (t0, t1) in enumerate(spans):
        if S0 is None:
            S = torch.zeros((B, H, dk, dv), dtype=torch.float64)
        else:
            S = f(S0) if lens is None else f(S0[i:i + 1])
        for t in range(t0, t1):
            S = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
            O[:, :, t] = abs(scale) * torch.einsum("bhkv,bhk->bhv", S, q[:, :, t])
        last.append(S)
    return (O if magnitude or scale >= 0 else -O), torch.cat(last)


def lin_backward(x, scale, S0=None, dS=None, lens=None, first=0, magnitude=False):
    """dQ, dK, dV, dg, dS0 (all fp64; rows outside the sequences zero); scale > 0."""
    f = (lambda t: t.double().abs()) if magnitude else (lambda t: t.double())
    H = x["V"].shape[1]
    Hk = x["Q"].shape[1]
    q, k, v, do = _heads(f(x["Q"]), H), _heads(f(x["K"]), H), f(x["V"]), f(x["dO"])
    B, _, T, dv = v.shape
    dk = q.shape[-1]
    a = _decay(x["g"], B, H, T)
    dQ, dK, dV, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros((B, H, T)).double()
    spans = [(0, T)] if lens is None else [(first + s, first + e) for s, e in _spans(B, T, lens)]
    out = []
    zeros = torch.zeros((B, H, dk, dv), dtype=torch.float64)
    for i, (t0, t1) in enumerate(spans):
        pick = lambda S: zeros if S is None else f(S) if lens is None else f(S[i:i + 1])  # noqa: E731
        S, before = pick(S0), []
        for t in range(t0, t1):
            before.append(a[:, :, t, None, None] * S)
            S = before[-1] + k[:, :, t, :, None] * v[:, :, t, None, :]
        D = pick(dS)
        for t in reversed(range(t0, t1)):
            old = before[t - t0]
            D = D + scale * q[:, :, t, :, None] * do[:, :, t, None, :]
            after = old + k[:, :, t, :, None] * v[:, :, t, None, :]
            dQ[:, :, t] = scale * torch.einsum("bhkv,bhv->bhk", after, do[:, :, t])
            dK[:, :, t] = torch.einsum("bhkv,bhv->bhk", D, v[:, :, t])
            dV[:, :, t] = torch.einsum("bhkv,bhk->bhv", D, k[:, :, t])
            dg[:, :, t] = (D * old).sum((-1, -2))
            D = a[:, :, t, None, None] * D
        out.append(D)
    shared = lambda y: y.unflatten(1, (Hk, H // Hk)).sum(2)  # noqa: E731
    if x["g"].dim() == 1:
        dg = dg.sum((0, 2))
    return shared(dQ), shared(dK), dV, dg, torch.cat(out)


def gate_norm(O, Z, w, eps, act):
    o, z = O.double().transpose(1, 2), Z.double()
    n = o / torch.sqrt(o.square().mean(-1, keepdim=True) + eps)
    f = z * torch.sigmoid(z) if act == "silu" else torch.sigmoid(z)
    return n * (1.0 if w is None else w.double()) * f


def residual_norm(X, Y, w_post, s, alpha, w_pre, eps):
    rms = lambda t: t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)  # noqa: E731
    x, y = X.double(), Y.double()
    if w_post is not None:
        y = rms(y) * w_post.double()
    if s is not None:
        y = y * s.double()
    r = x + alpha * y
    n = rms(r)
    return r, n if w_pre is None else n * w_pre.double()
