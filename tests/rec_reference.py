"""Plain fp64 implementations of the gated linear recurrence of every channel (token by token and in
reverse) and of the norm and rotation of queries and keys, for the GPU tests.  Beside each result of
the recurrence stands a bound of what fp32 arithmetic may leave of it.

The bound, per token: exponentials, reciprocals and roots are right to 2^-22 each, a = exp(g) also
to 2^-22 |g|, and 1 - a to 2^-21 where the series gives way to the difference (|g| = 1/4): a and u are
right to EPS (1 + |g|), EPS = 2^-20, of themselves.  With M the recurrence over absolute values,
E_t = a E_{t-1} + EPS (1 + |g_t|) M_t bounds the error of h, whatever the order of the sums (a
product of decays adds 2^-24 a token); the gradients' bounds follow from theirs term by term.

A sigmoid below 2^-126 is none of fp32's normal numbers and counts as 0: s(A) of the decay "power"
(w <= 2), or what "sigmoid" leaves of 1 (w = 1).  With sqrt(1 - a^2) that takes away
b = sqrt(1 - exp(-2 w s)) <= sqrt(2 w s) < 2^-61.5, and of dA and dw
D z b'(g) w s = D z a^2 w s / b <= D z sqrt(w s): FLOOR of their factors at most, beside what EPS
bounds."""
import torch

EPS, FLOOR = 2.0 ** -20, 2.0 ** -61


def rec_inputs(seed, B, T, D, decay="power", gate=True, dtype=torch.float32, n_state=None, slow=False):
    """X, A, I, dH in dtype, w, h0, dh in fp32 (CPU)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    A = r(B, T, D) * 2
    if decay == "log":
        A = torch.nn.functional.logsigmoid(A + (6.0 if slow else 1.0))
    elif slow:
        A = A + (6.0 if decay == "sigmoid" else -4.0)
    n = B if n_state is None else n_state
    return {"X": r(B, T, D).to(dtype), "A": A.to(dtype), "I": r(B, T, D).to(dtype) if gate else None,
            "w": 2.0 * torch.rand(D, generator=g) if decay == "power" else None, "h0": r(n, D), "dH": r(B, T, D).to(dtype),
            "dh": r(n, D)}


def gates(x, decay, norm):
    """g, a, b, b'(g), s(I), the factor from dg to dA, s(A), all fp64."""
    A = x["A"].double()
    s, rest = torch.sigmoid(A), torch.sigmoid(-A)
    if decay == "power":
        g = -x["w"].double() * s
        to_A = g * rest
    elif decay == "sigmoid":
        g, to_A = torch.nn.functional.logsigmoid(A), rest
    else:
        g, to_A = A, torch.ones_like(A)
    a, m = torch.exp(g), torch.expm1(g)
    if norm == "sqrt":
        b = torch.sqrt(-m * (2 + m))
        db = torch.where(b > 0, -a * a / b, 0.0)
    elif norm == "linear":
        b, db = -m, -a
    else:
        b, db = torch.ones_like(a), torch.zeros_like(a)
    i = torch.ones_like(a) if x["I"] is None else torch.sigmoid(x["I"].double())
    return g, a, b, db, i, to_A, s


def spans_of(B, T, lens, first):
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    at, out = first, []
    for n in lens:
        out.append((0, at, at + n))
        at += n
    return out


def rec_forward(x, decay, norm, h0=None, lens=None, first=0):
    """H, the last states, their bounds, and h and its magnitude and bound before every token; rows of no
    sequence are zero."""
    g, a, b, _, i, _, _ = gates(x, decay, norm)
    X = x["X"].double()
    u, floor = b * i * X, FLOOR * (decay != "log" and norm == "sqrt")
    eps = EPS * (1 + torch.where(torch.isfinite(g), g.abs(), 0.0))
    B, T, D = u.shape
    H, EH, before, Mb, Eb = (torch.zeros_like(u) for _ in range(5))
    last, Elast = [], []
    for k, (row, s, e) in enumerate(spans_of(B, T, lens, first)):
        h = torch.zeros(D, dtype=torch.float64, device=X.device) if h0 is None else h0[k].double()
        M, E = h.abs(), torch.zeros(D, dtype=torch.float64, device=X.device)
        for t in range(s, e):
            before[row, t], Mb[row, t], Eb[row, t] = h, M, E
            h = a[row, t] * h + u[row, t]
            M = a[row, t] * M + u[row, t].abs()
            E = a[row, t] * E + eps[row, t] * M + floor * (i * X)[row, t].abs()
            H[row, t], EH[row, t] = h, E
        last.append(h)
        Elast.append(E)
    return H, torch.stack(last), EH, torch.stack(Elast), (before, Mb, Eb)


def rec_backward(x, decay, norm, h0=None, dh=None, lens=None, first=0):
    """dX, dA, dI, dw, dh0 (dI, dw None without I, w), and their bounds."""
    g, a, b, db, i, to_A, sA = gates(x, decay, norm)
    _, _, _, _, (before, Mb, Eb) = rec_forward(x, decay, norm, h0, lens, first)
    X, dH = x["X"].double(), x["dH"].double()
    eps = EPS * (1 + torch.where(torch.isfinite(g), g.abs(), 0.0))
    B, T, D = X.shape
    dX, dI, dg, EX, EI, Eg, lost = (torch.zeros_like(X) for _ in range(7))
    floor = FLOOR * (decay != "log" and norm == "sqrt")
    d0, Ed0 = [], []
    for k, (row, s, e) in enumerate(spans_of(B, T, lens, first)):
        d = torch.zeros(D, dtype=torch.float64, device=X.device) if dh is None else dh[k].double()
        M, E = d.abs(), torch.zeros(D, dtype=torch.float64, device=X.device)
        for t in reversed(range(s, e)):
            at = (row, t)
            d, M = d + dH[at], M + dH[at].abs()
            E = E + 2.0 ** -23 * M
            z, rest = i[at] * X[at], 1 - i[at]
            dX[at], EX[at] = d * b[at] * i[at], b[at] * i[at] * (E + 4 * eps[at] * M) + floor * M * i[at]
            dI[at], EI[at] = d * b[at] * z * rest, (b[at] * z * rest).abs() * (E + 4 * eps[at] * M) + floor * M * z.abs()
            lost[at] = floor * M * z.abs()
            dg[at] = d * (a[at] * before[at] + z * db[at])
            into = a[at] * Mb[at] + (z * db[at]).abs()
            Eg[at] = into * (E + 8 * eps[at] * M) + M * a[at] * Eb[at]
            d, M, E = a[at] * d, a[at] * M, a[at] * (E + eps[at] * M)
        d0.append(d)
        Ed0.append(E + 2.0 ** -23 * M)
    dw = Ew = None
    if decay == "power":
        dw, Ew = -(sA * dg).sum((0, 1)), (sA * (Eg + 2.0 ** -20 * dg.abs()) + lost).sum((0, 1))
    dA, EA = dg * to_A, to_A.abs() * (Eg + 2 * eps * dg.abs()) + lost
    if x["I"] is None:
        dI = EI = None
    return (dX, dA, dI, dw, torch.stack(d0)), (EX, EA, EI, Ew, torch.stack(Ed0))


# ---- queries and keys ------------------------------------------------------------------------


def qk_rotate(x, freqs, positions, pairs, axis, back=False):
    """x [B, T, heads, d] fp64 turned by its positions ([B, T], or [axes, B, T] with axis)."""
    if freqs is None:
        return x
    r = 2 * freqs.numel()
    p = positions.double()
    p = p[..., None] if axis is None else p[list(axis)].permute(1, 2, 0)
    angle = (p * freqs.double())[:, :, None]
    c, s = angle.cos(), angle.sin() * (-1 if back else 1)
    at = (slice(0, r // 2), slice(r // 2, r)) if pairs == "halves" else (slice(0, r, 2), slice(1, r, 2))
    y = x.clone()
    y[..., at[0]] = x[..., at[0]] * c - x[..., at[1]] * s
    y[..., at[1]] = x[..., at[0]] * s + x[..., at[1]] * c
    return y


def qk_forward(x, w, freqs, positions, norm, eps, pairs, axis):
    """[B, heads, T, d]."""
    x = x.double()
    n = x if norm == "none" else x / torch.sqrt((x.square().mean(-1, True) if norm == "rms" else
                                                 x.square().sum(-1, True)) + eps)
    return qk_rotate(n if w is None else n * w.double(), freqs, positions, pairs, axis).transpose(1, 2)


def qk_backward(dy, x, w, freqs, positions, norm, eps, pairs, axis):
    """dx [B, T, heads, d] and dw, and both over absolute values."""
    x = x.double()
    dn = qk_rotate(dy.double().transpose(1, 2), freqs, positions, pairs, axis, back=True)
    # of a turned pair either value may be as large as both together
    mag = dn.abs()
    if freqs is not None:
        r = 2 * freqs.numel()
        at = (slice(0, r // 2), slice(r // 2, r)) if pairs == "halves" else (slice(0, r, 2), slice(1, r, 2))
        both = dn[..., at[0]].abs() + dn[..., at[1]].abs()
        mag[..., at[0]], mag[..., at[1]] = both, both
    wd = torch.ones(x.shape[-1]).double() if w is None else w.double()
    if norm == "none":
        return dn * wd, mag * wd.abs(), (dn * x).sum((0, 1, 2)), (mag * x.abs()).sum((0, 1, 2))
    inv = 1.0 / x.shape[-1] if norm == "rms" else 1.0
    rstd = (inv * x.square().sum(-1, True) + eps).rsqrt()
    n, u, m = x * rstd, dn * wd, mag * wd.abs()
    dx = rstd * (u - n * inv * (u * n).sum(-1, True))
    mx = rstd * (m + n.abs() * inv * (m * n.abs()).sum(-1, True))
    return dx, mx, (dn * n).sum((0, 1, 2)), (mag * n.abs()).sum((0, 1, 2))
