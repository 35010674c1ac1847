"""Plain 64-bit forms of the gated linear recurrence and of the norm-and-rotation, token by
token from their definitions, and the error bounds their float32 kernels are held to.

Bounds.  u = 2^-24 (half a float32 step, relative).
Recurrence.  Per token the kernels form alpha with a relative error of at most (16 + 8 |g|) u
(2 u from the SFU's ex2, the rounding of g and of its product with log2 e, each |g| u, and the
errors of exp(A_log), softplus and the product behind g, at most 5 |g| u), the input f beta x
with at most 32 u (one SFU quotient, exponential and root each for beta and f, and their
products; 1 - alpha keeps its relative accuracy) and what the exponents' own rounding adds:
e^{-|v|} is 2^p with p = -|v| log2 e, whose rounding and that of the constant log2 e are together
at most 1.25 u |p|, so 1.25 u |v| relative, for v = b (beta, where b < 0) and v = z (softplus,
where z < 0; it reaches alpha through g, f and dg/da).  And one rounding for each multiply-add, of
which the carry joins of a chunk add a few.  Let m_t = alpha m_{t-1} + |input| be the recurrence
of the absolute values.  The error of h_t is then at most u (48 m_t + N_t), where N collects what
the decays' errors add up to over the memory: N_t = alpha (N_{t-1} + (20 + 8 |g|) m_{t-1})
+ 1.25 (|b| + |z|) |input|, the |g| with its factor 1 + |z| / 6.
The backward is the same recurrence run the other way on dh, with (m', N') for (m, N), and
products of the two: each gradient is held to u (96 M + cross terms), M its value with every
term's absolute value taken.  Sums over tokens add an absolute sum of their terms' bounds.
Stores add half a step of their type."""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F64 = torch.float64


def gates(a, b, A_log, dt_bias, scale, given):
    """g, alpha, beta (or None), f in 64 bits, differentiable."""
    a = a.to(F64)
    if given:
        g, beta = a, None if b is None else b.to(F64)
    else:
        z = a + dt_bias.to(F64)
        g = -torch.exp(A_log.to(F64)) * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
        beta = None if b is None else torch.sigmoid(b.to(F64))
    alpha = torch.exp(g)
    if scale == "tied":
        f = -torch.expm1(g)
    elif scale == "unit":
        f = torch.sqrt(-torch.expm1(2 * g))
    else:
        f = torch.ones_like(g)
    return g, alpha, beta, f


def spans(shape, cu):
    """(index of the row's tokens) of each sequence; tensors are [B, T, D] or [T, D]."""
    if cu is None:
        return [(i, slice(0, shape[1])) for i in range(shape[0])]
    return [slice(lo, hi) for lo, hi in zip(cu, cu[1:])]


def _rows(v, where):
    return v[where[0]][where[1]] if isinstance(where, tuple) else v[where]


def recurrence(x, a, b, A_log, dt_bias, h0, *, cu=None, scale="none", given=False):
    """h and ht in 64 bits, differentiable (one sequence after another)."""
    g, alpha, beta, f = gates(a, b, A_log, dt_bias, scale, given)
    u = f * x.to(F64) if beta is None else f * beta * x.to(F64)
    hs, hts = [], []
    where = spans(x.shape, cu)
    for i, w in enumerate(where):
        al, ul = _rows(alpha, w), _rows(u, w)
        cur = torch.zeros(x.shape[-1], dtype=F64) if h0 is None else h0[i].to(F64)
        out = []
        for t in range(al.shape[0]):
            cur = al[t] * cur + ul[t]
            out.append(cur)
        hs.append(torch.stack(out) if out else ul * 0)
        hts.append(cur)
    if cu is None:
        h = torch.stack(hs) if hs else u
    else:
        h = torch.cat(hs) if hs else u[:0]
    ht = torch.stack(hts) if hts else torch.zeros(0, x.shape[-1], dtype=F64)
    return h, ht


def exponents(a, b, A_log, dt_bias, g, given):
    """(1.25 (|b| + |z|) where they are negative, |g| times 1 + |z| / 6)."""
    if given:
        return torch.zeros_like(g), g.abs()
    z = (-(a.to(F64) + dt_bias.to(F64))).clamp(min=0)
    v = z if b is None else z + (-b.to(F64)).clamp(min=0)
    return 1.25 * v, g.abs() * (1 + z / 6)


def _scan(al, ul, start, ga, more=None):
    """(value, m, N) of the recurrence over [T, D], as lists of the values before and after
    each token."""
    h, m, n = start.clone(), start.abs(), torch.zeros_like(start)
    before, after = [], []
    for t in range(al.shape[0]):
        before.append((h, m, n))
        n = al[t] * (n + (20 + 8 * ga[t]) * m)
        if more is not None:
            n = n + more[t] * ul[t].abs()
        h, m = al[t] * h + ul[t], al[t] * m + ul[t].abs()
        after.append((h, m, n))
    cols = [torch.stack([r[k] for r in rows]) if rows else torch.zeros(0, al.shape[1], dtype=F64)
            for rows in (before, after) for k in range(3)]
    return cols, (h, m, n)


def forward_bounds(x, a, b, A_log, dt_bias, h0, *, cu=None, scale="none", given=False):
    """{name: (value, bound)} of h and ht before any store rounding."""
    g, alpha, beta, f = gates(a, b, A_log, dt_bias, scale, given)
    u = f * x.to(F64) if beta is None else f * beta * x.to(F64)
    more, ga = exponents(a, b, A_log, dt_bias, g, given)
    H, E, F, FE = [], [], [], []
    for i, w in enumerate(spans(x.shape, cu)):
        start = torch.zeros(x.shape[-1], dtype=F64) if h0 is None else h0[i].to(F64)
        cols, (h, m, n) = _scan(_rows(alpha, w), _rows(u, w), start, _rows(ga, w), _rows(more, w))
        H.append(cols[3])
        E.append(U * (48 * cols[4] + cols[5]))
        F.append(h)
        FE.append(U * (48 * m + n))
    join = torch.stack if cu is None else torch.cat
    return {"h": (join(H), join(E)), "ht": (torch.stack(F), torch.stack(FE))}


def backward_bounds(x, a, b, A_log, dt_bias, h0, dh, dht, *, cu=None, scale="none", given=False):
    """{name: (value, bound)} of the gradients, by the formulas."""
    g, alpha, beta, f = gates(a, b, A_log, dt_bias, scale, given)
    xx = x.to(F64)
    be = torch.ones_like(g) if beta is None else beta
    if scale == "tied":
        fp = -alpha
    elif scale == "unit":
        fp = torch.where(f > 0, -alpha * alpha / f, 0.0)
    else:
        fp = torch.zeros_like(g)
    more, gabs = exponents(a, b, A_log, dt_bias, g, given)
    names = ["dx", "da"] + ([] if b is None else ["db"])
    per = {k: [] for k in names}
    per_e = {k: [] for k in names}
    dh0, dh0_e = [], []
    A = bias = A_e = bias_e = torch.zeros(x.shape[-1], dtype=F64)
    for i, w in enumerate(spans(x.shape, cu)):
        al, gg, bb, ff, xr, fr = (_rows(v, w) for v in (alpha, g, be, f, xx, fp))
        zero = torch.zeros(x.shape[-1], dtype=F64)
        start = zero if h0 is None else h0[i].to(F64)
        mo, gm = _rows(more, w), _rows(gabs, w)
        cols, _ = _scan(al, ff * bb * xr, start, gm, mo)
        prev, pm, pn = cols[0], cols[1], cols[2]
        end = zero if dht is None else dht[i].to(F64)
        # lambda_t = dh_t + alpha_{t+1} lambda_{t+1}; the first factor (1) brings dht in
        T = al.shape[0]
        if T == 0:
            dh0.append(end)
            dh0_e.append(zero)
            for k in names:
                per[k].append(xr * 0)
                per_e[k].append(xr * 0)
            continue
        after = torch.cat([al[1:], torch.ones_like(al[:1])]).flip(0)
        ga = torch.cat([gm[1:], torch.zeros_like(gm[:1])]).flip(0)
        cols, _ = _scan(after, _rows(dh.to(F64), w).flip(0), end, ga)
        lam, lm, ln = (cols[k].flip(0) for k in (3, 4, 5))
        dh0.append(al[0] * lam[0])
        dh0_e.append(U * (al[0] * (ln[0] + (68 + 8 * gm[0]) * lm[0])))

        def put(k, v, mag, cross):
            e = U * ((96 + mo) * mag + cross)
            per[k].append(v)
            per_e[k].append(e)
            return v, e

        rel = 96 + 8 * gm + mo
        put("dx", lam * ff * bb, lm * ff * bb, ln * ff * bb)
        if b is not None:
            db, mag, cross = lam * ff * xr, lm * ff * xr.abs(), ln * ff * xr.abs()
            # beta (1 - beta), without the cancellation in 1 - beta
            slope = 1.0 if given else bb * torch.sigmoid(-_rows(b, w).to(F64))
            put("db", db * slope, mag * slope, cross * slope)
        dg = al * lam * prev + lam * bb * xr * fr
        mag = al * lm * pm + lm * (bb * xr * fr).abs()
        cross = al * (ln * pm + lm * pn) + ln * (bb * xr * fr).abs() + rel * mag
        if given:
            put("da", dg, mag, cross)
        else:
            z = _rows(a, w).to(F64) + dt_bias.to(F64)
            sl = torch.exp(A_log.to(F64)) * torch.sigmoid(z)
            v, e = put("da", -dg * sl, mag * sl, cross * sl)
            bias = bias + v.sum(0)
            bias_e = bias_e + e.sum(0) + U * 64 * v.abs().sum(0)
            A = A + (dg * gg).sum(0)
            A_e = A_e + (U * ((96 + mo) * mag + cross) * gg.abs()).sum(0) + U * 64 * (dg * gg).abs().sum(0)
    join = torch.stack if cu is None else torch.cat
    out = {k: (join(per[k]), join(per_e[k])) for k in names}
    out["dh0"] = (torch.stack(dh0), torch.stack(dh0_e))
    if not given:
        out["dA_log"], out["ddt_bias"] = (A, A_e), (bias, bias_e)
    return out


def check(name, got, value, bound, stored=None):
    """`got` within its bound (and half a step of the type it is stored in) of the value."""
    got = got.detach().cpu()
    half = HALF_STEP[stored or got.dtype]
    d = (got.to(F64) - value).abs()
    # values below the smallest normal number are held to its step
    lim = bound * (1 + half) + half * value.abs() + 1e-37
    assert got.shape == value.shape, f"{name}: {tuple(got.shape)} for {tuple(value.shape)}"
    assert torch.isfinite(got).all(), f"{name}: not finite"
    bad = d > lim
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float((d / lim).max()):.3g} of the bound")


# ---- norm and rotation ------------------------------------------------------------------------


def norm_rope(x, pos, inv_freq, w, *, norm="rms", eps=1e-6, scale=1.0, interleaved=False):
    """One of q, k [..., H, d] in 64 bits, differentiable."""
    x = x.to(F64) if x.dtype != F64 else x
    if norm == "rms":
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    elif norm == "l2":
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) + eps)
    if w is not None:
        x = x * (w if w.dtype == F64 else w.to(F64))
    x = x * scale
    if inv_freq is None or inv_freq.numel() == 0:
        return x
    r = 2 * inv_freq.numel()
    # the angle modulo a turn: position * inv_freq is below 2^53 steps of 2^-24 here
    ang = (pos.to(F64)[..., None] * inv_freq.to(F64))[..., None, :]
    c, s = ang.cos(), ang.sin()
    if interleaved:
        p, q = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([p * c - q * s, q * c + p * s], -1).flatten(-2)
    else:
        p, q = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([p * c - q * s, q * c + p * s], -1)
    return torch.cat([y, x[..., r:]], -1)


def rope_pair_size(y, r, interleaved):
    """The length of each value's pair (what a rotation's rounding is relative to)."""
    y = y.abs()
    if r == 0:
        return y
    if interleaved:
        m = (y[..., 0:r:2] + y[..., 1:r:2]).repeat_interleave(2, -1)
    else:
        m = y[..., :r // 2] + y[..., r // 2:r]
        m = torch.cat([m, m], -1)
    return torch.cat([m, y[..., r:]], -1)
