"""The operators that perf measurements run: the gated linear recurrence (a scan over long
sequences, its backward pass, its one-token step) and the norm-and-rotation of queries and keys
(forward and backward), with their plain forms.

    listed()            the named cases
    draw(rng)           one more case of the same ranges
    prepare(case, seed) a case's inputs on the GPU
    run(state)          one pass: the plain form, or with `own` the library's entry points
    work(case)          bytes and operations a pass cannot do without
    exact(case, seed)   run()'s outputs from the definitions, in 64 bits

The recurrence, per channel (x the stream, a and b the decay and write gate logits):
    g_t = -exp(A_log) softplus(a_t + dt_bias),  alpha_t = e^g_t,  beta_t = sigmoid(b_t),
    h_t = alpha_t h_{t-1} + s(alpha_t) beta_t x_t,
    s = 1 ("none"), 1 - alpha ("tied") or sqrt(1 - alpha^2) ("unit").
The norm and rotation, per token and head: n = x / sqrt(mean(x^2) + eps) * w ("rms") or
x / sqrt(sum(x^2) + eps) ("l2"); the first `rot` channels are rotated in pairs by
position * inv_freq; queries are multiplied by a scale.
"""
import math

import torch

own = False

EPS = 1e-6


def _rec(name, op, **kw):
    c = dict(name=name, op=op, B=1, T=1, D=1, dtype="bf16", scale="none", write_gate=True,
             gates="logits", packed=0, fused=False)
    c.update(kw)
    return c


def _rot(name, op, **kw):
    c = dict(name=name, op=op, T=1, Hq=1, Hk=1, d=64, rot=64, dtype="bf16", norm="rms",
             interleaved=False, fused=False, far=8192, theta=1e6)
    c.update(kw)
    return c


def listed():
    return [
        # the mixed q|k|v stream of an 8K-token prefill layer (16 key, 64 value heads of 128),
        # smoothed by its own gates
        _rec("rec_fwd_8k_mixed", "rec_fwd", T=8192, D=12288),
        # one very long sequence over few channels: the scan has to be split along time
        _rec("rec_fwd_128k", "rec_fwd", T=131072, D=1024, scale="tied", write_gate=False),
        # a packed batch of ragged prompts, gates as slices of one projection's output
        _rec("rec_fwd_packed", "rec_fwd", B=48, T=20011, D=4096, scale="unit", packed=48,
             fused=True),
        # a small float32 batch of odd sizes
        _rec("rec_fwd_f32_odd", "rec_fwd", B=3, T=257, D=515, dtype="f32"),
        # a training pass over an 8K sequence of hidden size 4096: forward, then backward
        _rec("rec_train_8k", "rec_train", T=8192, D=4096),
        # the backward pass alone, float32, odd sizes
        _rec("rec_bwd_f32_odd", "rec_bwd", B=3, T=1037, D=1027, dtype="f32", scale="unit"),
        # decode: 256 sequences' mixed streams, and one sequence of hidden size 4096
        _rec("rec_step_256", "rec_step", B=256, D=12288),
        _rec("rec_step_1", "rec_step", B=1, D=4096, scale="unit"),
        # q and k of an 8K-token prefill layer, in the delta rule's own norm
        _rot("rot_fwd_8k", "rot_fwd", T=8192, Hq=16, Hk=16, d=128, rot=128, norm="l2"),
        # decode of a grouped-query attention layer: 256 tokens far into their contexts, slices
        # of the fused projection, a quarter of each head rotated
        _rot("rot_fwd_256_gqa", "rot_fwd", T=256, Hq=32, Hk=2, d=256, rot=64, fused=True,
             far=262144, theta=1e7),
        # the backward of both at 8K tokens, and at odd sizes in float32
        _rot("rot_bwd_8k", "rot_bwd", T=8192, Hq=16, Hk=16, d=128, rot=128),
        _rot("rot_bwd_f32_odd", "rot_bwd", T=777, Hq=5, Hk=1, d=80, rot=40, dtype="f32",
             interleaved=True, theta=1e4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.55:
        op = rng.choice(["rec_fwd", "rec_fwd", "rec_train", "rec_bwd", "rec_step"])
        most = 1 << (25 if op == "rec_fwd" else 24)  # elements
        scale, gate = rng.choice(["none", "tied", "unit"]), rng.random() < 0.7
        gates = "given" if rng.random() < 0.2 else "logits"
        D = _log_int(rng, 8, 12288)
        if rng.random() < 0.5:
            D = max(8, D // 8 * 8)
        if op == "rec_step":
            return dict(op=op, B=_log_int(rng, 1, min(4096, most // D)), T=1, D=D, dtype=dtype,
                        scale=scale, write_gate=gate, gates=gates, packed=0, fused=False)
        T = _log_int(rng, 1, min(131072, most // D))
        B = _log_int(rng, 1, max(1, min(64, most // (T * D))))
        packed = B if B > 1 and rng.random() < 0.4 else 0
        if packed:
            T = T * B
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, scale=scale, write_gate=gate, gates=gates,
                    packed=packed, fused=gates == "logits" and rng.random() < 0.4)
    op = rng.choice(["rot_fwd", "rot_bwd"])
    d = rng.choice([64, 128, 256, 96, 80, 40, 192, 112])
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hk * rng.choice([1, 2, 4, 5, 8])
    T = _log_int(rng, 1, max(1, min(65536, (1 << 25) // ((Hq + Hk) * d))))
    return dict(op=op, T=T, Hq=Hq, Hk=Hk, d=d, rot=rng.choice([d, d, d // 4 * 2, d // 8 * 2]),
                dtype=dtype, norm=rng.choice(["rms", "rms", "l2"]),
                interleaved=rng.random() < 0.3, fused=rng.random() < 0.5,
                far=rng.choice([4096, 32768, 262144]), theta=rng.choice([1e4, 1e6, 1e7]))


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """Packed batches: `packed` lengths that add up to T, from empty to several times the mean."""
    n, T = case["packed"], case["T"]
    w = [((i * 7919 + 13) % 31) ** 2 for i in range(n)]
    total = max(1, sum(w))
    cu, acc = [0], 0
    for x in w:
        acc += x
        cu.append(T * acc // total)
    cu[-1] = T
    return cu


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, f32 = _dt(case), torch.float32

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=f32).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, device="cuda", generator=gen, dtype=f32) * (hi - lo) + lo

    s = dict(case=dict(case))
    if case["op"].startswith("rec"):
        B, T, D = case["B"], case["T"], case["D"]
        cu = _lengths(case) if case["packed"] else None
        if case["op"] == "rec_step":
            lead = (B,)
        else:
            lead = (T,) if cu else (B, T)
        if case["fused"]:  # slices of one projection's output
            proj = normal(*lead, (3 if case["write_gate"] else 2) * D)
            s["x"], s["a"] = proj[..., :D], proj[..., D:2 * D]
            s["b"] = proj[..., 2 * D:] if case["write_gate"] else None
        else:
            s["x"], s["a"] = normal(*lead, D), normal(*lead, D)
            s["b"] = normal(*lead, D) if case["write_gate"] else None
        s["A_log"] = uniform(0.0, math.log(16.0), D)
        s["dt_bias"] = uniform(-4.0, -1.0, D)
        if case["gates"] == "given":  # log-decays and write gates themselves, in float32
            s["a"] = -s["A_log"].exp() * torch.nn.functional.softplus(s["a"].float() + s["dt_bias"])
            s["b"] = torch.sigmoid(s["b"].float()) if s["b"] is not None else None
            s["A_log"] = s["dt_bias"] = None
        s["h0"] = uniform(-1.0, 1.0, B, D)
        s["cu"] = cu
        if case["op"] in ("rec_train", "rec_bwd"):
            s["dh"] = normal(*lead, D)
            s["dht"] = normal(B, D, dtype=f32)
        if cu:
            n = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device="cuda")
            first = torch.tensor(cu[:-1], device="cuda")
            full = n > 0
            s["seq"] = dict(full=full, first=first[full], last=(first + n - 1)[full])
        return s
    T, Hq, Hk, d, r = (case[k] for k in ("T", "Hq", "Hk", "d", "rot"))
    if case["fused"]:  # q | k | v of one projection
        qkv = normal(T, (Hq + 2 * Hk) * d)
        s["q"] = qkv[:, :Hq * d].unflatten(1, (Hq, d))
        s["k"] = qkv[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    else:
        s["q"], s["k"] = normal(T, Hq, d), normal(T, Hk, d)
    s["pos"] = torch.randint(0, case["far"], (T,), device="cuda", generator=gen)
    i = torch.arange(0, r, 2, device="cuda", dtype=torch.float64)
    s["inv_freq"] = torch.pow(case["theta"], -i / max(1, r)).float()
    rms = case["norm"] == "rms"
    s["qw"] = uniform(0.5, 1.5, d) if rms else None
    s["kw"] = uniform(0.5, 1.5, d) if rms else None
    s["scale"] = d ** -0.5
    if case["op"] == "rot_bwd":
        s["dq"], s["dk"] = normal(T, Hq, d), normal(T, Hk, d)
    return s


# ---- the plain forms --------------------------------------------------------------------------


def _gates(s):
    """alpha, s(alpha) and beta in float32, and what the backward needs of them."""
    case, a, b = s["case"], s["a"].float(), s["b"]
    if case["gates"] == "given":
        g, slope = a, None
        beta = b
    else:
        z = a + s["dt_bias"]
        neg = -s["A_log"].exp()
        g = neg * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
        slope = neg / (1 + torch.exp(-z))
        beta = None if b is None else 1 / (1 + torch.exp(-b.float()))
    alpha = torch.exp(g)
    if case["scale"] == "tied":
        f = -torch.expm1(g)
    elif case["scale"] == "unit":
        f = torch.sqrt(-torch.expm1(2 * g))
    else:
        f = None
    return g, slope, alpha, beta, f


def _scan(alpha, u):
    """h_t = alpha_t h_{t-1} + u_t along dimension 1, by doubling."""
    n = 1
    while n < u.shape[1]:
        u = torch.cat([u[:, :n], u[:, n:] + alpha[:, n:] * u[:, :-n]], 1)
        alpha = torch.cat([alpha[:, :n], alpha[:, n:] * alpha[:, :-n]], 1)
        n *= 2
    return u


def _times(x, *fs):
    for f in fs:
        x = x if f is None else x * f
    return x


def _plain_fwd(s, alpha, beta, f):
    """The float32 states h [*, T, D] and the final states."""
    u = _times(s["x"].float(), f, beta).clone()  # the inputs stay as they are
    if s["cu"]:
        seq = s["seq"]
        u[seq["first"]] += alpha[seq["first"]] * s["h0"][seq["full"]]
        cut = alpha.clone()
        cut[seq["first"]] = 0
        h = _scan(cut[None], u[None])[0]
        ht = s["h0"].clone()
        ht[seq["full"]] = h[seq["last"]]
        return h, ht, cut
    u[:, 0] += alpha[:, 0] * s["h0"]
    h = _scan(alpha, u)
    return h, h[:, -1].clone(), alpha


def _plain_bwd(s, gates, h, cut):
    g, slope, alpha, beta, f = gates
    case, cu = s["case"], s["cu"]
    dh = s["dh"].float().clone()
    if cu:
        seq = s["seq"]
        dh[seq["last"]] += s["dht"][seq["full"]]
        after = torch.cat([cut[1:], torch.zeros_like(cut[:1])], 0)[None]
        lam = _scan(after.flip(1), dh[None].flip(1)).flip(1)[0]
        prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]], 0)
        prev[seq["first"]] = s["h0"][seq["full"]]
        dh0 = s["dht"].clone()
        dh0[seq["full"]] = (alpha * lam)[seq["first"]]
    else:
        dh[:, -1] += s["dht"]
        after = torch.cat([alpha[:, 1:], torch.zeros_like(alpha[:, :1])], 1)
        lam = _scan(after.flip(1), dh.flip(1)).flip(1)
        prev = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
        dh0 = alpha[:, 0] * lam[:, 0]
    x = s["x"].float()
    dx = _times(lam, f, beta)
    dg = alpha * lam * prev
    if case["scale"] == "tied":
        dg = dg - alpha * _times(lam * x, beta)
    elif case["scale"] == "unit":
        dg = dg - torch.where(f > 0, alpha * alpha / f, 0.0) * _times(lam * x, beta)
    out = dict(dx=dx.to(s["x"].dtype), dh0=dh0)
    if beta is not None:
        db = _times(lam * x, f)
        out["db"] = (db * beta * (1 - beta)).to(s["x"].dtype) if slope is not None else db
    if slope is None:
        out["da"] = dg
    else:
        da = dg * slope
        over = tuple(range(da.dim() - 1))
        out["da"] = da.to(s["x"].dtype)
        out["ddt_bias"] = da.sum(over, dtype=torch.float64).float()
        out["dA_log"] = (dg * g).sum(over, dtype=torch.float64).float()
    return out


def _plain_rec(s):
    case = s["case"]
    gates = _gates(s)
    _, _, alpha, beta, f = gates
    if case["op"] == "rec_step":
        s["h0"].copy_(alpha * s["h0"] + _times(s["x"].float(), f, beta))
        return dict(h=s["h0"].to(s["x"].dtype), state=s["h0"])
    h, ht, cut = _plain_fwd(s, alpha, beta, f)
    out = dict(h=h.to(s["x"].dtype), ht=ht) if case["op"] != "rec_bwd" else {}
    if case["op"] != "rec_fwd":
        out.update(_plain_bwd(s, gates, h, cut))
    return out


def _norm(case, x, w):
    """The normalised rows, the factor that normalised them, and the rows times the weight."""
    ss = (x * x).sum(-1, keepdim=True)
    inv = torch.rsqrt(ss / case["d"] + EPS) if case["norm"] == "rms" else torch.rsqrt(ss + EPS)
    n = x * inv
    return n, inv, n if w is None else n * w


def _turn(s, y, back=False):
    """The first `rot` channels rotated in pairs by position * inv_freq (64 bits: far positions)."""
    case = s["case"]
    r = case["rot"]
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    c, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    sn = -sn if back else sn
    if case["interleaved"]:
        p, q = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([p * c - q * sn, q * c + p * sn], -1).flatten(-2)
    else:
        p, q = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([p * c - q * sn, q * c + p * sn], -1)
    return torch.cat([turned, y[..., r:]], -1)


def _plain_rot(s):
    case = s["case"]
    out = {}
    for name, w, scale in (("q", s["qw"], s["scale"]), ("k", s["kw"], 1.0)):
        x = s[name].float()
        n, inv, y = _norm(case, x, w)
        if case["op"] == "rot_fwd":
            out[name] = (_turn(s, y) * scale).to(s[name].dtype)
            continue
        dy = _turn(s, s["d" + name].float() * scale, back=True)
        if w is not None:
            out["d" + name + "w"] = (dy * n).sum((0, 1), dtype=torch.float64).float()
            dy = dy * w
        m = (dy * n).sum(-1, keepdim=True)
        m = m / case["d"] if case["norm"] == "rms" else m
        out["d" + name] = (inv * (dy - n * m)).to(s[name].dtype)
    return out


# ---- one pass ---------------------------------------------------------------------------------


def _own_rec(s):
    import gated_deltanet_sequence_gdn_b200 as G
    case = s["case"]
    kw = dict(input_scale=case["scale"], gates_precomputed=case["gates"] == "given")
    args = (s["x"], s["a"], s["b"], s["A_log"], s["dt_bias"])
    if case["op"] == "rec_step":
        return dict(h=G.gdn_linrec_step(*args, s["h0"], **kw), state=s["h0"])
    kw["cu_seqlens"] = s["cu"]
    if case["op"] == "rec_fwd":
        h, ht = G.gdn_linrec_fwd(*args, s["h0"], **kw)
        return dict(h=h, ht=ht)
    out, states = {}, None
    if case["op"] == "rec_train":
        out["h"], out["ht"], states = G.gdn_linrec_fwd(*args, s["h0"], want_states=True, **kw)
    grads = G.gdn_linrec_bwd(*args, s["h0"], s["dh"], s["dht"], states=states, **kw)
    out.update((k, v) for k, v in grads.items() if v is not None)
    return out


def _own_rot(s):
    import gated_deltanet_sequence_gdn_b200 as G
    case = s["case"]
    kw = dict(norm=case["norm"], eps=EPS, scale=s["scale"], interleaved=case["interleaved"])
    args = (s["q"], s["k"], s["pos"], s["inv_freq"], s["qw"], s["kw"])
    if case["op"] == "rot_fwd":
        q, k = G.gdn_qk_norm_rope(*args, **kw)
        return dict(q=q, k=k)
    grads = G.gdn_qk_norm_rope_bwd(*args, s["dq"], s["dk"], **kw)
    return {dict(dq_weight="dqw", dk_weight="dkw").get(k, k): v
            for k, v in grads.items() if v is not None}


def run(state):
    rec = state["case"]["op"].startswith("rec")
    if own:
        return _own_rec(state) if rec else _own_rot(state)
    return _plain_rec(state) if rec else _plain_rot(state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("rec"):
        B, D = case["B"], case["D"]
        n = (case["T"] if case["packed"] else B * case["T"]) * D
        ge = 4 if case["gates"] == "given" else e
        ins = e + ge * (2 if case["write_gate"] else 1)  # x, a, b
        state = 2 * 4 * B * D                            # h0 in, the final state out
        if case["op"] in ("rec_fwd", "rec_step"):
            return dict(bytes=n * (ins + e) + state, flops=12 * n)
        both = n * (2 * ins + e)                         # x, a, b, dh in; dx, da, db out
        if case["op"] == "rec_bwd":
            return dict(bytes=both + 2 * state, flops=30 * n)
        return dict(bytes=both + n * e + 2 * state, flops=40 * n)
    n = case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
    per_token = 8 * case["T"]
    if case["op"] == "rot_fwd":
        return dict(bytes=2 * e * n + per_token, flops=8 * n)
    return dict(bytes=3 * e * n + per_token, flops=16 * n)


# ---- the definitions in 64 bits ---------------------------------------------------------------


def _exact_rec(s):
    case = s["case"]
    leaf = {k: s[k].double().requires_grad_(True)
            for k in ("x", "a", "b", "A_log", "dt_bias") if s[k] is not None}
    with torch.enable_grad():
        if case["gates"] == "given":
            g, beta = leaf["a"] * 1.0, leaf.get("b")
        else:
            g = -torch.exp(leaf["A_log"]) * torch.nn.functional.softplus(
                leaf["a"] + leaf["dt_bias"], threshold=1000.0)
            beta = torch.sigmoid(leaf["b"]) if "b" in leaf else None
        alpha = torch.exp(g)
        u = leaf["x"] if beta is None else beta * leaf["x"]
        if case["scale"] == "tied":
            u = u * -torch.expm1(g)
        elif case["scale"] == "unit":
            u = u * torch.sqrt(-torch.expm1(2 * g))
        u = u * 1.0
    al, ul = alpha.detach(), u.detach()
    h0 = s["h0"].double()
    if case["op"] == "rec_step":
        state = al * h0 + ul
        return dict(h=state, state=state)
    cu = s["cu"]
    # token by token; dense batches take all their rows at once
    spans = [(i, c, d) for i, (c, d) in enumerate(zip(cu, cu[1:]))] if cu else [(None, 0, case["T"])]
    h, prev, ht = torch.empty_like(ul), torch.empty_like(ul), h0.clone()

    def at(t, v):
        return v[t] if cu else v[:, t]

    for i, lo, hi in spans:
        cur = h0[i] if cu else h0
        for t in range(lo, hi):
            at(t, prev).copy_(cur)
            cur = torch.addcmul(at(t, ul), at(t, al), cur, out=at(t, h))
        if hi > lo:
            (ht[i] if cu else ht).copy_(cur)
    out = dict(h=h, ht=ht) if case["op"] != "rec_bwd" else {}
    if case["op"] == "rec_fwd":
        return out
    lam, dh0 = s["dh"].double(), s["dht"].double().clone()
    for i, lo, hi in spans:
        carry = (dh0[i] if cu else dh0).clone()
        for t in range(hi - 1, lo - 1, -1):
            at(t, lam).add_(carry)
            torch.mul(at(t, al), at(t, lam), out=carry)
        (dh0[i] if cu else dh0).copy_(carry)
    names = [k for k in ("x", "a", "b", "A_log", "dt_bias") if k in leaf]
    grads = torch.autograd.grad([alpha, u], [leaf[k] for k in names], [lam * prev, lam])
    out["dh0"] = dh0
    out.update(("d" + k, v) for k, v in zip(names, grads))
    return out


def _exact_rot(s):
    case = s["case"]
    r, out = case["rot"], {}
    ang = s["pos"].double()[:, None, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(ang), ang)
    for name, w, scale in (("q", s["qw"], s["scale"]), ("k", s["kw"], 1.0)):
        x = s[name].double().requires_grad_(True)
        leaves = [x] if w is None else [x, w.double().requires_grad_(True)]
        with torch.enable_grad():
            total = x.square().sum(-1, keepdim=True)
            y = x / torch.sqrt(total / case["d"] + EPS if case["norm"] == "rms" else total + EPS)
            y = y * scale if w is None else y * (leaves[1] * scale)
            if case["interleaved"]:
                z = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * turn
                head = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * turn
                head = torch.cat([z.real, z.imag], -1)
            y = torch.cat([head, y[..., r:]], -1)
        if case["op"] == "rot_fwd":
            out[name] = y.detach()
            continue
        got = torch.autograd.grad([y], leaves, [s["d" + name].double()])
        out.update(zip(("d" + name, "d" + name + "w"), got))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rec(s) if case["op"].startswith("rec") else _exact_rot(s)
