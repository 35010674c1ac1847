"""The gated linear recurrence on the GPU (gdn_linrec_fwd, gdn_linrec_bwd, gdn_linrec_step)
against the plain 64-bit form, element by element, to bounds derived in plain_linrec.py."""
import math

import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from tests import plain_linrec as P

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def make(B, T, D, dtype, *, cu=None, gate=True, given=False, seed=0, fused=False):
    """CPU inputs of one batch (and the views the GPU call gets)."""
    gen = torch.Generator().manual_seed(seed)
    lead = (T,) if cu is not None else (B, T)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    proj = rnd(*lead, 3 * D).to(dtype)
    x, a, b = proj[..., :D], proj[..., D:2 * D], proj[..., 2 * D:]
    A_log = torch.rand(D, generator=gen) * math.log(16.0)
    dt_bias = torch.rand(D, generator=gen) * 3 - 4
    if given:
        a = -A_log.exp() * torch.nn.functional.softplus(a.float() + dt_bias)
        b = torch.sigmoid(b.float())
        A_log = dt_bias = None
    s = dict(x=x, a=a, b=b if gate else None, A_log=A_log, dt_bias=dt_bias, h0=rnd(B, D),
             dh=rnd(*lead, D).to(dtype), dht=rnd(B, D))
    dev = {k: None if v is None else v.contiguous().cuda() for k, v in s.items()}
    if fused and not given:
        p = proj.cuda()
        dev.update(x=p[..., :D], a=p[..., D:2 * D], b=p[..., 2 * D:] if gate else None)
    return s, dev


NAMES = ("x", "a", "b", "A_log", "dt_bias", "h0")


def ins(s, *more):
    return [s[k] for k in NAMES + more]


def check_all(s, d, *, cu=None, scale="none", given=False, wide=False, states=True, bwd=True):
    kw = dict(cu_seqlens=cu, input_scale=scale, gates_precomputed=given)
    pk = dict(cu=cu, scale=scale, given=given)
    n = cu[-1] if cu is not None else None
    cut = (lambda v: v[:n]) if cu is not None else (lambda v: v)
    h, ht, st = G.gdn_linrec_fwd(*ins(d), out_f32=wide, want_states=True, **kw)
    assert h.dtype == (F32 if wide else d["x"].dtype)
    c = {k: (cut(v) if v is not None and k in ("x", "a", "b", "dh") else v) for k, v in s.items()}
    want = P.forward_bounds(*ins(c), **pk)
    P.check("h", cut(h), *want["h"])
    P.check("ht", ht, *want["ht"])
    if not bwd:
        return
    dh = d["dh"].float() if wide else d["dh"]
    grads = G.gdn_linrec_bwd(*ins(d), dh, d["dht"], states=st if states else None, grad_f32=wide,
                             **kw)
    want = P.backward_bounds(*ins(c, "dh", "dht"), **pk)
    assert (grads["db"] is None) == (d["b"] is None)
    for k, (v, e) in want.items():
        got = grads[k] if k in ("dA_log", "ddt_bias", "dh0") else cut(grads[k])
        P.check(k, got, v, e)


@pytest.mark.parametrize("T", [1, 2, 7, 63, 64, 65, 128, 129, 200, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths(T, dtype):
    check_all(*make(2, T, 72, dtype, seed=T), states=T % 2 == 0)


@pytest.mark.parametrize("D", [1, 2, 3, 31, 33, 64, 65, 127, 130, 200])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_widths(D, dtype):
    check_all(*make(3, 133, D, dtype, seed=D))


@pytest.mark.parametrize("scale", ["none", "tied", "unit"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("dtype,wide", [(F32, False), (BF16, False), (BF16, True)])
def test_modes(scale, gate, given, dtype, wide):
    s, d = make(2, 150, 70, dtype, gate=gate, given=given, seed=5)
    check_all(s, d, scale=scale, given=given, wide=wide)
    check_all(s, d, scale=scale, given=given, wide=wide, states=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 96, 37])
def test_slices_of_one_projection(dtype, D):
    check_all(*make(2, 131, D, dtype, fused=True, seed=D))
    cu = [0, 40, 131]
    check_all(*make(2, 131, D, dtype, cu=cu, fused=True, seed=D), cu=cu)


LENGTHS = [[5, 64, 0, 130, 1], [0, 0], [300], [0, 3, 0, 0, 65, 64, 63, 0], [1] * 40]


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_packed(lens, dtype):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s, d = make(len(lens), cu[-1], 66, dtype, cu=cu, seed=len(lens))
    check_all(s, d, cu=cu)
    check_all(s, d, cu=cu, scale="unit", states=False)
    # each sequence bit for bit its own call's
    h, ht = G.gdn_linrec_fwd(*ins(d), cu_seqlens=cu)
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        one = [d[k][None, lo:hi] for k in ("x", "a", "b")]
        h1, ht1 = G.gdn_linrec_fwd(*one, d["A_log"], d["dt_bias"], d["h0"][i:i + 1])
        assert torch.equal(h1[0], h[lo:hi]) and torch.equal(ht1[0], ht[i])


def test_many_packed_sequences():
    lens = [(i * 37) % 90 for i in range(700)]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s, d = make(len(lens), cu[-1], 40, F32, cu=cu, seed=9)
    h, ht = G.gdn_linrec_fwd(*ins(d), cu_seqlens=torch.tensor(cu))
    want = P.forward_bounds(*ins(s), cu=cu)
    P.check("h", h, *want["h"])
    P.check("ht", ht, *want["ht"])


def test_rows_behind_the_last_sequence_stay():
    cu = [0, 70, 75]
    s, d = make(2, 200, 64, BF16, cu=cu, seed=3)
    for k in ("x", "a", "b", "dh"):
        d[k][75:] = float("nan")
    h = torch.full_like(d["x"], 7.0)
    G.gdn_linrec_fwd(*ins(d), cu_seqlens=cu, h=h)
    assert (h[75:] == 7.0).all()
    for k in ("x", "a", "b", "dh"):
        s[k] = s[k][:75]
    P.check("h", h[:75], *P.forward_bounds(*ins(s), cu=cu)["h"])
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], cu_seqlens=cu)
    for k, (v, e) in P.backward_bounds(*ins(s, "dh", "dht"), cu=cu).items():
        P.check(k, g[k] if k in ("dA_log", "ddt_bias", "dh0") else g[k][:75], v, e)


def test_no_states_given_and_none_wanted():
    s, d = make(2, 100, 50, F32, seed=1)
    d["h0"] = s["h0"] = None
    h, ht = G.gdn_linrec_fwd(*ins(d), want_ht=False)
    assert ht is None
    P.check("h", h, *P.forward_bounds(*ins(s))["h"])
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], None, want_dh0=False)
    assert g["dh0"] is None
    s["dht"] = None
    want = P.backward_bounds(*ins(s, "dh", "dht"))
    for k in ("dx", "da", "db", "dA_log", "ddt_bias"):
        P.check(k, g[k], *want[k])


def test_empty():
    s, d = make(3, 0, 20, F32)
    h, ht = G.gdn_linrec_fwd(*ins(d))
    assert h.shape == (3, 0, 20) and torch.equal(ht, d["h0"])
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"])
    assert torch.equal(g["dh0"], d["dht"]) and not g["dA_log"].any() and not g["ddt_bias"].any()
    s, d = make(0, 9, 20, F32)
    h, ht = G.gdn_linrec_fwd(*ins(d))
    assert h.shape == (0, 9, 20) and ht.shape == (0, 20)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(dtype):
    _, d = make(2, 300, 136, dtype, seed=4)
    h, ht = G.gdn_linrec_fwd(*ins(d))
    x, st = d["x"].clone(), d["h0"].clone()
    d2 = dict(d, x=x, h0=st)
    h2, ht2 = G.gdn_linrec_fwd(*ins(d2), h=x, ht=st)
    assert h2 is x and ht2 is st and torch.equal(h2, h) and torch.equal(ht2, ht)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_continued_in_pieces(dtype):
    """Chunk-aligned pieces with the state carried are bit for bit the whole call."""
    _, d = make(2, 320, 70, dtype, seed=6)
    h, ht = G.gdn_linrec_fwd(*ins(d), out_f32=True)
    st, outs = d["h0"], []
    for lo, hi in ((0, 64), (64, 256), (256, 320)):
        part = [d[k][:, lo:hi].contiguous() for k in ("x", "a", "b")]
        o, st = G.gdn_linrec_fwd(*part, d["A_log"], d["dt_bias"], st, out_f32=True)
        outs.append(o)
    assert torch.equal(torch.cat(outs, 1), h) and torch.equal(st, ht)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale,gate,given", [("none", True, False), ("tied", False, False),
                                              ("unit", True, True)])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 37), (5, 128), (300, 264), (1, 4096)])
def test_step(dtype, scale, gate, given, N, D):
    s, d = make(N, 1, D, dtype, gate=gate, given=given, seed=N)
    want = P.forward_bounds(*ins(s), scale=scale, given=given)
    state = d["h0"].clone()
    one = [None if d[k] is None else d[k][:, 0] for k in ("x", "a", "b")]
    h = G.gdn_linrec_step(*one, d["A_log"], d["dt_bias"], state, input_scale=scale,
                          gates_precomputed=given)
    P.check("h", h, want["h"][0][:, 0], want["h"][1][:, 0])
    P.check("state", state, *want["ht"])


def test_step_strided_and_in_place():
    s, d = make(6, 1, 64, BF16, fused=True, seed=2)
    want = P.forward_bounds(*ins(s))
    one = [d[k][:, 0] for k in ("x", "a", "b")]
    h = G.gdn_linrec_step(*one, d["A_log"], d["dt_bias"], d["h0"], h=one[0])
    assert h.data_ptr() == d["x"].data_ptr()
    P.check("h", h, want["h"][0][:, 0], want["h"][1][:, 0])


def test_steps_continue_a_prefill():
    s, d = make(4, 140, 48, F32, seed=8)
    want = P.forward_bounds(*ins(s))
    cut = [d[k][:, :130].contiguous() for k in ("x", "a", "b")]
    _, st = G.gdn_linrec_fwd(*cut, d["A_log"], d["dt_bias"], d["h0"])
    for t in range(130, 140):
        one = [d[k][:, t] for k in ("x", "a", "b")]
        h = G.gdn_linrec_step(*one, d["A_log"], d["dt_bias"], st)
        P.check(f"h[{t}]", h, want["h"][0][:, t], want["h"][1][:, t])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extreme_gates(dtype):
    """Logits at which softplus or the sigmoid saturate, both infinities, slow and fast
    channels: the definitions' limits, no NaN."""
    s, d = make(1, 130, 64, dtype, seed=7)
    big = torch.tensor([-200.0, -80.0, -20.0, -8.0, 0.0, 30.0, 200.0, float("inf"),
                        float("-inf")])
    for k in ("a", "b"):
        v = s[k].clone()
        v[0, :, :9] = big.to(dtype)
        v[0, 64:70] = big[3].to(dtype)
        s[k] = v
        d[k] = v.cuda()
    for scale in ("none", "tied", "unit"):
        h, ht = G.gdn_linrec_fwd(*ins(d), input_scale=scale)
        g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], input_scale=scale)
        for k, v in [("h", h), ("ht", ht), *g.items()]:
            assert torch.isfinite(v).all(), (scale, k)
        fin = torch.isfinite(s["a"][0, 0].float())
        c = {k: (v[..., fin] if v is not None else None) for k, v in s.items()}
        want = P.forward_bounds(*ins(c), scale=scale)
        P.check("h", h[..., fin.cuda()], *want["h"])
        for k, (v, e) in P.backward_bounds(*ins(c, "dh", "dht"), scale=scale).items():
            P.check(f"{scale} {k}", g[k][..., fin.cuda()], v, e)


def test_nan_stays_in_its_channel_and_behind_it():
    _, d = make(2, 200, 70, F32, seed=11)
    h, ht = G.gdn_linrec_fwd(*ins(d))
    d["x"] = d["x"].clone()
    d["x"][1, 100, 33] = float("nan")
    h2, ht2 = G.gdn_linrec_fwd(*ins(d))
    bad = torch.isnan(h2)
    assert bad[1, 100:, 33].all() and int(bad.sum()) == 100 and torch.isnan(ht2).sum() == 1
    assert torch.equal(h2[~bad], h[~bad])


def test_gradients_against_differences():
    """sum(h R) + sum(ht S) along a direction: central differences of the float32 output (the
    64-bit form gives both values; the kernel's gradients give the slope)."""
    s, d = make(2, 90, 20, F32, seed=12)
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], input_scale="unit")
    gen = torch.Generator().manual_seed(1)

    def value(eps, name, v):
        t = {k: None if x is None else x.double() for k, x in s.items()}
        t[name] = t[name] + eps * v
        h, ht = P.recurrence(*ins(t), scale="unit")
        return float((h * t["dh"]).sum() + (ht * t["dht"]).sum())

    want = P.backward_bounds(*ins(s, "dh", "dht"), scale="unit")
    for name in NAMES:
        v = torch.randn(s[name].shape, generator=gen, dtype=torch.float64)
        slope = (value(1e-6, name, v) - value(-1e-6, name, v)) / 2e-6
        got = float((g["d" + name].cpu().double() * v).sum())
        # the gradients' bound, and 1e-7 of the terms for the difference itself
        lim = float((want["d" + name][1] * v.abs()).sum()) + 1e-7 * float(
            (want["d" + name][0] * v).abs().sum() + 1)
        lim += 2.0 ** -24 * float((want["d" + name][0] * v).abs().sum())
        assert abs(got - slope) <= lim, (name, got, slope, lim)


def test_same_bits_every_time_and_from_two_streams():
    _, d = make(1, 5000, 200, BF16, seed=13)
    h, ht, st = G.gdn_linrec_fwd(*ins(d), want_states=True)
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], states=st)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(10):
        s = streams[i % 2]
        h2, ht2, st2 = G.gdn_linrec_fwd(*ins(d), want_states=True, stream=s)
        got.append((h2, ht2, st2, G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], states=st2,
                                                   stream=s)))
    torch.cuda.synchronize()
    for h2, ht2, st2, g2 in got:
        assert torch.equal(h, h2) and torch.equal(ht, ht2) and torch.equal(st, st2)
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_captured_and_replayed():
    s, d = make(2, 777, 130, BF16, seed=14)
    ws = torch.empty(max(1, G.gdn_linrec_workspace_bytes(2, 777, 130)), dtype=torch.uint8,
                     device="cuda").fill_(255)
    wb = torch.empty(max(1, G.gdn_linrec_bwd_workspace_bytes(2, 777, 130)), dtype=torch.uint8,
                     device="cuda").fill_(255)

    def step():
        h, ht = G.gdn_linrec_fwd(*ins(d), workspace=ws)
        g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], workspace=wb)
        return [h, ht, *(g[k] for k in sorted(g))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    second = torch.cuda.CUDAGraph()  # another graph on the same workspaces
    with torch.cuda.graph(second):
        outs2 = step()
    for seed in (21, 22):
        _, e = make(2, 777, 130, BF16, seed=seed)
        for k in d:
            d[k].copy_(e[k])
        graph.replay()
        second.replay()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert all(torch.equal(o, w) for o, w in zip(outs2, want))


def test_workspace_needs_no_initialisation_and_is_checked():
    _, d = make(2, 300, 100, F32, seed=15)
    h, ht = G.gdn_linrec_fwd(*ins(d))
    need = G.gdn_linrec_workspace_bytes(2, 300, 100)
    if need:
        for fill in (0, 1, 2, 255):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            h2, ht2 = G.gdn_linrec_fwd(*ins(d), workspace=ws)
            assert torch.equal(h, h2) and torch.equal(ht, ht2)
        with pytest.raises(G.GDNError):
            G.gdn_linrec_fwd(*ins(d), workspace=ws[:need - 1])
    wb = torch.empty(G.gdn_linrec_bwd_workspace_bytes(2, 300, 100), dtype=torch.uint8,
                     device="cuda")
    with pytest.raises(G.GDNError):
        G.gdn_linrec_bwd(*ins(d), d["dh"], workspace=wb[:-1])


def test_long_narrow_and_wide():
    """A long sequence of few channels (many chunks in flight) and a wide short one, on a
    sample of channels."""
    for B, T, D, dtype in ((1, 20000, 8, F32), (1, 300, 6000, BF16), (70, 3, 100, F32)):
        s, d = make(B, T, D, dtype, seed=T)
        h, ht, st = G.gdn_linrec_fwd(*ins(d), want_states=True)
        g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], states=st)
        at = torch.arange(0, D, max(1, D // 12))
        c = {k: v[..., at] for k, v in s.items()}
        want = {**P.forward_bounds(*ins(c)), **P.backward_bounds(*ins(c, "dh", "dht"))}
        for k, (v, e) in want.items():
            got = {"h": h, "ht": ht}.get(k, g.get(k))
            P.check(f"{T}x{D} {k}", got.cpu()[..., at], v, e)


def test_refused_tensors():
    _, d = make(2, 20, 16, F32)
    ok = ins(d)
    with pytest.raises(ValueError):  # broadcast
        G.gdn_linrec_fwd(d["x"][:, :1].expand(2, 20, 16), *ok[1:])
    with pytest.raises(ValueError):  # channels not contiguous
        G.gdn_linrec_fwd(d["x"].transpose(1, 2).contiguous().transpose(1, 2), *ok[1:])
    with pytest.raises(ValueError):  # rows of the batch not a fixed distance apart
        G.gdn_linrec_fwd(torch.zeros(2, 30, 16, device="cuda")[:, :20], *ok[1:])
    with pytest.raises(ValueError):
        G.gdn_linrec_fwd(d["x"].cpu(), *ok[1:])
    with pytest.raises(ValueError):
        G.gdn_linrec_fwd(d["x"], d["a"].cpu(), *ok[2:])
    with pytest.raises(TypeError):
        G.gdn_linrec_fwd(d["x"], d["a"].bfloat16(), *ok[2:])
    with pytest.raises(ValueError):
        G.gdn_linrec_fwd(*ok, input_scale="both")
    with pytest.raises(ValueError):
        G.gdn_linrec_fwd(*ok, cu_seqlens=[0, 20])  # [B, T, D] is not packed
    packed = [v[0] for v in ok[:3]] + ok[3:5] + [d["h0"][:1]]
    for cu in ([0, 21], [1, 20], [0, 21, 20]):
        with pytest.raises((G.GDNError, ValueError)):
            G.gdn_linrec_fwd(*packed[:5], None, cu_seqlens=cu)
    with pytest.raises(TypeError):
        G.gdn_linrec_fwd(d["x"].half(), d["a"].half(), None, *ok[3:])
    with pytest.raises(ValueError):
        G.gdn_linrec_bwd(*ok, d["dh"], d["dht"], states=torch.zeros(1, 16, device="cuda"))


@pytest.mark.parametrize("T", [300, 5000])
def test_an_expired_wait_is_reported(T):
    """The first block of each cluster keeps its chunks' results to itself: the waits of the
    others end and say so, in one round or over several, and the next call is right again."""
    _, d = make(2, T, 70, F32, seed=16)
    h, ht, st = G.gdn_linrec_fwd(*ins(d), want_states=True)
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], states=st)
    torch.cuda.synchronize()
    try:
        G.gdn_test_set_wait_fault(3, 1 << 10)
        G.gdn_linrec_fwd(*ins(d))
        assert G.gdn_status() == -4
        G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], states=st)
        assert G.gdn_status() == -4
    finally:
        G.gdn_test_set_wait_fault(0, 0)
    h2, ht2 = G.gdn_linrec_fwd(*ins(d))
    g2 = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], states=st)
    assert torch.equal(h, h2) and torch.equal(ht, ht2)
    assert all(torch.equal(g[k], g2[k]) for k in g)
