"""Norm and rotation of q and k on the GPU (gdn_qk_norm_rope and its backward) against the
plain 64-bit form.

Bounds, u = 2^-24.  The norm's factor is one float32 sum of d squares (pairwise over lanes: at
most (d / 8 + 5) roundings deep at d <= 256, taken as 40 u), one root and reciprocal (4 u); the
weight, scale and rotation add a few roundings and the angle 2^-22 rad, each relative to the
length of the value's pair: 64 u of it in all.  The backward has the same factors twice and a
second sum whose terms are bounded by their absolute values: 160 u of them."""
import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from tests import plain_linrec as P

pytestmark = pytest.mark.gpu
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
U = P.U


def make(T, Hq, Hk, d, rot, dtype, *, seed=0, far=5000, theta=1e4, fused=False, weights=True):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    qkv = rnd(T, (Hq + 2 * Hk) * d).to(dtype)
    s = dict(q=qkv[:, :Hq * d].unflatten(1, (Hq, d)) if Hq else None,
             k=qkv[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)) if Hk else None,
             pos=torch.randint(0, far, (T,), generator=gen),
             inv_freq=(theta ** (-torch.arange(0, rot, 2, dtype=F64) / max(rot, 1))).float(),
             qw=torch.rand(d, generator=gen) + 0.5 if weights else None,
             kw=torch.rand(d, generator=gen) + 0.5 if weights else None,
             dq=rnd(T, Hq, d).to(dtype) if Hq else None,
             dk=rnd(T, Hk, d).to(dtype) if Hk else None)
    dev = {k: None if v is None else v.contiguous().cuda() for k, v in s.items()}
    if fused:
        p = qkv.cuda()
        dev["q"] = p[:, :Hq * d].unflatten(1, (Hq, d))
        dev["k"] = p[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    return s, dev


def args(s, *more):
    return [s[k] for k in ("q", "k", "pos", "inv_freq", "qw", "kw") + more]


def check(s, d, *, norm="rms", eps=1e-6, scale=1.0, interleaved=False, bwd=True, wide=False):
    kw = dict(norm=norm, eps=eps, scale=scale, interleaved=interleaved)
    rot = 0 if s["inv_freq"] is None else 2 * s["inv_freq"].numel()
    if norm != "rms":
        s, d = dict(s, qw=None, kw=None), dict(d, qw=None, kw=None)
    outs = G.gdn_qk_norm_rope(*args(d), **kw)
    for name, got, sc in (("q", outs[0], scale), ("k", outs[1], 1.0)):
        if s[name] is None:
            assert got is None
            continue
        y = P.norm_rope(s[name], s["pos"], s["inv_freq"], s[name + "w"],
                        **dict(kw, scale=sc))
        P.check(name, got, y, 64 * U * P.rope_pair_size(y, rot, interleaved))
    if not bwd:
        return
    gd = {k: None if d[k] is None else (d[k].float() if wide else d[k]) for k in ("dq", "dk")}
    grads = G.gdn_qk_norm_rope_bwd(*args(d), gd["dq"], gd["dk"], grad_f32=wide, **kw)
    for name, sc in (("q", scale), ("k", 1.0)):
        if s[name] is None:
            assert grads["d" + name] is None
            continue
        x = s[name].to(F64).requires_grad_(True)
        w = s[name + "w"]
        w = torch.ones(x.shape[-1], dtype=F64) if w is None else w.to(F64)
        w = w.requires_grad_(True)
        y = P.norm_rope(x, s["pos"], s["inv_freq"], w, **dict(kw, scale=sc))
        dx, dw = torch.autograd.grad(y, [x, w], s["d" + name].to(F64))
        # magnitudes: the rotated gradient by its pair's length, its share along n by the sum
        xd = x.detach()
        red = xd.square().mean(-1, keepdim=True) if norm == "rms" else \
            xd.square().sum(-1, keepdim=True)
        inv = 1 / torch.sqrt(red + eps) if norm in ("rms", "l2") else torch.ones_like(red)
        n = (xd * inv).abs()
        dy = P.rope_pair_size(s["d" + name].to(F64), rot, interleaved) * abs(sc)
        dn = dy * w.detach().abs()
        dot = (n * dn).mean(-1, keepdim=True) if norm == "rms" else \
            (n * dn).sum(-1, keepdim=True)
        mag = inv * (dn + n * dot) if norm in ("rms", "l2") else dn
        P.check("d" + name, grads["d" + name], dx, 160 * U * mag)
        if s[name + "w"] is not None:
            P.check("d" + name + "w", grads["d" + name + "_weight"], dw,
                    160 * U * (dy * n).sum((0, 1)))
        else:
            assert grads["d" + name + "_weight"] is None


@pytest.mark.parametrize("d", [1, 2, 6, 8, 40, 63, 64, 80, 96, 100, 128, 130, 192, 255, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes(d, dtype, interleaved):
    check(*make(9, 3, 2, d, d // 2 * 2, dtype, seed=d), interleaved=interleaved, scale=0.3)


@pytest.mark.parametrize("rot", [0, 2, 14, 16, 32, 62, 64, 96, 128])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
@pytest.mark.parametrize("interleaved", [False, True])
def test_partial_rotation(rot, norm, interleaved):
    for dtype in (F32, BF16):
        check(*make(7, 4, 1, 128, rot, dtype, seed=rot), norm=norm, interleaved=interleaved,
              scale=128 ** -0.5)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 2), (2, 5, 1), (300, 3, 3), (5000, 2, 1),
                                     (3, 7, 0), (3, 0, 4), (1, 64, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_and_heads(T, Hq, Hk, dtype):
    check(*make(T, Hq, Hk, 64, 64, dtype, seed=T))


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("d,Hq,Hk", [(64, 4, 2), (128, 2, 2), (256, 8, 1), (36, 3, 1)])
def test_slices_and_float32_gradients(fused, d, Hq, Hk):
    for dtype in (F32, BF16):
        check(*make(50, Hq, Hk, d, d // 4 * 2, dtype, seed=d, fused=fused), wide=True)


@pytest.mark.parametrize("theta", [1e4, 1e7])
def test_far_and_negative_positions(theta):
    """The angle stays exact where float32 products would not: up to a million tokens."""
    s, d = make(400, 2, 1, 64, 64, F32, far=1 << 20, theta=theta, seed=1)
    s["pos"][:5] = torch.tensor([-1, -77777, (1 << 20), 0, 1])
    d["pos"].copy_(s["pos"])
    check(s, d)


def test_batched_and_in_place():
    s, d = make(24, 2, 2, 128, 128, BF16, seed=3)
    q, k = G.gdn_qk_norm_rope(*args(d), scale=0.5)
    b = {n: d[n].reshape(4, 6, *d[n].shape[1:]) for n in ("q", "k", "pos")}
    qb, kb = G.gdn_qk_norm_rope(b["q"], b["k"], b["pos"], *args(d)[3:], scale=0.5)
    assert torch.equal(qb.flatten(0, 1), q) and torch.equal(kb.flatten(0, 1), k)
    q2, k2 = G.gdn_qk_norm_rope(*args(d), scale=0.5, q_out=d["q"], k_out=d["k"])
    assert q2 is d["q"] and torch.equal(q2, q) and torch.equal(k2, k)


def test_zero_rows():
    """A head of zeros: eps alone under the root, a finite gradient."""
    s, d = make(5, 2, 2, 64, 64, F32, seed=4)
    for n in ("q", "k"):
        s[n] = s[n].clone()
        s[n][2] = 0
        d[n][2] = 0
    check(s, d)
    check(s, d, norm="l2")


def test_nan_stays_in_its_head():
    _, d = make(6, 3, 1, 128, 128, F32, seed=5)
    q, k = G.gdn_qk_norm_rope(*args(d))
    d["q"] = d["q"].clone()
    d["q"][2, 1, 7] = float("nan")
    q2, k2 = G.gdn_qk_norm_rope(*args(d))
    bad = torch.isnan(q2)
    assert bad[2, 1].all() and int(bad.sum()) == 128
    assert torch.equal(q2[~bad], q[~bad]) and torch.equal(k2, k)
    _, d = make(6, 3, 1, 64, 32, F32, seed=5, weights=False)
    d["q"][3, 2, 40] = float("inf")  # behind the rotated channels, no norm
    q2, _ = G.gdn_qk_norm_rope(*args(d), norm=None)
    assert int((~torch.isfinite(q2)).sum()) == 1


def test_empty():
    _, d = make(0, 2, 1, 64, 64, F32)
    q, k = G.gdn_qk_norm_rope(*args(d))
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    g = G.gdn_qk_norm_rope_bwd(*args(d, "dq", "dk"))
    assert g["dq"].shape == (0, 2, 64) and not g["dq_weight"].any()


def test_same_bits_streams_and_graphs():
    _, d = make(3000, 4, 2, 128, 64, BF16, seed=6)
    first = G.gdn_qk_norm_rope_bwd(*args(d, "dq", "dk"))
    q, k = G.gdn_qk_norm_rope(*args(d))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [G.gdn_qk_norm_rope_bwd(*args(d, "dq", "dk"), stream=side) for _ in range(5)]
    q2, k2 = G.gdn_qk_norm_rope(*args(d), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(k, k2)
    for g in got:
        assert all(torch.equal(first[n], g[n]) for n in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q3, _ = G.gdn_qk_norm_rope(*args(d))
        g3 = G.gdn_qk_norm_rope_bwd(*args(d, "dq", "dk"))
    for _ in range(2):
        d["pos"].add_(17)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q3, G.gdn_qk_norm_rope(*args(d))[0])
        g = G.gdn_qk_norm_rope_bwd(*args(d, "dq", "dk"))
        assert all(torch.equal(g3[n], g[n]) for n in g)


def test_gradients_against_differences():
    s, d = make(6, 2, 1, 40, 20, F32, seed=7)
    g = G.gdn_qk_norm_rope_bwd(*args(d, "dq", "dk"), scale=0.7)
    gen = torch.Generator().manual_seed(2)
    for name, sc in (("q", 0.7), ("k", 1.0)):
        for what in (name, name + "w"):
            v = torch.randn(s[what].shape, generator=gen, dtype=F64)

            def value(eps):
                t = {n: s[n].to(F64) for n in (name, name + "w")}
                t[what] = t[what] + eps * v
                y = P.norm_rope(t[name], s["pos"], s["inv_freq"], t[name + "w"], scale=sc)
                return float((y * s["d" + name].to(F64)).sum())

            slope = (value(1e-5) - value(-1e-5)) / 2e-5
            got = g["d" + name if what == name else f"d{name}_weight"].cpu().to(F64)
            lim = 1e-6 * float((got * v).abs().sum() + 1)
            assert abs(float((got * v).sum()) - slope) <= lim, (what, slope)


def test_refused_tensors():
    _, d = make(4, 2, 1, 64, 64, F32)
    q, k, pos, f, qw, kw = args(d)
    with pytest.raises(ValueError):
        G.gdn_qk_norm_rope(q, k, pos[:3], f, qw, kw)
    with pytest.raises(TypeError):
        G.gdn_qk_norm_rope(q, k, pos.int(), f, qw, kw)
    with pytest.raises(TypeError):
        G.gdn_qk_norm_rope(q, k, pos, f.double(), qw, kw)
    with pytest.raises(ValueError):
        G.gdn_qk_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, pos, f, qw, kw)
    with pytest.raises(ValueError):
        G.gdn_qk_norm_rope(q[:1].expand(4, 2, 64), k, pos, f, qw, kw)
    with pytest.raises(ValueError):
        G.gdn_qk_norm_rope(q, k, pos, f, qw, kw, norm="layer")
    with pytest.raises(G.GDNError):  # weights belong to the RMS norm
        G.gdn_qk_norm_rope(q, k, pos, f, qw, kw, norm="l2")
    with pytest.raises(G.GDNError):  # more rotated channels than the head has
        G.gdn_qk_norm_rope(q, k, pos, torch.ones(40, device="cuda"), qw, kw)
    with pytest.raises(G.GDNError):
        G.gdn_qk_norm_rope(torch.zeros(2, 1, 300, device="cuda"), None, pos[:2], None, norm=None)
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(G.GDNError):
        G.gdn_qk_norm_rope_bwd(q, k, pos, f, qw, kw, d["dq"], d["dk"], workspace=ws)
