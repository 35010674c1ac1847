"""The gated linear recurrence and the norm-and-rotation of q and k without a GPU: argument
errors found on the host, the workspace sizes, and the plain 64-bit forms the GPU tests compare
with (their gradients against differences and against autograd)."""
import ctypes
import math

import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from tests import plain_linrec as P

FAKE = 0x10000
L = G.lib


def offsets(*v):
    return (ctypes.c_longlong * len(v))(*v)


def fwd(**kw):
    a = dict(x=FAKE, a=FAKE, b=FAKE, A=FAKE, t=FAKE, h0=None, cu=None, B=2, T=100, D=64, ldx=64,
             lda=64, ldb=64, dtype=1, flags=0, h=FAKE, ldh=64, ht=None, st=None, ws=FAKE, n=0)
    a.update(kw)
    return L.gdn_linrec_fwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(a=None), dict(h=None), dict(A=None), dict(t=None), dict(x=FAKE + 1),
    dict(h0=FAKE + 2), dict(ht=FAKE + 1), dict(st=FAKE + 2), dict(B=-1), dict(T=-1), dict(D=0),
    dict(dtype=2), dict(flags=1), dict(flags=64), dict(flags=8 | 16), dict(flags=32),
    dict(ldx=63), dict(lda=0), dict(ldb=-64), dict(ldh=63), dict(a=FAKE + 2, flags=2),
    dict(cu=offsets(0, 50, 101)), dict(cu=offsets(1, 50, 100)), dict(cu=offsets(0, 60, 50)),
    dict(dtype=0, x=FAKE + 2),
])
def test_forward_rejects(kw):
    assert fwd(**kw) == -1


def test_forward_limits():
    assert fwd(T=2 ** 31 - 1, D=2 ** 20, ldx=2 ** 20, lda=2 ** 20, ldb=2 ** 20, ldh=2 ** 20) == -2
    for kw in (dict(T=2 ** 30 + 1), dict(D=2 ** 21 + 1, ldx=2 ** 22, lda=2 ** 22, ldb=2 ** 22),
               dict(ldx=2 ** 21 + 1), dict(lda=2 ** 30), dict(ldb=2 ** 40), dict(ldh=2 ** 22),
               dict(B=2 ** 30, T=1)):
        assert fwd(**kw) == -2, kw
    need = G.gdn_linrec_workspace_bytes(2, 100, 64)
    assert need == 0  # only packed batches take one
    cu = offsets(0, 40, 100)
    need = L.gdn_linrec_workspace_bytes(cu, 2, 100, 64)
    assert need > 0
    for ws, n in ((FAKE, need - 1), (None, need), (FAKE + 8, need)):
        assert fwd(cu=cu, ws=ws, n=n) == -5
    assert fwd(B=0, cu=None) == 0                      # no sequence, nothing to write
    assert fwd(B=2, T=0, x=None, a=None, h=None) == 0  # no token, no final state wanted


def bwd(**kw):
    a = dict(x=FAKE, a=FAKE, b=FAKE, A=FAKE, t=FAKE, h0=None, cu=None, B=2, T=100, D=64, ldx=64,
             lda=64, ldb=64, dh=FAKE, lddh=64, dht=None, st=FAKE, dtype=1, flags=0, dx=FAKE,
             lddx=64, da=FAKE, ldda=64, db=FAKE, lddb=64, dA=FAKE, dt=FAKE, dh0=None, ws=FAKE,
             n=0)
    a.update(kw)
    return L.gdn_linrec_bwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(dh=None), dict(dx=None), dict(da=None), dict(db=None), dict(b=None), dict(dA=None),
    dict(dt=None), dict(dA=FAKE + 2), dict(lddh=1), dict(lddx=63), dict(ldda=63), dict(lddb=63),
    dict(dht=FAKE + 2), dict(dh0=FAKE + 2), dict(st=FAKE + 2), dict(flags=4), dict(flags=32,
    dx=FAKE + 2), dict(flags=2, da=FAKE + 2), dict(flags=24),
])
def test_backward_rejects(kw):
    assert bwd(**kw) == -1


def test_backward_workspace():
    assert bwd() == -5
    more = G.gdn_linrec_bwd_workspace_bytes(2, 100, 64)
    less = G.gdn_linrec_bwd_workspace_bytes(2, 100, 64, states_given=True)
    assert more > less > 0
    assert bwd(st=None, n=less) == -5
    assert G.gdn_linrec_bwd_workspace_bytes(0, 100, 64) == 0
    assert G.gdn_linrec_workspace_bytes(2, 100, 0) == 0


def step(**kw):
    a = dict(x=FAKE, a=FAKE, b=FAKE, A=FAKE, t=FAKE, st=FAKE, N=3, D=64, ldx=64, lda=64, ldb=64,
             dtype=1, flags=0, h=FAKE, ldh=64)
    a.update(kw)
    return L.gdn_linrec_step(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(st=None), dict(h=None), dict(st=FAKE + 2), dict(N=-1), dict(D=-3),
    dict(flags=32), dict(flags=24), dict(ldh=3), dict(ldx=3), dict(dtype=9), dict(A=None),
    dict(h=FAKE + 2, flags=4),
])
def test_step_rejects(kw):
    assert step(**kw) == -1


def test_step_of_nothing():
    assert step(N=0) == 0


def rope(**kw):
    a = dict(q=FAKE, k=FAKE, pos=FAKE, f=FAKE, qw=None, kw=None, n=5, Hq=4, Hk=2, d=64, rot=64,
             ldq=256, ldk=128, dtype=1, flags=64, eps=1e-6, scale=1.0, qo=FAKE, ldqo=256, ko=FAKE,
             ldko=128)
    a.update(kw)
    return L.gdn_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(pos=None), -1), (dict(pos=FAKE + 4), -1),
    (dict(f=None), -1), (dict(rot=63), -1), (dict(rot=66), -1), (dict(rot=-2), -1),
    (dict(ldq=255), -1), (dict(ldk=127), -1), (dict(ldqo=1), -1), (dict(ldko=1), -1),
    (dict(qo=None), -1), (dict(ko=FAKE + 1), -1), (dict(eps=-1.0), -1), (dict(eps=2.0), -1),
    (dict(eps=float("nan")), -1), (dict(flags=65), -1), (dict(flags=2), -1), (dict(n=-1), -1),
    (dict(Hq=-1), -1), (dict(flags=1, qw=FAKE), -1), (dict(qw=FAKE + 2), -1), (dict(d=0), -1),
    (dict(dtype=5), -1), (dict(d=257, ldq=2000, ldk=2000, ldqo=2000, ldko=2000), -2),
    (dict(n=0, q=None, k=None), 0), (dict(Hq=0, Hk=0), 0), (dict(flags=32), -1),
])
def test_rope_rejects(kw, code):
    assert rope(**kw) == code


def test_rope_backward_rejects():
    def bwd(**kw):
        a = dict(q=FAKE, k=FAKE, pos=FAKE, f=FAKE, qw=FAKE, kw=FAKE, n=5, Hq=4, Hk=2, d=64,
                 rot=64, ldq=256, ldk=128, gq=FAKE, ldgq=256, gk=FAKE, ldgk=128, dtype=1,
                 flags=64, eps=1e-6, scale=1.0, dq=FAKE, lddq=256, dk=FAKE, lddk=128, dqw=FAKE,
                 dkw=FAKE, ws=None, n2=0)
        a.update(kw)
        return L.gdn_qk_norm_rope_bwd(*a.values(), None)
    assert bwd() == -5
    for kw in (dict(gq=None), dict(gk=FAKE + 1), dict(ldgq=2), dict(dq=None), dict(lddk=4),
               dict(dqw=FAKE + 1), dict(flags=1), dict(flags=64 | 4)):
        assert bwd(**kw) == -1
    assert G.gdn_qk_norm_rope_bwd_workspace_bytes(5, 4, 2, 64) > 0
    assert G.gdn_qk_norm_rope_bwd_workspace_bytes(5, 4, 2, 64, "l2") == 0
    assert G.gdn_qk_norm_rope_bwd_workspace_bytes(0, 4, 2, 64) == 0


def test_tensors_of_the_host_are_refused():
    x = torch.zeros(1, 4, 8)
    w = torch.zeros(8)
    with pytest.raises(ValueError):
        G.gdn_linrec_fwd(x, x, x, w, w)
    with pytest.raises(ValueError):
        G.gdn_linrec_bwd(x, x, x, w, w, None, x)
    with pytest.raises(ValueError):
        G.gdn_linrec_step(x[0], x[0], None, w, w, x[0])
    with pytest.raises(ValueError):
        G.gdn_qk_norm_rope(x, x, torch.zeros(1), None)


def test_chunks():
    assert G.gdn_linrec_chunks(3, 65) == 6 and G.gdn_linrec_chunks(2, 0) == 0
    assert G.gdn_linrec_chunks(0, 0, [0, 5, 5, 134]) == 4
    assert G.gdn_linrec_chunks(0, 0, torch.tensor([0, 64])) == 1


# ---- the plain forms --------------------------------------------------------------------------


def inputs(B, T, D, cu=None, given=False):
    gen = torch.Generator().manual_seed(T)
    lead = (T,) if cu else (B, T)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    s = dict(x=r(*lead, D), a=r(*lead, D), b=r(*lead, D),
             A_log=r(D), dt_bias=r(D) - 2, h0=r(B, D))
    if given:
        s.update(a=-s["a"].exp() - 1e-3, b=torch.sigmoid(s["b"]), A_log=None, dt_bias=None)
    return s, r(*lead, D), r(B, D)


@pytest.mark.parametrize("scale", ["none", "tied", "unit"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 9]])
def test_plain_recurrence(scale, given, cu):
    """The formulas' gradients are autograd's, and those are the differences'."""
    B = 3 if cu else 2
    s, dh, dht = inputs(B, 9, 4, cu, given)
    kw = dict(cu=cu, scale=scale, given=given)
    names = [k for k in s if s[k] is not None]
    leaf = {k: s[k].clone().requires_grad_(True) for k in names}

    def f(*v):
        t = dict(s, **dict(zip(names, v)))
        return P.recurrence(*t.values(), **kw)

    assert torch.autograd.gradcheck(f, [leaf[k] for k in names], atol=1e-6)
    h, ht = f(*leaf.values())
    vb = P.forward_bounds(*s.values(), **kw)
    assert torch.allclose(vb["h"][0], h, rtol=1e-12, atol=0)
    assert torch.allclose(vb["ht"][0], ht, rtol=1e-12, atol=0)
    got = torch.autograd.grad([h, ht], [leaf[k] for k in names], [dh, dht])
    want = P.backward_bounds(*s.values(), dh, dht, **kw)
    for k, g in zip(names, got):
        assert torch.allclose(want["d" + k][0], g, rtol=1e-9, atol=1e-11), k
    # the definition itself, one channel by hand
    g, alpha, beta, f1 = P.gates(s["a"], s["b"], s["A_log"], s["dt_bias"], scale, given)
    seq = (slice(3, 9),) if cu else (1, slice(0, 9))
    cur = float(s["h0"][-1, 2])
    for t in range(alpha[seq].shape[0]):
        al = math.exp(float(g[seq][t, 2]))
        sc = {"none": 1.0, "tied": 1 - al, "unit": math.sqrt(1 - al * al)}[scale]
        cur = al * cur + sc * float(beta[seq][t, 2]) * float(s["x"][seq][t, 2])
        assert abs(cur - float(h.detach()[seq][t, 2])) < 1e-12 * max(1.0, abs(cur))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
def test_plain_rotation(interleaved, norm):
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(5, 2, 10, generator=gen, dtype=torch.float64)
    w = torch.rand(10, generator=gen, dtype=torch.float64) + 0.5
    f = torch.tensor([1.0, 0.3, 0.01])
    pos = torch.arange(5)
    y = P.norm_rope(x, pos, f, w, norm=norm, interleaved=interleaved)
    base = P.norm_rope(x, pos * 0, f, w, norm=norm, interleaved=interleaved)
    # a rotation of each pair: lengths kept, position 0 is no rotation, and the product of two
    # rows depends on the distance of their positions alone
    assert torch.allclose(y.square().sum(-1), base.square().sum(-1), rtol=1e-12)
    assert torch.allclose(y[..., 6:], base[..., 6:])
    assert torch.allclose(y[0], base[0])
    z = P.norm_rope(x, pos + 40, f, w, norm=norm, interleaved=interleaved)
    one = P.norm_rope(x.flip(0), pos.flip(0), f, w, norm=norm, interleaved=interleaved)
    two = P.norm_rope(x.flip(0), pos.flip(0) + 40, f, w, norm=norm, interleaved=interleaved)
    assert torch.allclose((y * one).sum(-1), (z * two).sum(-1), rtol=1e-9, atol=1e-9)
    leaf = [x.requires_grad_(True), w.requires_grad_(True)]
    assert torch.autograd.gradcheck(
        lambda a, b: P.norm_rope(a, pos, f, b, norm=norm, interleaved=interleaved, scale=0.3),
        leaf, atol=1e-6)
