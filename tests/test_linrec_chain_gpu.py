"""The gated linear recurrence, the norm-and-rotation and the delta rule together, as a mixing
layer runs them: the mixed [q | k | v] stream is smoothed by the recurrence, q and k leave it as
views, are normed and turned by their positions, and the chunk forward mixes them; decode steps
continue the prefill; the backward runs the other way.  Against the plain 64-bit forms and the
oracle, in max |err| / RMS(ref) with the chunk path's bars (tests/parity.py): the chain's own
operators are two orders nearer than those, so the bars stay the chunk kernel's."""
import numpy as np
import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from oracle import oracle as O
from tests import plain_linrec as P
from tests.parity import TOL, rel_err, rounding_ratio

pytestmark = pytest.mark.gpu
F64 = torch.float64


def layer(B, T, Hk, Hv, d, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    C = 2 * Hk * d + Hv * d
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    proj = rnd(B, T, 3 * C).to(dtype)  # one projection's output: the stream and its gates
    s = dict(proj=proj, A_log=torch.rand(C, generator=gen) * 2.7,
             dt_bias=torch.rand(C, generator=gen) * 3 - 4, state=rnd(B, C),
             a=rnd(B, T, Hv).to(dtype), b=rnd(B, T, Hv).to(dtype),
             A2=torch.rand(Hv, generator=gen) * 2.7, t2=torch.rand(Hv, generator=gen) * 3 - 4,
             h0=rnd(B, Hv, d, d) * 0.02, do=rnd(B, T, Hv, d).to(dtype),
             dht=rnd(B, Hv, d, d) * 0.02, z=rnd(B, T, Hv, d).to(dtype),
             nw=torch.rand(d, generator=gen) + 0.5,
             inv_freq=(1e4 ** (-torch.arange(0, d // 2, 2, dtype=F64) / (d // 2))).float(),
             pos=torch.arange(T).repeat(B, 1) + torch.tensor([[0], [100000]])[:B])
    return s, {k: v.cuda() for k, v in s.items()}


def parts(x, C):
    return x[..., :C], x[..., C:2 * C], x[..., 2 * C:]


def split(h, Hk, Hv, d):
    """q, k, v of the mixed stream, as views."""
    n = Hk * d
    return (h[..., :n].unflatten(-1, (Hk, d)), h[..., n:2 * n].unflatten(-1, (Hk, d)),
            h[..., 2 * n:].unflatten(-1, (Hv, d)))


def forward(s, Hk, Hv, d, dtype):
    C = s["A_log"].numel()
    kw = dict(norm="l2", scale=d ** -0.5)
    h, st, states = G.gdn_linrec_fwd(*parts(s["proj"], C), s["A_log"], s["dt_bias"], s["state"],
                                     want_states=True)
    q, k, v = split(h, Hk, Hv, d)
    q2, k2 = G.gdn_qk_norm_rope(q, k, s["pos"], s["inv_freq"], **kw)
    o, ht = G.gdn_chunk_fwd(q2, k2, v.contiguous(), s["a"], s["b"], s["A2"], s["t2"], s["h0"],
                            scale=1.0, l2norm=False, out_f32=True)
    return h, st, states, (q, k, v), (q2, k2), o, ht


def plain(s, Hk, Hv, d, h=None):
    C = s["A_log"].numel()
    if h is None:
        h, st = P.recurrence(*parts(s["proj"], C), s["A_log"], s["dt_bias"], s["state"])
    q, k, v = split(h, Hk, Hv, d)
    q2 = P.norm_rope(q, s["pos"], s["inv_freq"], None, norm="l2", scale=d ** -0.5)
    k2 = P.norm_rope(k, s["pos"], s["inv_freq"], None, norm="l2")
    return h, (q, k, v), (q2, k2)


def n64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_forward_and_decode(dtype, d):
    B, T, Hk, Hv = 2, 150, 2, 4
    s, g = layer(B, T, Hk, Hv, d, dtype, 1)
    h, st, _, _, (q2, k2), o, ht = forward(g, Hk, Hv, d, dtype)
    # bf16 rounds what one call hands to the next: there each call is held to the plain form of
    # what it was given
    ph, (_, _, pv), (pq, pk) = plain(s, Hk, Hv, d, None if dtype == torch.float32 else h.cpu())
    if dtype == torch.bfloat16:
        pq, pk = q2.cpu(), k2.cpu()
    ro, rht = O.gdn_fwd(n64(pq), n64(pk), n64(pv), n64(s["a"]), n64(s["b"]), n64(s["A2"]),
                        n64(s["t2"]), n64(s["h0"]), scale=1.0, l2norm=False)
    assert rel_err(o, ro) <= TOL[dtype]
    assert rel_err(ht, rht) <= TOL[dtype]
    y = G.gdn_rmsnorm_gated(o.to(dtype), g["z"], g["nw"])
    ry = O.rmsnorm_gated(n64(o.to(dtype)), n64(s["z"]), n64(s["nw"]))
    if dtype == torch.float32:
        assert rel_err(y, ry) <= TOL[dtype]
    else:  # a bf16 store alone is over that bar (tests/parity.py): one rounding of each value
        assert rounding_ratio(y, ry) <= 1
    if dtype != torch.float32:
        return
    # the last tokens one by one continue a shorter prefill
    cut = 140
    C = s["A_log"].numel()
    part = dict(g, proj=g["proj"][:, :cut].contiguous(), a=g["a"][:, :cut].contiguous(),
                b=g["b"][:, :cut].contiguous(), pos=g["pos"][:, :cut].contiguous())
    _, st, _, _, _, _, ht = forward(part, Hk, Hv, d, dtype)
    for t in range(cut, T):
        x = G.gdn_linrec_step(*parts(g["proj"][:, t], C), g["A_log"], g["dt_bias"], st)
        q, k, _ = split(x, Hk, Hv, d)
        G.gdn_qk_norm_rope(q, k, g["pos"][:, t].contiguous(), g["inv_freq"], norm="l2", q_out=q,
                           k_out=k)
        # the step norms again, which leaves unit rows as they are but for its 1e-6
        oo = G.gdn_recurrent_step(x, None, None, g["a"][:, t].contiguous(),
                                  g["b"][:, t].contiguous(), g["A2"], g["t2"], ht, Hk=Hk, Hv=Hv,
                                  dk=d, dv=d)
        assert rel_err(oo, ro[:, t]) <= TOL[dtype], t


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_backward(dtype, d):
    B, T, Hk, Hv = 2, 100, 1, 2
    s, g = layer(B, T, Hk, Hv, d, dtype, 2)
    C = s["A_log"].numel()
    h, _, states, (q, k, v), (q2, k2), _, _ = forward(g, Hk, Hv, d, dtype)
    cg = G.gdn_chunk_bwd(q2, k2, v.contiguous(), g["a"], g["b"], g["A2"], g["t2"], g["h0"],
                         g["do"], g["dht"], scale=1.0, l2norm=False)
    rg = G.gdn_qk_norm_rope_bwd(q, k, g["pos"], g["inv_freq"], None, None, cg["dq"], cg["dk"],
                                norm="l2", scale=d ** -0.5, grad_f32=True)
    dh = torch.cat([rg["dq"].flatten(2), rg["dk"].flatten(2), cg["dv"].flatten(2)], -1)
    lg = G.gdn_linrec_bwd(*parts(g["proj"], C), g["A_log"], g["dt_bias"], g["state"], dh,
                          states=states, grad_f32=True)
    # the same in 64 bits: the oracle's gradients at q, k, v, then autograd through the plain
    # forms (of the bf16 values that each call was given)
    leaf = {n: s[n].double().requires_grad_(True) for n in ("proj", "A_log", "dt_bias", "state")}
    ph, _ = P.recurrence(*parts(leaf["proj"], C), leaf["A_log"], leaf["dt_bias"], leaf["state"])
    mid = (ph if dtype == torch.float32 else h.cpu().double()).detach().requires_grad_(True)
    _, (pq, pk, pv), (pq2, pk2) = plain(s, Hk, Hv, d, mid)
    if dtype == torch.float32:
        at = (n64(pq2), n64(pk2), n64(pv))
    else:
        at = (n64(q2), n64(k2), n64(v))
    want = O.gdn_bwd(*at, n64(s["a"]), n64(s["b"]), n64(s["A2"]), n64(s["t2"]), n64(s["h0"]),
                     n64(s["do"]), n64(s["dht"]), scale=1.0, l2norm=False)
    wq, wk, wv = (torch.from_numpy(np.asarray(want[n])).double() for n in ("dq", "dk", "dv"))
    dmid, = torch.autograd.grad([pq2, pk2, pv], [mid], [wq, wk, wv])
    assert rel_err(dh, dmid.numpy()) <= TOL[dtype]
    grads = torch.autograd.grad([ph], list(leaf.values()), [dmid])
    got = dict(proj=torch.cat([lg["dx"], lg["da"], lg["db"]], -1), A_log=lg["dA_log"],
               dt_bias=lg["ddt_bias"], state=lg["dh0"])
    for n, r in zip(leaf, grads):
        assert rel_err(got[n], r.numpy()) <= TOL[dtype], n
