"""Calls one right after another: the kernels of a call come in while the one before them is
ending, and calls in one stream may share a workspace, whatever their sizes.  Every result is the
one that the call gives by itself, bit for bit, also from a captured graph."""
import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from tests.test_linrec_gpu import ins, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# packed and dense, short and long, lone blocks and clusters, with and without a write gate
CASES = [
    dict(B=1, T=2000, D=64, dtype=BF),
    dict(B=3, T=400, D=130, dtype=F32, cu=[0, 7, 7, 390]),
    dict(B=40, T=64, D=512, dtype=BF, gate=False),
    dict(B=5, T=900, D=96, dtype=BF, cu=[0, 300, 301, 500, 500, 900]),
    dict(B=1, T=1, D=8, dtype=F32),
    dict(B=2, T=700, D=33, dtype=F32, given=True),
]


def run(d, c, ws=None):
    kw = dict(cu_seqlens=c.get("cu"), gates_precomputed=c.get("given", False), workspace=ws)
    h, ht = G.gdn_linrec_fwd(*ins(d), **kw)
    grads = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], **kw)  # recomputes the states
    n = c["cu"][-1] if c.get("cu") else None
    out = dict(h=h[:n] if n else h, ht=ht)
    for k, v in grads.items():
        if v is not None:
            out[k] = v[:n] if n and k in ("dx", "da", "db") else v
    return out


def inputs():
    return [make(**c, seed=i)[1] for i, c in enumerate(CASES)]


def alone(data):
    want = []
    for d, c in zip(data, CASES):
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in run(d, c).items()})
        torch.cuda.synchronize()
    return want


def workspace():
    need = max(G.gdn_linrec_bwd_workspace_bytes(c["B"], c["T"], c["D"], c.get("cu"),
                                                gates_precomputed=c.get("given", False))
               for c in CASES)
    return torch.empty(need, dtype=torch.uint8, device="cuda")


def same(got, want):
    assert got.keys() == want.keys()
    for k in got:
        assert torch.equal(got[k], want[k]), k


def test_calls_in_a_row_share_a_workspace():
    data, ws = inputs(), workspace()
    want = alone(data)
    order = [(7 * i + i * i) % len(CASES) for i in range(60)]
    got = [run(data[j], CASES[j], ws) for j in order]
    torch.cuda.synchronize()
    for j, g in zip(order, got):
        same(g, want[j])


def test_the_same_row_from_a_graph():
    data, ws = inputs(), workspace()
    want = alone(data)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [run(d, c, ws) for d, c in zip(data, CASES)]
    for _ in range(3):
        for g in got:
            for v in g.values():
                v.zero_()
        graph.replay()
        for d in data:  # what follows a replay comes after all of it
            d["x"].add_(0)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            same(g, w)


def test_weights_gradients_in_a_row():
    """The launch that joins the weights' gradients reads the partial sums of its own call."""
    gen = torch.Generator().manual_seed(5)
    calls = []
    for tokens, hq, hk, d in ((700, 4, 2, 64), (9, 8, 1, 128), (2500, 2, 2, 40)):
        r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
        calls.append((r(tokens, hq, d), r(tokens, hk, d), torch.arange(tokens).cuda(),
                      torch.rand(d // 4, generator=gen).cuda(), r(d), r(d), r(tokens, hq, d),
                      r(tokens, hk, d)))
    need = max(G.gdn_qk_norm_rope_bwd_workspace_bytes(c[0].shape[0], c[0].shape[1], c[1].shape[1],
                                                      c[0].shape[2]) for c in calls)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = []
    for c in calls:
        torch.cuda.synchronize()
        want.append(G.gdn_qk_norm_rope_bwd(*c))
        torch.cuda.synchronize()
    order = [(i * i + 1) % 3 for i in range(45)]
    got = [G.gdn_qk_norm_rope_bwd(*calls[j], workspace=ws) for j in order]
    torch.cuda.synchronize()
    for j, g in zip(order, got):
        same(g, want[j])
