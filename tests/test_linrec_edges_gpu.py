"""The gated linear recurrence at the edges of a call: rows that no sequence holds, buffers that
are input and output at once, infinities, expired waits, far strides."""
import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from tests import plain_linrec as P
from tests.test_linrec_gpu import ins, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("cu", [[0, 70, 75], [0], [0, 0, 0]])
def test_rows_of_no_sequence_are_zeros(cu, given, dtype):
    """What the call allocates holds zeros behind the last sequence: those tokens are not read,
    so their outputs are none and their gradients are zero."""
    s, d = make(len(cu) - 1, 200, 72, dtype, cu=cu, given=given, seed=3)
    kw = dict(cu_seqlens=cu, gates_precomputed=given)
    for _ in range(2):
        stale = [torch.full((200, 72), float("nan"), device="cuda", dtype=t)
                 for t in (dtype, F32) for _ in range(6)]
        del stale  # what the call allocates next
        h, ht = G.gdn_linrec_fwd(*ins(d), **kw)
        g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], **kw)
        for k, v in [("h", h), ("dx", g["dx"]), ("da", g["da"]), ("db", g["db"])]:
            assert not v[cu[-1]:].any(), k
            assert torch.isfinite(v).all(), k
    mine = torch.full((200, 72), 7.0, device="cuda", dtype=dtype)
    G.gdn_linrec_fwd(*ins(d), h=mine, **kw)  # the caller's own rows stay
    assert (mine[cu[-1]:] == 7.0).all() and torch.equal(mine[:cu[-1]], h[:cu[-1]])


def backward_into(d, T, D, dh0):
    """The C entry point with the caller's dh0; everything else contiguous.  Returns dx."""
    x = d["x"]
    B = x.shape[0]
    code = {F32: G.F32, BF16: G.BF16}[x.dtype]
    outs = [torch.empty_like(x) for _ in range(3)]
    sums = [torch.empty(D, device="cuda") for _ in range(2)]
    need = G.gdn_linrec_bwd_workspace_bytes(B, T, D)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    p = [d[k].data_ptr() for k in ("x", "a", "b", "A_log", "dt_bias", "h0")]
    st = G.lib.gdn_linrec_bwd(*p, None, B, T, D, D, D, D, d["dh"].data_ptr(), D,
                              d["dht"].data_ptr(), None, code, 0, outs[0].data_ptr(), D,
                              outs[1].data_ptr(), D, outs[2].data_ptr(), D, sums[0].data_ptr(),
                              sums[1].data_ptr(), dh0.data_ptr(), ws.data_ptr(), need,
                              torch.cuda.current_stream().cuda_stream)
    assert st == 0
    return outs[0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D", [(1, 1024, 64), (2, 5000, 40), (3, 200, 600), (1, 4096, 16)])
def test_final_states_in_the_place_of_the_first(B, T, D, dtype):
    """ht = h0 and dh0 = dht, where a cluster's blocks all read what one of them writes."""
    _, d = make(B, T, D, dtype, seed=T)
    h, ht = G.gdn_linrec_fwd(*ins(d))
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"])
    for _ in range(20):
        both = d["h0"].clone()
        h2, ht2 = G.gdn_linrec_fwd(*ins(dict(d, h0=both)), ht=both)
        assert ht2 is both and torch.equal(both, ht) and torch.equal(h2, h)
        both = d["dht"].clone()
        dx = backward_into(dict(d, dht=both), T, D, both)
        assert torch.equal(both, g["dh0"]) and torch.equal(dx, g["dx"])


@pytest.mark.parametrize("B,T,D", [(2, 300, 64), (1, 5000, 64), (300, 200, 128)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tiles_that_do_not_come_are_reported(B, T, D, dtype):
    """The tiles' copies are not asked for: the waits for them end and say so, in lone blocks and
    in clusters, and the next call is right again."""
    _, d = make(B, T, D, dtype, seed=17)
    h, ht, st = G.gdn_linrec_fwd(*ins(d), want_states=True)
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], states=st)
    assert G.gdn_status() == 0
    try:
        G.gdn_test_set_wait_fault(4, 1 << 10)
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


def test_every_argument_by_name_and_on_another_stream():
    s, d = make(2, 70, 40, F32, seed=18)
    named = {k: d[k] for k in ("x", "a", "b", "A_log", "dt_bias", "h0")}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    h, ht = G.gdn_linrec_fwd(**named, stream=side)
    g = G.gdn_linrec_bwd(**named, dh=d["dh"], dht=d["dht"], stream=side)
    state = d["h0"].clone()
    side.wait_stream(torch.cuda.current_stream())
    one = {k: d[k][:, 0] for k in ("x", "a", "b")}
    h1 = G.gdn_linrec_step(**one, A_log=d["A_log"], dt_bias=d["dt_bias"], state=state, stream=side)
    torch.cuda.synchronize()
    P.check("h", h, *P.forward_bounds(*ins(s))["h"])
    P.check("dx", g["dx"], *P.backward_bounds(*ins(s, "dh", "dht"))["dx"])
    P.check("first", h1, *(v[:, 0] for v in P.forward_bounds(*ins(s))["h"]))


def test_step_of_one_token_of_a_long_batch():
    """Sequences further apart than a scan's tokens may be: a token of a [N, T, D] batch."""
    N, T, D = 3, 1100, 2048  # 2.25M elements from sequence to sequence
    s, d = make(N, 1, D, F32, seed=21)
    want = P.forward_bounds(*ins(s))
    far = {k: torch.zeros(N, T, D, device="cuda") for k in ("x", "a", "b")}
    for k in far:
        far[k][:, 700] = d[k][:, 0]
    out = torch.zeros(N, T, D, device="cuda")
    state = d["h0"].clone()
    h = G.gdn_linrec_step(*(far[k][:, 700] for k in ("x", "a", "b")), d["A_log"], d["dt_bias"],
                          state, h=out[:, 700])
    P.check("h", h, want["h"][0][:, 0], want["h"][1][:, 0])
    P.check("state", state, *want["ht"])
    out[:, 700] = 0
    assert not out.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", ["none", "unit"])
def test_infinities(dtype, scale):
    """An infinite input or state leaves its channel without a finite value from there on (NaN
    where products of decays have underflowed, as 0 x inf) and reaches nothing else; so does an
    infinite gradient, the other way."""
    s, d = make(2, 260, 70, dtype, seed=19)
    d["A_log"][33:36] = 2.7  # fast channels: 8 tokens' product of decays is 0
    for c in (33, 34):
        d["a"][:, :, c] = 5.0
    kw = dict(input_scale=scale)
    h, ht = G.gdn_linrec_fwd(*ins(d), **kw)
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], **kw)
    e = dict(d, x=d["x"].clone(), h0=d["h0"].clone())
    e["x"][1, 100, 33] = float("inf")
    e["x"][0, 70, 35] = float("-inf")
    e["h0"][0, 34] = float("inf")
    h2, ht2 = G.gdn_linrec_fwd(*ins(e), **kw)
    bad = torch.zeros_like(h, dtype=torch.bool)
    bad[1, 100:, 33] = bad[0, 70:, 35] = bad[0, :, 34] = True
    assert torch.equal(~torch.isfinite(h2), bad)
    assert torch.equal(h2[~bad], h[~bad])
    assert torch.equal(~torch.isfinite(ht2), bad[:, -1]) and torch.equal(ht2[~bad[:, -1]],
                                                                         ht[~bad[:, -1]])
    g2 = G.gdn_linrec_bwd(*ins(e), d["dh"], d["dht"], **kw)
    assert torch.equal(g2["dx"], g["dx"]) and torch.equal(g2["dh0"], g["dh0"])
    assert torch.equal(g2["da"][~bad], g["da"][~bad])
    one = torch.zeros_like(bad)
    one[1, 100, 33] = one[0, 70, 35] = True
    assert torch.equal(g2["db"][~one], g["db"][~one])
    e = dict(d, dh=d["dh"].clone(), dht=d["dht"].clone())
    e["dh"][1, 100, 33] = float("inf")
    e["dht"][0, 34] = float("-inf")
    g2 = G.gdn_linrec_bwd(*ins(e), e["dh"], e["dht"], **kw)
    bad = torch.zeros_like(bad)
    bad[1, :101, 33] = bad[0, :, 34] = True
    for k in ("dx", "da", "db"):
        assert torch.equal(g2[k][~bad], g[k][~bad]), k
        assert not torch.isfinite(g2[k][bad]).any(), k
    rest = ~bad[:, 0]
    assert not torch.isfinite(g2["dh0"][~rest]).any() and torch.equal(g2["dh0"][rest],
                                                                      g["dh0"][rest])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_what_a_workspace_holds_before_the_call_does_not_matter(dtype):
    """A packed batch's table, the states and the blocks' sums, over memory of any content."""
    cu = [0, 130, 130, 131, 700, 1500]
    _, d = make(len(cu) - 1, cu[-1], 88, dtype, cu=cu, seed=20)
    size = (len(cu) - 1, cu[-1], 88, cu)
    need, more = G.gdn_linrec_workspace_bytes(*size), G.gdn_linrec_bwd_workspace_bytes(*size)
    assert more > need > 0
    h, ht = G.gdn_linrec_fwd(*ins(d), cu_seqlens=cu)
    g = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], cu_seqlens=cu)
    for fill in (0, 1, 127, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        h2, ht2 = G.gdn_linrec_fwd(*ins(d), cu_seqlens=cu, workspace=ws)
        assert torch.equal(h, h2) and torch.equal(ht, ht2)
        ws = torch.full((more,), fill, dtype=torch.uint8, device="cuda")
        g2 = G.gdn_linrec_bwd(*ins(d), d["dh"], d["dht"], cu_seqlens=cu, workspace=ws)
        assert all(torch.equal(g[k], g2[k]) for k in g)
    with pytest.raises(G.GDNError):
        G.gdn_linrec_fwd(*ins(d), cu_seqlens=cu, workspace=ws[:need - 1])
    with pytest.raises(G.GDNError):
        G.gdn_linrec_bwd(*ins(d), d["dh"], cu_seqlens=cu, workspace=ws[:more - 1])


@pytest.mark.parametrize("T", [1, 65, 100, 192, 250, 300])
@pytest.mark.parametrize("scale,gate,given", [("none", True, False), ("tied", False, False),
                                              ("unit", True, True)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_do_not_depend_on_the_split(dtype, scale, gate, given, T):
    """A sequence in a batch that fills the machine (tiles of one chunk, lone blocks), by itself
    (tiles of several chunks, ends inside them, clusters), and with a channel more (rows whose
    pairs are not aligned and that no TMA takes): bit for bit the same."""
    B, D = 700, 64
    _, d = make(B, T, D, dtype, gate=gate, given=given, seed=T)
    kw = dict(input_scale=scale, gates_precomputed=given, grad_f32=True)

    def grads(s):
        g = G.gdn_linrec_bwd(*ins(s), s["dh"].float(), s["dht"], **kw)
        return {k: g[k] for k in ("dx", "da", "db", "dh0") if g[k] is not None}

    want = grads(d)
    seq = ("x", "a", "b", "dh", "h0", "dht")
    for r in (0, B - 1):
        one = {k: v[r:r + 1] if k in seq and v is not None else v for k, v in d.items()}
        for k, v in grads(one).items():
            assert torch.equal(v, want[k][r:r + 1]), k
    wide = {k: None if v is None else torch.cat([v, v[..., :1]], -1) for k, v in d.items()}
    for k, v in grads(wide).items():
        assert torch.equal(v[..., :D], want[k]), k
