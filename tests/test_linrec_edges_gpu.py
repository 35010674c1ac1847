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
