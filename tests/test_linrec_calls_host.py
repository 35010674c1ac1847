"""How the entry points of the gated linear recurrence and of the norm-and-rotation take their
arguments, without a GPU."""
import inspect

import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G

HERE = torch.zeros(2, 8)
W = torch.zeros(8)


@pytest.mark.parametrize("fn,kw", [
    (G.gdn_linrec_fwd, dict(x=HERE, a=HERE, A_log=W, dt_bias=W, cu_seqlens=[0, 2])),
    (G.gdn_linrec_bwd, dict(x=HERE, a=HERE, b=None, A_log=W, dt_bias=W, h0=None, dh=HERE,
                            cu_seqlens=[0, 2])),
    (G.gdn_linrec_step, dict(x=HERE, a=HERE, b=None, A_log=W, dt_bias=W, state=HERE)),
])
def test_every_argument_has_its_name(fn, kw):
    """By name all the way: what is wrong with these calls is that the tensors are the host's."""
    assert list(inspect.signature(fn).parameters)[0] == "x"
    assert inspect.signature(fn).parameters["stream"].kind is inspect.Parameter.KEYWORD_ONLY
    with pytest.raises(ValueError, match="CUDA device"):
        fn(**kw)
    with pytest.raises(TypeError, match="x must be a tensor"):
        fn(**dict(kw, x=None))
    with pytest.raises(TypeError, match="x must be a tensor"):
        fn(**{k: v for k, v in kw.items() if k != "x"})


@pytest.mark.parametrize("fn,more", [(G.gdn_qk_norm_rope, ()),
                                     (G.gdn_qk_norm_rope_bwd, (None, None, None, None))])
def test_neither_q_nor_k(fn, more):
    with pytest.raises(ValueError, match="q and k"):
        fn(None, None, torch.zeros(1), None, *more)


def test_workspace_queries_take_the_sequences_from_the_offsets():
    """Whatever B says: the library reads B + 1 offsets."""
    cu = list(range(0, 4000, 8))
    n, T = len(cu) - 1, cu[-1]
    for B in (0, 1, n, 10 ** 6):
        assert G.gdn_linrec_workspace_bytes(B, T, 64, cu) == \
            G.lib.gdn_linrec_workspace_bytes((G._ll * (n + 1))(*cu), n, T, 64) > 0
        assert G.gdn_linrec_bwd_workspace_bytes(B, T, 64, torch.tensor(cu)) == \
            G.lib.gdn_linrec_bwd_workspace_bytes((G._ll * (n + 1))(*cu), n, T, 64, 0, 0) > 0


def test_rotation_workspace_query_of_refused_sizes():
    query = G.gdn_qk_norm_rope_bwd_workspace_bytes
    assert query(2 ** 30 - 1, 4, 2, 64) == query(10 ** 6, 4, 2, 64) > 0
    for sizes in ((2 ** 30, 4, 2, 64), (2 ** 62, 4, 2, 64), (5, 2 ** 20, 1, 64),
                  (5, 2 ** 31 - 1, 2 ** 31 - 1, 64), (5, 4, 2, 257), (5, 0, 0, 64)):
        assert query(*sizes) == 0, sizes
    with pytest.raises(ValueError, match="norm"):
        query(5, 4, 2, 64, "layer")


def test_step_strides():
    """A step's sequences may be further apart than a scan's tokens (a GPU test takes such a
    step); here the limit behind that, and that nothing else gets past it."""
    a = dict(x=1 << 16, a=1 << 16, b=1 << 16, A=1 << 16, t=1 << 16, st=1 << 16, N=3, D=64,
             ldx=64, lda=64, ldb=64, dtype=1, flags=0, h=1 << 16, ldh=64)
    for k in ("ldx", "lda", "ldb", "ldh"):
        assert G.lib.gdn_linrec_step(*dict(a, **{k: 2 ** 32 + 1}).values(), None) == -2
        assert G.lib.gdn_linrec_step(*dict(a, **{k: 2 ** 32, "N": -1}).values(), None) == -1
    far = dict(a, ldx=2 ** 32, lda=2 ** 32, ldb=2 ** 32, N=0)
    assert G.lib.gdn_linrec_step(*far.values(), None) == 0


def test_the_distance_of_a_write_gate_that_is_not_there():
    """ldb and lddb count with b and db alone (no token, so that nothing is launched; in the
    backward the workspace's check, behind all others, ends the call)."""
    p = 1 << 16
    for b, st in ((None, 0), (p, -2)):
        assert G.lib.gdn_linrec_fwd(p, p, b, p, p, None, None, 2, 0, 64, 64, 64, 2 ** 30, 1, 0, p,
                                    64, None, None, None, 0, None) == st
        assert G.lib.gdn_linrec_step(p, p, b, p, p, p, 0, 64, 64, 64, 2 ** 33, 1, 0, p, 64,
                                     None) == st
    for db, st in ((None, -5), (p, -2)):
        assert G.lib.gdn_linrec_bwd(p, p, db, p, p, None, None, 2, 100, 64, 64, 64, 64, p, 64, None,
                                    p, 1, 0, p, 64, p, 64, db, 2 ** 30, p, p, None, None, 0,
                                    None) == st
