"""Norm and rotation of q and k where something besides the call's own rows could reach the
results: shared memory that an earlier kernel left."""
import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from tests import test_qk_rope_gpu as R

pytestmark = pytest.mark.gpu
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64


def stain():
    """Leaves NaN in the shared memory of every multiprocessor: a scan of NaN keeps its folds
    and its tiles there, 100 KB a block and two blocks a multiprocessor."""
    x = torch.full((148 * 8, 64, 64), float("nan"), device="cuda")
    w = torch.zeros(64, device="cuda")
    G.gdn_linrec_fwd(x, x, x, w, w)


@pytest.mark.parametrize("d", [2, 4, 6, 10, 36, 100, 130, 250])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_heads_whose_last_lane_is_not_full(d, interleaved, norm, monkeypatch):
    """The whole head is rotated and its channels do not fill the lanes that hold them."""
    for name in ("gdn_qk_norm_rope", "gdn_qk_norm_rope_bwd"):
        fn = getattr(G, name)

        def stained(*a, fn=fn, **kw):
            stain()
            return fn(*a, **kw)

        monkeypatch.setattr(G, name, stained)
    for dtype in (F32, BF16):
        R.check(*R.make(9, 3, 2, d, d, dtype, seed=d), norm=norm, interleaved=interleaved)
