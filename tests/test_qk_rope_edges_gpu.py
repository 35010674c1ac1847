"""Norm and rotation of q and k where something besides the call's own rows could reach the
results (shared memory that an earlier kernel left), and far positions."""
from fractions import Fraction

import pytest
import torch

import gated_deltanet_sequence_gdn_b200 as G
from tests import plain_linrec as P
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


def two_pi(bits):
    """round(2^bits * 2 pi), by Machin's formula in integers."""
    def arctan_inverse(n, one):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    one = 1 << (bits + 32)
    pi = 4 * (4 * arctan_inverse(5, one) - arctan_inverse(239, one))
    return (2 * pi + (1 << 31)) >> 32


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("theta", [1e4, 1e7])
@pytest.mark.parametrize("bits", [20, 31, 36, 40, 52, 62])
def test_positions_of_many_bits(bits, theta, interleaved):
    """Angles of positions far beyond what float64 products hold, against turns formed in
    integers.  Bound, u = 2^-24, relative to the length of the value's pair: the turn is held in
    64 bits, rounded once, which a position multiplies: |position| 2^-65 turns; its top 32 bits
    (2^-32 turns) become a float of half turns (2^-25 half turns): 1.7 u rad; cosine and sine
    are within 2 u each, the product and the sum of the rotation round twice more: 8 u."""

    d = 64
    s, dev = R.make(12, 2, 1, d, d, F32, seed=bits, theta=theta, weights=False)
    pos = [1 << bits, -(1 << bits), (1 << bits) - 1, 1 - (1 << bits)]
    gen = torch.Generator().manual_seed(bits)
    pos += torch.randint(1 << (bits - 1), 1 << bits, (8,), generator=gen).tolist()
    dev["pos"].copy_(torch.tensor(pos))
    unit = Fraction(two_pi(256), 1 << 256)
    ang = torch.empty(12, d // 2, dtype=F64)
    for t, p in enumerate(pos):
        for i, f in enumerate(s["inv_freq"].tolist()):
            turn = p * Fraction(f) / unit
            ang[t, i] = float((turn - round(turn)) * unit)
    c, sn = ang.cos()[:, None], ang.sin()[:, None]
    outs = G.gdn_qk_norm_rope(dev["q"], dev["k"], dev["pos"], dev["inv_freq"], norm=None,
                              interleaved=interleaved)
    for name, got in zip("qk", outs):
        x = s[name].to(F64)
        if interleaved:
            p, q = x[..., 0::2], x[..., 1::2]
            y = torch.stack([p * c - q * sn, q * c + p * sn], -1).flatten(-2)
        else:
            p, q = x[..., :d // 2], x[..., d // 2:]
            y = torch.cat([p * c - q * sn, q * c + p * sn], -1)
        far = torch.tensor([abs(v) for v in pos], dtype=F64)[:, None, None]
        rad = 6.2831853072 * far * 2.0 ** -65
        P.check(f"{name} at 2^{bits}", got, y,
                (8 * P.U + rad) * P.rope_pair_size(x, d, interleaved))


def test_frequencies_of_any_size_and_sign():
    """Whole turns a token, none at all, the other way round: the bound of above."""
    s, dev = R.make(40, 2, 1, 16, 16, F32, seed=1, far=1 << 24, weights=False)
    freq = torch.tensor([0.0, 1e-30, -1e-30, 1e-9, -0.37, 6.2831855, 12345.678, -7e6])
    s["inv_freq"] = freq
    unit = Fraction(two_pi(256), 1 << 256)
    ang = torch.tensor([[float((t - round(t)) * unit) for t in (p * Fraction(f) / unit
                                                                for f in freq.tolist())]
                        for p in s["pos"].tolist()], dtype=F64)
    c, sn = ang.cos()[:, None], ang.sin()[:, None]
    outs = G.gdn_qk_norm_rope(dev["q"], dev["k"], dev["pos"], freq.cuda(), norm=None)
    for name, got in zip("qk", outs):
        x = s[name].to(F64)
        p, q = x[..., :8], x[..., 8:]
        y = torch.cat([p * c - q * sn, q * c + p * sn], -1)
        rad = 6.2831853072 * s["pos"].to(F64)[:, None, None] * 2.0 ** -65
        P.check(name, got, y, (8 * P.U + rad) * P.rope_pair_size(x, 16, False))
