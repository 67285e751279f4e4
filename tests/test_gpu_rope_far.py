"""Rotary positions that need int64, against angles in exact arithmetic."""

from fractions import Fraction

import pytest
import torch

from draft_util import half_step

pytestmark = pytest.mark.gpu

# pi to 50 decimals (its error times any turn here is far below 2^-100)
TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


def _reduced(position: int, w: float) -> float:
    """position * w - 2 pi k in [-pi, pi], the product and the reduction exact."""
    t = position * Fraction(w) / TWO_PI
    return float((t - round(t)) * TWO_PI)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("top", [31, 33, 36, 40])
def test_positions_past_32_bits(splitkv, top, interleaved):
    """The float64 steps round the whole angle four times (position, frequency in turns and its constant, their product):
    |t| 2^-51 rad; the rest as in rope_ref's bound, scale (|a| + |b|) 2^-21."""
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(32, interleaved=interleaved)
    g = torch.Generator().manual_seed(top)
    pos = torch.randint(-2 ** top, 2 ** top, (40,), generator=g)
    pos[:4] = torch.tensor([2 ** top, -2 ** top, 2 ** top - 1, 0])
    x = torch.randn(40, 2, 32, generator=g)
    h = rot.freqs.numel()
    ang = torch.tensor([[_reduced(p, w) for w in rot.freqs.tolist()] for p in pos.tolist()], dtype=torch.float64)[:, None]
    whole = pos.double().abs()[:, None, None] * rot.freqs
    ia = torch.arange(0, 2 * h, 2) if interleaved else torch.arange(h)
    ib = ia + 1 if interleaved else ia + h
    for turn, sign in ((rot.forward, 1.0), (rot.backward, -1.0)):
        got = turn(pos.cuda(), x.cuda()).double().cpu()
        a, b = x[..., ia].double(), x[..., ib].double()
        c, s = torch.cos(ang), sign * torch.sin(ang)
        lim = (a.abs() + b.abs()) * (2.0 ** -21 + whole * 2.0 ** -51)
        for at, want in ((ia, a * c - b * s), (ib, b * c + a * s)):
            assert ((got[..., at] - want).abs() <= lim + half_step(torch.float32) * (want.abs() + lim)).all()


def test_int64_and_int32_positions_agree(splitkv):
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(64, rotary_dim=48)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (70,), generator=torch.Generator().manual_seed(1)).cuda()
    x = torch.randn(70, 3, 64, device="cuda").bfloat16()
    assert torch.equal(rot.forward(pos, x), rot.forward(pos.int(), x))
