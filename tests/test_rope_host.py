"""Frequency tables against the documented formulas where the first tests do not go (CPU)."""

import math

import pytest


@pytest.mark.parametrize("factor", [0.25, 0.999, 1.0, 1.5, 40.0])
def test_parts_scale_under_any_factor(splitkv, factor):
    """By parts the rotated vectors are multiplied by 0.1 ln(factor) + 1, also below one; the others leave them."""
    from context_block_sparse_b200.rotary import SCALINGS
    for name, kind in SCALINGS.items():
        freqs, scale = splitkv.splitkv_rope_freqs(64, 10000.0, kind, factor, 4096)
        assert scale == pytest.approx(0.1 * math.log(factor) + 1 if name == "parts" else 1.0, rel=1e-15)
        assert (freqs > 0).all()
