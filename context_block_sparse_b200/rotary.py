"""Rotary positions for queries and keys (splitkv_rope), with long-context scalings.

    rot = Rotary(128, base=10000.0, scaling="parts", factor=8.0, original_len=4096)
    q, k = rot.forward(positions, q, k)          # [n, heads, d] each, positions [n]
    dq, dk = rot.backward(positions, dq, dk)     # the transpose: gradients of the unrotated q, k

`SplitKVAttention(rotary=rot)` applies it inside the attention, forward and backward.  All arithmetic runs in
the library's kernel; this module holds the frequency table and allocates outputs.
"""

from __future__ import annotations

from typing import Optional

import torch

from ._abi import ROPE_SCALE_BASE, ROPE_SCALE_LINEAR, ROPE_SCALE_NONE, ROPE_SCALE_PARTS
from .draft_calls import splitkv_rope, splitkv_rope_freqs

SCALINGS = {"none": ROPE_SCALE_NONE, "linear": ROPE_SCALE_LINEAR, "base": ROPE_SCALE_BASE, "parts": ROPE_SCALE_PARTS}


class Rotary:
    """Frequencies w_i = base^(-2i / rotary_dim) of a head's first rotary_dim elements.

    interleaved: pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2).
    scaling: "none"; "linear" (positions divided by factor); "base" (base raised so that the slowest pair is
    stretched by factor); "parts" (pairs that turn at least turns_high times over original_len positions kept,
    those below turns_low stretched by factor, linear between, and rotated vectors multiplied by
    0.1 ln(factor) + 1)."""

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, base: float = 10000.0,
                 interleaved: bool = False, scaling: str = "none", factor: float = 1.0, original_len: float = 0.0,
                 turns_low: float = 1.0, turns_high: float = 32.0, device: Optional[torch.device] = None):
        if scaling not in SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(SCALINGS)}")
        rotary_dim = head_dim if rotary_dim is None else int(rotary_dim)
        if rotary_dim < 2 or rotary_dim % 2 or rotary_dim > head_dim:
            raise ValueError("rotary_dim must be even, between 2 and head_dim")
        self.head_dim = int(head_dim)
        self.rotary_dim = rotary_dim
        self.interleaved = bool(interleaved)
        freqs, self.scale = splitkv_rope_freqs(rotary_dim, base, SCALINGS[scaling], factor, original_len, turns_low,
                                               turns_high)
        self.freqs = torch.from_numpy(freqs)      # float64, radians per position
        self._on = {}                             # per device (uploaded once; before a graph is captured)
        if torch.cuda.is_available():
            device = torch.device("cuda" if device is None else device)
            self._table(torch.cuda.current_device() if device.index is None else device.index)

    def _table(self, index: int) -> torch.Tensor:
        t = self._on.get(index)
        if t is None:
            t = self._on[index] = self.freqs.to(torch.device("cuda", index))
        return t

    def _apply(self, positions, q, k, out, adjoint: bool):
        d = self.head_dim
        if q.dim() != 3 or q.shape[2] != d:
            raise ValueError(f"q must be [n, heads, {d}]")
        if k is not None and (k.dim() != 3 or k.shape[2] != d):
            raise ValueError(f"k must be [n, heads, {d}]")
        dev = q.get_device()
        if dev < 0:
            raise ValueError("q must be a CUDA tensor")
        q_out, k_out = (None, None) if out is None else out if k is not None else (out[0], None)
        return splitkv_rope(positions, self._table(dev), self.scale, q, k, q_out, k_out, self.interleaved, adjoint)

    def forward(self, positions, q, k=None, out=None):
        """q [n, Hq, d] (and k [n, Hk, d]) at positions [n] (int32 or int64); float32, bfloat16 or float16, the
        last dimension contiguous.  Returns q', or (q', k').  out: a tuple of outputs; out=(q, k) works in place."""
        return self._apply(positions, q, k, out, False)

    def backward(self, positions, dq, dk=None, out=None):
        """Gradients of the unrotated q (and k) from those of the rotated ones; arguments as forward."""
        return self._apply(positions, dq, dk, out, True)
