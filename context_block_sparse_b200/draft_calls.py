"""Bindings of the rotary and draft-tree entry points (include/splitkv.h): splitkv_rope_freqs on the host, and the calls
on tensors from the torch extension _draft_ext (ext/draft_ext.cpp), which raises ImportError when it is not built.

Tensors may be strided: the last dimension is contiguous, the others have any stride (in 16-byte steps where the
header says so).  A call runs on its tensors' device and that device's current stream.
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch  # noqa: F401  (the extension's libraries)

from . import SplitKVError, _lib
from ._abi import ROPE_SCALE_NONE
from ._draft_ext import splitkv_rope, splitkv_tree_attn, splitkv_tree_commit, splitkv_tree_verify  # noqa: F401


def splitkv_rope_freqs(rotary_dim: int, base: float = 10000.0, scaling: int = ROPE_SCALE_NONE, factor: float = 1.0,
                       original_len: float = 0.0, turns_low: float = 1.0, turns_high: float = 32.0):
    """Frequencies (radians per position, float64 [rotary_dim / 2]) and the factor on rotated vectors."""
    out = np.zeros(max(0, int(rotary_dim)) // 2, dtype=np.float64)
    scale = ctypes.c_double()
    status = _lib.splitkv_rope_freqs(
        int(rotary_dim), float(base), int(scaling), float(factor), float(original_len), float(turns_low),
        float(turns_high), out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ctypes.byref(scale))
    if status:
        raise SplitKVError("splitkv_rope_freqs", status)
    return out, scale.value
