"""Positions that SplitKVAttention hands to its Rotary (host side; no GPU)."""

import numpy as np
import torch


def _attention(splitkv, lens, anchors, bs=4):
    from context_block_sparse_b200.torch_api import SplitKVAttention
    att = SplitKVAttention.__new__(SplitKVAttention)
    att.device = torch.device("cpu")
    att.plan = splitkv.splitkv_plan(lens, anchors, bs, 4, 2, 64, 64, 8)
    att._ctx_pos = att._row_pos = None
    att._place()
    return att


def _positions(lens, anchors, bs=4):
    starts = np.concatenate([[0], np.cumsum(lens)])
    ctx = [i for n in lens for i in range(n)]
    rows = [a - max(s for s in starts if s <= a) + r for a in anchors for r in range(bs)]
    return ctx, rows


def test_a_plan_update_of_the_same_sizes_keeps_the_tensors(splitkv):
    """A captured graph holds the position tensors: they are written over, not replaced."""
    att = _attention(splitkv, [30, 130], [5, 35, 140])
    ctx, rows = att._ctx_pos, att._row_pos
    assert (ctx.tolist(), rows.tolist()) == _positions([30, 130], [5, 35, 140])
    for lens, anchors in (([100, 60], [10, 70, 120]), ([160], [0, 1, 159])):
        splitkv.splitkv_plan_update(att.plan, lens, anchors)
        att._place()
        assert att._ctx_pos is ctx and att._row_pos is rows
        assert (ctx.tolist(), rows.tolist()) == _positions(lens, anchors)
    splitkv.splitkv_plan_update(att.plan, [90, 20], [10, 70])
    att._place()
    assert (att._ctx_pos.tolist(), att._row_pos.tolist()) == _positions([90, 20], [10, 70])
