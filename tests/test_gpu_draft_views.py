"""Rotary and draft-tree calls on views: what lies apart is taken, what does not is refused and left alone."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rd", [64, 40])
def test_rotary_between_views_of_one_buffer(splitkv, dt, rd):
    """Inputs and outputs side by side in every token, and in every head, of one buffer."""
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(64, rotary_dim=rd)
    pos = torch.arange(37, dtype=torch.int32, device="cuda") * 11
    buf = torch.randn(37, 12, 64, device="cuda").to(dt)
    keep = buf.clone()
    want = rot.forward(pos, keep[:, :4], keep[:, 4:6])
    rot.forward(pos, buf[:, :4], buf[:, 4:6], out=(buf[:, 6:10], buf[:, 10:]))
    assert torch.equal(buf[:, :6], keep[:, :6])
    assert torch.equal(buf[:, 6:10], want[0]) and torch.equal(buf[:, 10:], want[1])
    halves = torch.randn(37, 3, 2, 64, device="cuda").to(dt)
    keep = halves.clone()
    rot.forward(pos, halves[:, :, 0], out=(halves[:, :, 1],))
    assert torch.equal(halves[:, :, 0], keep[:, :, 0])
    assert torch.equal(halves[:, :, 1], rot.forward(pos, keep[:, :, 0].contiguous()))


def test_rotary_refuses_outputs_that_meet(splitkv):
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(64)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    buf = torch.randn(9, 8, 64, device="cuda")
    keep = buf.clone()
    q, k = buf[:, :4], buf[:, 4:6]
    for args, out in (((q, k), (k, k)), ((q, buf[:, 4:8]), (buf[:, 4:8], q)), ((q, k), (q, buf[:, 3:5])),
                      ((q, q), (q, q)), ((q, k), (buf[:, 2:6], torch.empty_like(k)))):
        with pytest.raises((splitkv.SplitKVError, ValueError)):
            rot.forward(pos, *args, out=out)
    assert torch.equal(buf, keep)
