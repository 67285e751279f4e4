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


def _accepted(dev="cuda"):
    g = torch.Generator().manual_seed(0)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.randperm(12, generator=g).int().view(3, 4).to(dev)
    return dict(table=table, lens=i(30, 0, 15), ptr=i(0, 4, 9, 11), path=i(0, 2, -1, 0, 1, 4, 0, -1, -1).view(3, 3),
                count=i(2, 3, 1))


def test_commit_between_views_of_one_arena(splitkv):
    """Keys beside values in every page, layers inside the pages, and the new rows behind them in the same buffer."""
    from context_block_sparse_b200.draft_tree import commit_draft
    a = _accepted()
    args = (a["table"], a["lens"])
    for layers_first in (True, False):
        cache = 2 * 12 * 2 * 16 * 2 * 64
        arena = torch.randn(cache + 2 * 2 * 11 * 2 * 64, device="cuda").bfloat16()
        new = arena[cache:].view(2, 2, 11, 2, 64)                                   # [k / v, layers, nodes, heads, d]
        pages = arena[:cache].view(2, 12, 2, 16, 2, 64) if layers_first else arena[:cache].view(12, 2, 2, 16, 2, 64).transpose(0, 1)
        k, v = pages[:, :, 0], pages[:, :, 1]
        kk, vv, kb, vb = k.clone(), v.clone(), new[0].clone(), new[1].clone()
        commit_draft(k, v, *args, new[0], new[1], a["ptr"], a["path"], a["count"])
        commit_draft(kk, vv, *args, kb, vb, a["ptr"], a["path"], a["count"])
        assert torch.equal(k, kk) and torch.equal(v, vv) and torch.equal(new[0], kb) and torch.equal(new[1], vb)


def test_commit_refuses_sources_in_a_cache(splitkv):
    from context_block_sparse_b200.draft_tree import commit_draft
    a = _accepted()
    k, v = (torch.randn(12, 16, 2, 64, device="cuda").bfloat16() for _ in range(2))
    keep, new = k.clone(), torch.randn(11, 2, 64, device="cuda").bfloat16()
    inside = k[3, :11]
    for kb, vb, kc, vc in ((inside, new, k, v), (new, inside, k, v), (new, new, k, k)):
        with pytest.raises(splitkv.SplitKVError):
            commit_draft(kc, vc, a["table"], a["lens"], kb, vb, a["ptr"], a["path"], a["count"])
    assert torch.equal(k, keep)
    commit_draft(k, v, a["table"], a["lens"], inside.clone(), new, a["ptr"], a["path"], a["count"])


@pytest.mark.parametrize("bound", [4, 5, 4000, 2 ** 31 - 1])
def test_commit_without_a_path_under_any_bound(splitkv, bound):
    """Every node in order; a bound below a sequence's nodes leaves that sequence out and is recorded."""
    from context_block_sparse_b200.draft_tree import check_status, commit_draft, new_status
    a = _accepted()
    k, v = (torch.randn(12, 16, 2, 64, device="cuda").bfloat16() for _ in range(2))
    kb, vb = (torch.randn(11, 2, 64, device="cuda").bfloat16() for _ in range(2))
    want, status = (k.clone(), v.clone()), new_status()
    for b in range(3):
        n0, n1, at = int(a["ptr"][b]), int(a["ptr"][b + 1]), int(a["lens"][b])
        for i in range(n1 - n0 if n1 - n0 <= bound else 0):
            page, slot = int(a["table"][b, (at + i) // 16]), (at + i) % 16
            want[0][page, slot], want[1][page, slot] = kb[n0 + i], vb[n0 + i]
    commit_draft(k, v, a["table"], a["lens"], kb, vb, a["ptr"], max_nodes=bound, status=status)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    if bound < 5:
        with pytest.raises(splitkv.SplitKVError):
            check_status(status)
    check_status(status)


def test_a_step_reports_what_it_left_out(splitkv):
    """tree.check() after the documented calls raises for a bad token, path row or page of any of them."""
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention, commit_draft, verify_draft
    a = _accepted()
    tree = SplitKVTreeAttention(4, 2, 64, 5)
    k, v = (torch.randn(12, 16, 2, 64, device="cuda").bfloat16() for _ in range(2))
    q, kb, vb = (torch.randn(11, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    probs = torch.softmax(torch.randn(11, 30, device="cuda"), -1)
    parents = torch.tensor([-1, 0, 1, 2, -1, 0, 1, 2, 3, -1, 0], dtype=torch.int32, device="cuda")
    tokens, u = torch.zeros(11, dtype=torch.int32, device="cuda"), torch.rand(11, device="cuda")

    def step(tokens=tokens, path=a["path"], table=a["table"]):
        tree.forward(q, kb, vb, a["ptr"], None, k, v, table, a["lens"], 0.125)
        verify_draft(probs, None, tokens, parents, a["ptr"], u, u[:3], max_nodes=5, status=tree.status)
        commit_draft(k, v, a["table"], a["lens"], kb, vb, a["ptr"], path, a["count"], status=tree.status)

    step()
    tree.check()
    bad_token, bad_path, bad_table = tokens.clone(), a["path"].clone(), a["table"].clone()
    bad_token[3], bad_path[1, 1], bad_table[0, 0] = 30, 5, 12
    for kw in (dict(tokens=bad_token), dict(path=bad_path), dict(table=bad_table)):
        step(**kw)
        with pytest.raises(splitkv.SplitKVError):
            tree.check()
        step()
        tree.check()
