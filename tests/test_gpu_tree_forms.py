"""Tree attention in every form of its kernels: row tiles of 16, 32 and 64 rows on mma.sync, of 32, 64, 128 and 256 on
tcgen05."""

import pytest
import torch

from draft_util import assert_within, tree_ref
from test_gpu_tree_attn import Case

pytestmark = pytest.mark.gpu

# kernel, nodes of G = 4 query heads a KV head (the row tile's rows); at d = 64 128 rows are another form than at d = 128
FORMS = [("mma", 4), ("mma", 8), ("mma", 30), ("tcgen05", 4), ("tcgen05", 15), ("tcgen05", 30), ("tcgen05", 60)]


def _forward(c, scale, **over):
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    a = dict(q=c.q, kb=c.kb, vb=c.vb, node_ptr=c.ptr, mask=c.mask, k_cache=c.k, v_cache=c.v, page_table=c.table,
             context_lens=c.lens)
    a.update(over)
    tree = SplitKVTreeAttention(c.hq, c.hkv, c.d, c.max_nodes)
    got = tree.forward(*(None if x is None else x.cuda() for x in a.values()), scale)
    tree.check()
    return got


def _ref(c, scale):
    return tree_ref(c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel,nodes", FORMS)
@pytest.mark.parametrize("at,gap", [(0, 12), (0, 15), (0, 18), (9000, 15), (-1, 18), (9000, 2), (0, 2)])
def test_weights_far_below_the_largest(splitkv, monkeypatch, kernel, nodes, d, at, gap):
    """float16: one key (of the context, or node 0) stands `gap` above all others, and its V is 0 (for a small gap: 1), so
    that O is what the others weigh together.  A weight is held to 2^-11 of itself, or to 2^-37 of the row's largest
    where that is more (P is lifted to 2^12 at the reference, and float16 is good to 2^-25): sum |v| 2^-37 on top of the
    ordinary bound."""
    monkeypatch.setenv("SPLITKV_TREE_KERNEL", kernel)
    c = Case([nodes], [10000], 4, 1, d, 64, "fp16", kind="block", seed=nodes)
    for x in (c.q, c.kb, c.k):
        x.zero_()
    c.q[..., 0] = 8.0
    where = (c.table[0, at // 64].item(), at % 64) if at >= 0 else None
    key, v = (c.kb[0], c.vb[0]) if where is None else (c.k[where], c.v[where])
    c.v.abs_()
    c.vb.abs_()
    key[:, 0] = float(gap)
    v[:] = 1.0 if gap < 3 else 0.0
    scale = 0.125
    o, lse, to, tl = _ref(c, scale)
    vs = c.v[c.table[0].long()].flatten(0, 1)[:10000, 0].double().abs().sum(0) + c.vb[:, 0].double().abs().sum(0)
    got = _forward(c, scale)
    assert_within("o", got[0], o, to + vs * 2.0 ** -37, torch.float16)
    assert_within("lse", got[1], lse, tl, torch.float32)
