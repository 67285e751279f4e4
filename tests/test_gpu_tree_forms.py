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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel,nodes", FORMS)
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.3, 1e-40])
def test_scale_of_any_sign(splitkv, monkeypatch, kernel, nodes, d, scale):
    """Masked scores are minus infinity under any scale: behind the context's end, in the tree, on pages of NaN."""
    monkeypatch.setenv("SPLITKV_TREE_KERNEL", kernel)
    for dt in ("bf16", "fp16"):
        c = Case([nodes, 3], [140, 0], 4, 1, d, 16, dt, seed=9)
        c.check(_forward(c, scale), ref=_ref(c, scale))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel,nodes", FORMS)
def test_rows_behind_the_last_sequence(splitkv, monkeypatch, kernel, nodes, d):
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    monkeypatch.setenv("SPLITKV_TREE_KERNEL", kernel)
    c = Case([nodes, 2], [300, 20], 4, 1, d, 16, extra=40, seed=2)
    tree = SplitKVTreeAttention(4, 1, d, c.max_nodes)
    o, lse = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda"), torch.full(c.q.shape[:2], 7.0, device="cuda")
    tree.forward(*(x.cuda() for x in (c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens)), d ** -0.5, o=o, lse=lse)
    assert (o[nodes + 2:] == 7).all() and (lse[nodes + 2:] == 7).all()
    c.check((o, lse))


@pytest.mark.parametrize("page", [1, 2, 4])
@pytest.mark.parametrize("nodes", [1, 9, 30, 90])
def test_pages_below_eight_tokens(splitkv, nodes, page):
    c = Case([nodes, max(1, nodes // 2)], [300, 77], 8, 2, 128, page, seed=nodes)
    c.check(c.call())


PAGES = 18000     # of 128 tokens of 1024 elements: 2.36e9 elements, 4.7 GB, for the keys and for the values


@pytest.fixture(scope="module")
def far_cache():
    k = torch.empty(PAGES, 128, 1024, dtype=torch.bfloat16, device="cuda")
    return k, torch.empty_like(k)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel,nodes", FORMS)
def test_cache_past_32_bits(splitkv, monkeypatch, far_cache, kernel, nodes, d):
    monkeypatch.setenv("SPLITKV_TREE_KERNEL", kernel)
    hkv = 1024 // d
    c = Case([nodes], [300], 4 * hkv, hkv, d, 128, seed=12)
    k, v = (x.view(PAGES, 128, hkv, d) for x in far_cache)
    table = torch.tensor([[PAGES - 1, 3, PAGES - 2]], dtype=torch.int32)
    for i in range(3):
        k[table[0, i]], v[table[0, i]] = c.k[c.table[0, i]].cuda(), c.v[c.table[0, i]].cuda()
    c.check(_forward(c, d ** -0.5, page_table=table, k_cache=k, v_cache=v))


def test_commit_into_a_cache_past_32_bits(splitkv, far_cache):
    from context_block_sparse_b200.draft_tree import commit_draft
    k, v = (x.view(PAGES, 128, 8, 128) for x in far_cache)
    g = torch.Generator().manual_seed(1)
    kb, vb = (torch.randn(5, 8, 128, generator=g).bfloat16().cuda() for _ in range(2))
    far, near = PAGES - 1, 2
    k[far], v[far], k[near], v[near] = 0, 0, 0, 0
    # the page where the low 32 bits of the far page's byte offset would land (17999 * 2^18 = 2^32 + 1615 * 2^18; its offset
    # in elements, 17999 * 2^17, is past 2^31 and below 2^32)
    alias = far * 2 ** 18 % 2 ** 32 // 2 ** 18
    assert alias == 1615
    k[alias], v[alias] = 0, 0
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    commit_draft(k, v, i(near, far)[None], i(126), kb, vb, i(0, 5), i(0, 1, 3, 4)[None], i(4))
    assert torch.equal(k[near, 126:], kb[:2]) and torch.equal(v[near, 126:], vb[:2])
    assert torch.equal(k[far, :2], kb[3:]) and torch.equal(v[far, :2], vb[3:])
    assert (k[far, 2:] == 0).all() and (k[near, :126] == 0).all() and (v[alias] == 0).all() and (k[alias] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel,nodes", FORMS)
@pytest.mark.parametrize("lens", [[300, 20, 0, 1500], [40] * 4])
def test_in_the_place_of_the_queries(splitkv, monkeypatch, kernel, nodes, d, lens):
    """o = q: the same bits as into memory of its own; over anything else it is refused."""
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    monkeypatch.setenv("SPLITKV_TREE_KERNEL", kernel)
    c = Case([nodes, 1, nodes, max(1, nodes // 2)] * 8, lens * 8, 8, 2, d, 16, seed=nodes)
    tree = SplitKVTreeAttention(8, 2, d, c.max_nodes)
    a = [x.cuda() for x in (c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens)]
    o, lse = tree.forward(*a, d ** -0.5)
    at = a[0].clone()
    got = tree.forward(at, *a[1:], d ** -0.5, o=at)
    assert got[0] is at and torch.equal(at, o) and torch.equal(got[1], lse)
    room = torch.zeros(2 * at.numel(), dtype=at.dtype, device="cuda")
    inner = room[8:8 + at.numel()].view(at.shape)
    with pytest.raises(splitkv.SplitKVError):
        tree.forward(inner, *a[1:], d ** -0.5, o=room[:at.numel()].view(at.shape))
    with pytest.raises(splitkv.SplitKVError):
        tree.forward(at, *a[1:], d ** -0.5, o=room[:at.numel()].view(at.shape), lse=room.view(torch.float32)[:lse.numel()].view(lse.shape))
