"""splitkv_tree_attn / SplitKVTreeAttention on the GPU against the 64-bit form."""

import numpy as np
import pytest
import torch

from draft_util import assert_within, random_parents, tree_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Case:
    """A cache with scattered pages, trees behind each sequence; everything unused holds NaN."""

    def __init__(self, counts, lens, hq, hkv, d, page, dt="bf16", kind="tree", seed=0, width=None, extra=0, spare=3):
        from context_block_sparse_b200.draft_tree import tree_mask
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        dt = DT[dt]
        B = len(counts)
        self.counts, self.hq, self.hkv, self.d, self.page = counts, hq, hkv, d, page
        self.max_nodes = max(1, max(counts)) if width is None else width
        ptr = np.concatenate([[0], np.cumsum(counts)])
        nq = int(ptr[-1]) + extra                       # rows behind the last sequence
        per = max(1, max(-(-n // page) for n in lens))
        pages = B * per + spare
        self.table = torch.from_numpy(rng.permutation(pages)[:B * per].astype(np.int32).reshape(B, per))
        rnd = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
        self.q, self.kb, self.vb = rnd(nq, hq, d), rnd(nq, hkv, d), rnd(nq, hkv, d)
        self.k = torch.full((pages, page, hkv, d), float("nan"), dtype=dt)
        self.v = self.k.clone()
        for b in range(B):
            t = torch.arange(lens[b])
            if len(t):
                self.k[self.table[b].long()[t // page], t % page] = rnd(len(t), hkv, d)
                self.v[self.table[b].long()[t // page], t % page] = rnd(len(t), hkv, d)
        self.ptr, self.lens = torch.from_numpy(ptr.astype(np.int32)), torch.tensor(lens, dtype=torch.int32)
        if kind == "block":
            self.mask = None
        else:
            par = np.concatenate([random_parents(rng, n, kind) for n in counts if n] or [np.zeros(0, int)])
            m = tree_mask(par, ptr, self.max_nodes)
            self.mask = torch.zeros(nq, self.max_nodes + seed % 3, dtype=torch.bool)   # odd row lengths
            self.mask[:m.shape[0], :self.max_nodes] = torch.from_numpy(m)

    def call(self, tree=None, out_dtype=None, **over):
        from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
        tree = tree or SplitKVTreeAttention(self.hq, self.hkv, self.d, self.max_nodes)
        dev = lambda x: x.cuda() if x is not None else None  # noqa: E731
        a = dict(q=self.q, kb=self.kb, vb=self.vb, node_ptr=self.ptr, mask=self.mask, k_cache=self.k, v_cache=self.v,
                 page_table=self.table, context_lens=self.lens)
        a.update(over)
        return tree.forward(*(dev(a[n]) for n in ("q", "kb", "vb", "node_ptr", "mask", "k_cache", "v_cache",
                                                   "page_table", "context_lens")), self.d ** -0.5, out_dtype=out_dtype)

    def ref(self):
        return tree_ref(self.q, self.kb, self.vb, self.ptr, self.mask, self.k, self.v, self.table, self.lens,
                        self.d ** -0.5)

    def check(self, got, out_dtype=None, ref=None, rows=None):
        o, lse, to, tl = ref or self.ref()
        n = int(self.ptr[-1]) if rows is None else rows
        assert_within("o", got[0][:n], o[:n], to[:n], out_dtype or self.q.dtype)
        assert_within("lse", got[1][:n], lse[:n], tl[:n], torch.float32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("counts,lens,hq,hkv,page", [
    ([1], [1], 1, 1, 16),                                  # one token behind one token
    ([1], [0], 4, 1, 16),                                  # no context at all
    ([3], [1000], 8, 2, 16),
    ([16] * 5, [0, 1, 63, 64, 65], 8, 2, 32),               # around a key tile
    ([1, 0, 7, 4], [130, 77, 0, 513], 8, 8, 64),            # a sequence without nodes, heads of their own
    ([17, 30], [300, 31], 4, 2, 16),                        # 17 nodes: two row groups, ragged
    ([5, 8], [700, 129], 32, 4, 128),                       # eight heads a KV head
    ([40, 64, 1], [200, 333, 50], 4, 1, 256),               # many row tiles
    ([256, 3], [70, 640], 2, 1, 8),                         # the widest tree; pages of 8
    ([2, 2], [129, 5], 3, 1, 1),                            # pages of a single token, three heads
    ([20, 32, 17], [130, 700, 0], 4, 1, 64),                # one full row tile, ragged
    ([33, 64, 20], [1000, 127, 300], 16, 4, 128),           # pairs of row tiles, some with one of them empty
    ([3, 2], [129, 256], 80, 1, 16),                        # 80 heads on one: a node's rows cross the row groups
    ([130, 129, 1], [128, 0, 127], 3, 1, 32),               # two tree tiles; rows of a node across row tiles
    ([32, 30, 5], [1000, 257, 130], 8, 2, 64),              # row tiles of 128 rows, odd and even numbers of key tiles
    ([128, 100], [0, 600], 2, 2, 16),                       # 128 nodes
])
def test_matches_64_bits(splitkv, counts, lens, hq, hkv, page, dt, d):
    c = Case(counts, lens, hq, hkv, d, page, dt, seed=len(counts) + page)
    c.check(c.call())


@pytest.mark.parametrize("kind", ["chain", "block"])
@pytest.mark.parametrize("out", [None, torch.float32])
def test_masks_and_float32_output(splitkv, kind, out):
    c = Case([9, 16, 2], [400, 17, 0], 8, 2, 128, 32, kind=kind, seed=4)
    c.check(c.call(out_dtype=out), out)


@pytest.mark.parametrize("B", [129, 300])
def test_many_sequences(splitkv, B):
    """More sequences than threads of a CTA, many of them short or empty."""
    rng = np.random.default_rng(B)
    counts = rng.integers(0, 4, B).tolist()
    lens = (rng.integers(0, 90, B) * (rng.random(B) < 0.7)).tolist()
    c = Case(counts, lens, 4, 2, 64, 16, seed=B, width=4)
    c.check(c.call())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [1, 4, 12, 30, 60])
@pytest.mark.parametrize("out", [None, torch.float32])
def test_more_units_than_ctas(splitkv, nodes, d, out):
    """Units that lie in one CTA's stretch, of one key tile and of several, beside such as are cut."""
    rng = np.random.default_rng(nodes)
    counts = np.minimum(nodes, rng.integers(nodes // 2, nodes + 1, 48).clip(1)).tolist()
    lens = rng.integers(0, 700, 48).tolist()
    c = Case(counts, lens, 32, 8, d, 64, seed=nodes, width=nodes)
    c.check(c.call(out_dtype=out), out)


def test_long_context_and_wide_rows(splitkv):
    c = Case([8, 33], [9001, 4100], 8, 2, 128, 64, seed=11)
    c.check(c.call())


def test_rows_that_see_nothing_and_lowest_scores(splitkv):
    """Rows without a key give 0 and -inf; scores at the type's lowest finite value still count."""
    c = Case([6, 5], [0, 40], 4, 2, 64, 16, seed=3)
    c.mask[1] = False
    c.mask[4] = False
    c.mask[7] = False                      # sees its context only
    got = c.call()
    c.check(got)
    assert (got[0][1] == 0).all() and (got[1][4] == float("-inf")).all()
    c.q[:] = 0
    c.q[..., 0] = 1e4
    c.k[..., 0] = -1e4                     # every context score is -1e8 / 8; the tree's are ordinary
    c.kb[..., 0] = 0
    ref = c.ref()
    c.check(c.call(), ref=ref)
    c.kb[..., 0] = -1e4
    ref = c.ref()
    got = c.call()
    c.check(got, ref=ref)
    assert torch.isfinite(got[1][5:].cpu()).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(8, 4), (4, 4)])
def test_unseen_values_stay_away(splitkv, value, d, heads):
    """Infinities and NaN in nodes that a row does not see, in cache slots behind the context, in pages of nobody:
    only the rows that see them meet them."""
    c = Case([12, 70], [35, 100], *heads, d, 16, seed=6)     # the cache's unused slots are NaN already
    c.mask[0, 0], c.mask[12, 0] = True, True
    dark = [3, 12 + 40, 12 + 66]                             # nodes that only themselves see
    for r in dark:
        b0 = 0 if r < 12 else 12
        for i in range(b0, 12 if b0 == 0 else 82):
            if i != r:
                c.mask[i, r - b0] = False
        c.vb[r, :, 5] = value
    c.vb[12 + 41, 1, 9] = value                              # and one that others may see
    c.check(c.call())
    c.kb[3] = value                                          # an unseen key's score is no number
    c.mask[3, 3] = False
    c.check(c.call())


def test_rows_behind_the_last_sequence(splitkv):
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    c = Case([3, 4], [50, 20], 4, 2, 64, 16, extra=5, seed=2)
    tree = SplitKVTreeAttention(4, 2, 64, c.max_nodes)
    o = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full(c.q.shape[:2], 7.0, device="cuda")
    a = [x.cuda() for x in (c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens)]
    tree.forward(*a, 64 ** -0.5, o=o, lse=lse)
    assert (o[7:] == 7).all() and (lse[7:] == 7).all()
    c.check((o, lse))


def test_strides(splitkv):
    """Queries inside a fused projection, keys and values interleaved in one cache, a head-major cache."""
    c = Case([9, 4], [200, 90], 4, 2, 128, 16, seed=8)
    ref = c.ref()
    qkv = torch.cat([c.q, c.kb, c.vb], 1).cuda()
    both = torch.stack([c.k, c.v], 1).cuda()                       # [pages, 2, page, heads, d]
    hm = both.permute(0, 1, 3, 2, 4).contiguous()                  # [pages, 2, heads, page, d]
    table = torch.cat([c.table, c.table], 1).cuda()[:, :c.table.shape[1]]
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    tree = SplitKVTreeAttention(4, 2, 128, c.max_nodes)
    for kc, vc in ((both[:, 0], both[:, 1]), (hm[:, 0].transpose(1, 2), hm[:, 1].transpose(1, 2))):
        got = tree.forward(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], c.ptr.cuda(), c.mask.cuda(), kc, vc, table, c.lens.cuda(),
                           128 ** -0.5)
        c.check(got, ref=ref)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scale_of_any_sign(splitkv, scale):
    for nodes in (5, 60):
        _check_scale(Case([nodes], [140], 4, 2, 64, 16, seed=9), scale)


def _check_scale(c, scale):
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    tree = SplitKVTreeAttention(4, 2, 64, c.max_nodes)
    got = tree.forward(*(x.cuda() for x in (c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens)), scale)
    c.check(got, ref=tree_ref(c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens, scale))


def test_bad_device_arrays_are_recorded_and_skipped(splitkv):
    """A page outside the cache, a length beyond the table and a node range beyond the rows: absent, and recorded."""
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    c = Case([4, 4, 4], [100, 60, 30], 4, 2, 64, 16, seed=5)
    tree = SplitKVTreeAttention(4, 2, 64, c.max_nodes)
    good = c.call(tree)
    tree.check()
    for bad_page in (-1, -2, -3, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[1, 1] = bad_page                                     # keys 16..31 of sequence 1
        got = c.call(tree, page_table=table)
        with pytest.raises(splitkv.SplitKVError):
            tree.check()
        assert torch.equal(got[0][:4], good[0][:4]) and torch.equal(got[0][8:], good[0][8:])
        keep = torch.cat([torch.arange(16), torch.arange(32, 60)])
        c2 = Case([4, 4, 4], [100, 60, 30], 4, 2, 64, 16, seed=5)
        # the same sequence with those keys moved out: gather the kept ones into its pages
        pages = c2.table[1].long()
        kk, vv = c.k[pages[keep // 16], keep % 16].clone(), c.v[pages[keep // 16], keep % 16].clone()
        t = torch.arange(len(keep))
        c2.k[pages[t // 16], t % 16], c2.v[pages[t // 16], t % 16] = kk, vv
        c2.lens[1] = len(keep)
        c2.check(got)
    lens = c.lens.clone()
    lens[2] = 10 ** 6
    c.call(tree, context_lens=lens)        # clamped to the table: reads the sequence's own pages only
    with pytest.raises(splitkv.SplitKVError):
        tree.check()
    lens[2] = -5
    got = c.call(tree, context_lens=lens)
    with pytest.raises(splitkv.SplitKVError):
        tree.check()
    # (another length moves the cuts between the CTAs: the other sequences' results keep their values, not their bits)
    c.check(got, rows=8)
    ptr = c.ptr.clone()
    ptr[3] = 99                            # past the rows: the last sequence has no nodes
    got = c.call(tree, node_ptr=ptr)
    with pytest.raises(splitkv.SplitKVError):
        tree.check()
    c.check(got, rows=8)
    tree.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [20, 60, 120])
def test_bad_pages_under_wide_trees(splitkv, nodes, d):
    """The same in row tiles of 64, 128 and 256 rows: keys on bad pages are absent, whatever half or tile they are in."""
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    lens = [300, 200]
    c = Case([nodes, nodes - 7], lens, 4, 2, d, 16, seed=15)
    tree = SplitKVTreeAttention(4, 2, d, c.max_nodes)
    table = c.table.clone()
    table[0, 6], table[0, 17], table[1, 0], table[1, 12] = -1, c.k.shape[0], -2 ** 31, 2 ** 31 - 1
    got = c.call(tree, page_table=table)
    with pytest.raises(splitkv.SplitKVError):
        tree.check()
    c2 = Case([nodes, nodes - 7], lens, 4, 2, d, 16, seed=15)
    for b, bad in enumerate(([6, 17], [0, 12])):
        keep = torch.tensor([t for t in range(lens[b]) if t // 16 not in bad])
        pages, t = c.table[b].long(), torch.arange(len(keep))
        c2.k[pages[t // 16], t % 16] = c.k[pages[keep // 16], keep % 16]
        c2.v[pages[t // 16], t % 16] = c.v[pages[keep // 16], keep % 16]
        c2.lens[b] = len(keep)
    c2.check(got)


@pytest.mark.parametrize("kernel", ["mma", "tcgen05"])
@pytest.mark.parametrize("counts,lens,hq,hkv,d", [
    ([1], [3000], 8, 2, 128), ([3, 2], [64, 700], 8, 2, 64), ([40, 9], [513, 20], 4, 1, 128), ([30, 7], [300, 0], 8, 2, 64)])
def test_asked_kernel(splitkv, monkeypatch, kernel, counts, lens, hq, hkv, d):
    monkeypatch.setenv("SPLITKV_TREE_KERNEL", kernel)
    c = Case(counts, lens, hq, hkv, d, 16, seed=17)
    c.check(c.call())


def test_offsets_past_32_bits(splitkv):
    """Pages beyond 2^31 elements (and 2^32 bytes) of a large cache."""
    c = Case([6], [300], 8, 8, 128, 128, seed=12)
    ref = c.ref()
    pages = 18000                                                  # 2.36e9 elements, 4.7 GB each
    k = torch.empty(pages, 128, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    for i in range(3):
        k[table[0, i]], v[table[0, i]] = c.k[c.table[0, i]].cuda(), c.v[c.table[0, i]].cuda()
    got = c.call(page_table=table.cuda(), k_cache=k, v_cache=v)
    c.check(got, ref=ref)


@pytest.mark.parametrize("args", [([6], [300], 8, 8, 128, 128), ([16, 9], [900, 257], 8, 2, 128, 64),
                                  ([40], [2000], 4, 1, 64, 16), ([32, 20], [700, 1500], 8, 2, 64, 64),
                                  ([60, 33], [1500, 400], 8, 2, 128, 64)])
def test_cold_caches(splitkv, args):
    """Late keys and values (nothing in L2, the GPU just woken): products queue up behind the softmax's waits."""
    import time
    c = Case(*args, seed=12)
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    tree = SplitKVTreeAttention(c.hq, c.hkv, c.d, c.max_nodes)
    a = [x.cuda() for x in (c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens)]
    ref = c.ref()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for k in range(6):
        flush.fill_(k)
        torch.cuda.synchronize()
        time.sleep(0.02)
        c.check(tree.forward(*a, c.d ** -0.5), ref=ref)


def test_streams_graphs_and_determinism(splitkv):
    """Another stream; two captured graphs replayed at once with changed lengths and data (each has its own workspace);
    the same bits every time."""
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    c = Case([8, 16, 3], [900, 70, 2000], 8, 2, 128, 32, seed=13)
    tree = SplitKVTreeAttention(8, 2, 128, c.max_nodes)
    a = [x.cuda() for x in (c.q, c.kb, c.vb, c.ptr, c.mask, c.k, c.v, c.table, c.lens)]
    want = tree.forward(*a, 128 ** -0.5)
    c.check(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [tree.forward(*a, 128 ** -0.5) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(tree.forward(*a, 128 ** -0.5))
        graphs.append(gr)
    a[8].copy_(torch.tensor([33, 0, 1500], dtype=torch.int32))     # new lengths
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    c.lens = torch.tensor([33, 0, 1500], dtype=torch.int32)
    ref = c.ref()
    for out in outs:
        c.check(out, ref=ref)
        assert torch.equal(out[0], outs[0][0]) and torch.equal(out[1], outs[0][1])


def test_refusals(splitkv):
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention
    c = Case([3], [20], 4, 2, 64, 16)
    with pytest.raises(ValueError, match="node_ptr"):
        c.call(node_ptr=c.ptr.long())
    with pytest.raises(ValueError, match="columns"):
        c.call(mask=c.mask[:, :1])
    with pytest.raises(ValueError, match="mask must be"):
        c.call(mask=c.mask.float())
    with pytest.raises(ValueError, match="kb must be"):
        c.call(kb=c.kb.half())
    with pytest.raises(ValueError, match="v_cache has shape"):
        c.call(v_cache=c.v[:-1])
    with pytest.raises(ValueError, match="context_lens"):
        c.call(context_lens=c.lens[:0])
    with pytest.raises(splitkv.SplitKVError):                       # pages of 12
        c.call(k_cache=c.k[:, :12], v_cache=c.v[:, :12])
    with pytest.raises(splitkv.SplitKVError):                       # 257 nodes
        c.call(SplitKVTreeAttention(4, 2, 64, 257), mask=None)
    odd = torch.zeros(3, 4, 72, dtype=torch.bfloat16, device="cuda")[..., 4:68]    # rows off 16 bytes
    with pytest.raises(splitkv.SplitKVError):
        c.call(q=odd)
    empty = c.call(q=c.q[:0], kb=c.kb[:0], vb=c.vb[:0], mask=c.mask[:0], node_ptr=torch.zeros(2, dtype=torch.int32))
    assert empty[0].shape == (0, 4, 64)
