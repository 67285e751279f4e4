"""Verification and commit on the GPU against their 64-bit forms, and whole speculative steps."""

import numpy as np
import pytest
import torch

from draft_util import random_parents, tree_ref, assert_within, verify_ref

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _drafts(counts, V, kind, seed, dt=torch.float32, certain=False, sharp=2.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    ptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(ptr[-1])
    parents = np.concatenate([random_parents(rng, c, kind) for c in counts if c] or [np.zeros(0, int)]).astype(np.int32)
    logits = torch.randn(n, V, generator=g) * sharp
    target = torch.softmax(logits, -1).to(dt)
    draft = torch.softmax(logits + 0.7 * torch.randn(n, V, generator=g), -1).to(dt)
    rows = torch.from_numpy((parents + np.repeat(ptr[:-1], counts)).clip(0)).long()
    tokens = torch.multinomial(draft[rows].float(), 1, generator=g)[:, 0] if n else torch.zeros(0, dtype=torch.int64)
    return dict(target=target, draft=None if certain else draft, tokens=tokens.int(), parents=torch.from_numpy(parents),
                node_ptr=torch.from_numpy(ptr), u_accept=torch.rand(n, generator=g),
                u_sample=torch.rand(len(counts), generator=g)), max(1, max(counts, default=1))


def _verify(a, max_nodes, max_path=None, status=None, **over):
    from context_block_sparse_b200.draft_tree import verify_draft
    a = {**a, **over}
    dev = {k: v.cuda() if v is not None else None for k, v in a.items()}
    return verify_draft(dev["target"], dev["draft"], dev["tokens"], dev["parents"], dev["node_ptr"], dev["u_accept"],
                        dev["u_sample"], max_nodes, max_path, status)


def _same(got, a, max_path):
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    want = verify_ref(f(a["target"]), f(a["draft"]), a["tokens"].numpy(), a["parents"].numpy(), a["node_ptr"].numpy(),
                      f(a["u_accept"]), f(a["u_sample"]), max_path)
    for name, x, y in zip(("path", "count", "next"), got, want):
        assert np.array_equal(x.cpu().numpy(), y), name
    return want


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("counts,V", [([1], 1), ([2], 5), ([16], 32000), ([7, 1, 0, 12], 1001), ([40, 33, 20], 4096),
                                      ([5] * 33, 517), ([9, 4], 70001)])
def test_verify_matches_the_walk(splitkv, counts, V, dt, kind, certain):
    for seed in range(3):
        a, mx = _drafts(counts, V, kind, seed, DT[dt], certain)
        _same(_verify(a, mx), a, mx)


def test_verify_covers_every_ending(splitkv):
    """Among many small trees: full acceptance, a first rejection, several rejected siblings."""
    seen = set()
    for certain in (False, True):
        a, mx = _drafts([6] * 400, 12, "tree", 5, certain=certain, sharp=1.0)
        _, count, _ = _same(_verify(a, mx), a, mx)
        seen |= set(count.tolist())
    assert {1, 2, 3} <= seen


def test_verify_tokens_int64_and_short_paths(splitkv):
    a, mx = _drafts([10, 10, 3], 300, "chain", 1, sharp=0.0)
    a["draft"] = a["target"].clone()                    # equal rows: everything is accepted
    got = _verify(a, mx, tokens=a["tokens"].long())
    assert got[2].dtype == torch.int64 and got[1].tolist() == [10, 10, 3]
    _same(got, a, mx)
    short = _verify(a, mx, max_path=4)
    assert short[0].shape == (3, 4) and short[1].tolist() == [4, 4, 3]
    _same(short, a, 4)


def test_verify_strided_rows(splitkv):
    a, mx = _drafts([8, 5], 1024, "tree", 2)
    wide = torch.zeros(13, 1030)
    wide[:, :1024] = a["target"]
    both = torch.zeros(2, 13, 1027)
    both[1, :, 3:] = a["draft"]
    from context_block_sparse_b200.draft_tree import verify_draft
    d = {k: v.cuda() for k, v in a.items()}
    got = verify_draft(wide.cuda()[:, :1024], both.cuda()[1, :, 3:], d["tokens"], d["parents"], d["node_ptr"],
                       d["u_accept"], d["u_sample"], mx)
    _same(got, a, mx)


def test_verify_edges(splitkv):
    """Residuals without mass, rows without mass, infinities and NaN, numbers at 0 and just below 1, equal siblings."""
    V = 2000
    t, q = torch.zeros(3, V), torch.zeros(3, V)
    t[:, 7], q[:, 7] = 0.5, 1.0
    t[:, 1999] = 0.5
    base = dict(target=t, draft=q, tokens=torch.tensor([0, 7, 7]).int(), parents=torch.tensor([-1, 0, 0]).int(),
                node_ptr=torch.tensor([0, 3]).int(), u_accept=torch.tensor([0.0, 0.75, 0.75]),
                u_sample=torch.tensor([0.3]))
    got = _verify(base, 3)
    assert _same(got, base, 3)[2][0] == 1999 and got[1].item() == 1     # both rejected: what is left is 1999
    for us in (0.0, float(np.nextafter(np.float32(1), np.float32(0)))):
        a, mx = _drafts([6, 6], 5000, "tree", 3)
        a["u_sample"][:] = us
        _same(_verify(a, mx), a, mx)
        a["u_accept"][:] = us
        _same(_verify(a, mx), a, mx)
    none = dict(base, target=torch.zeros(3, V))
    got = _verify(none, 3)
    assert got[2].item() == -1 and got[1].item() == 1
    lost = dict(base, target=q * 0.25, u_accept=torch.tensor([0.0, 0.9, 0.9]))   # the residual is empty: p itself
    assert _same(_verify(lost, 3), lost, 3)[2][0] == 7
    odd = {k: v.clone() for k, v in base.items()}
    odd["target"][:, 5], odd["target"][:, 6], odd["target"][:, 8] = float("nan"), float("inf"), -1.0
    odd["draft"][:, 1999] = float("nan")
    _same(_verify(odd, 3), odd, 3)


@pytest.mark.parametrize("u,token", [(-0.5, 1), (float("nan"), 1), (float("-inf"), 1), (1.0, 3), (2.5, 3), (float("inf"), 3)])
def test_verify_numbers_outside_the_unit_interval(splitkv, u, token):
    """A next token is the first or the last one with mass, never left unwritten."""
    a = dict(target=torch.tensor([[0.0, 0.25, 0.5, 0.25, 0.0]]), draft=None, tokens=torch.zeros(1).int(),
             parents=torch.tensor([-1]).int(), node_ptr=torch.tensor([0, 1]).int(), u_accept=torch.zeros(1),
             u_sample=torch.tensor([u]))
    assert _verify(a, 1)[2].item() == token


def test_verify_bad_nodes_are_recorded(splitkv):
    from context_block_sparse_b200.draft_tree import check_status, new_status
    status = new_status()
    a, mx = _drafts([6, 6], 100, "tree", 4)
    _verify(a, mx, status=status)
    check_status(status)
    for name, at, value in (("tokens", 2, 100), ("tokens", 8, -1), ("parents", 3, 3), ("parents", 9, -7),
                            ("parents", 4, 2 ** 31 - 1)):
        b = {k: v.clone() for k, v in a.items()}
        b[name][at] = value
        got = _verify(b, mx, status=status)
        with pytest.raises(splitkv.SplitKVError):
            check_status(status)
        _same(got, b, mx)                                  # that node is never reached
    for ptr in ([0, 6, 99], [0, 7, 6], [-3, 6, 12]):
        got = _verify(a, mx, status=status, node_ptr=torch.tensor(ptr).int())
        with pytest.raises(splitkv.SplitKVError):
            check_status(status)
    assert got[1][0].item() == 0 and got[2][0].item() == -1 and (got[0][0] == -1).all()


@pytest.mark.parametrize("certain", [False, True])
def test_verify_keeps_the_targets_distribution(splitkv, certain):
    """The first token behind the root over 200k sequences: each frequency within five standard deviations of p."""
    V, B, k = 6, 200000, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.softmax(torch.randn(V, generator=g, device="cuda") * 1.2, 0)
    q = torch.softmax(torch.randn(V, generator=g, device="cuda") * 1.2, 0)
    n = B * (k + 1)
    if certain:
        kids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:k]]).expand(B, k)
    else:
        kids = torch.multinomial(q.expand(B, V), k, replacement=True, generator=g)
    tokens = torch.cat([torch.zeros(B, 1, dtype=torch.int64, device="cuda"), kids], 1).reshape(-1)
    parents = torch.tensor([-1] + [0] * k, dtype=torch.int32, device="cuda").repeat(B)
    from context_block_sparse_b200.draft_tree import verify_draft
    path, count, nxt = verify_draft(p.expand(n, V), None if certain else q.expand(n, V), tokens.int(), parents,
                                    torch.arange(0, n + 1, k + 1, dtype=torch.int32, device="cuda"),
                                    torch.rand(n, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda"),
                                    max_nodes=k + 1)
    taken = path[:, 1].long()
    first = torch.where(taken > 0, tokens.view(B, k + 1).gather(1, taken.clamp(min=0)[:, None])[:, 0], nxt.long())
    freq = torch.bincount(first, minlength=V).double() / B
    sd = torch.sqrt(p.double() * (1 - p.double()) / B)
    assert ((freq - p.double()).abs() <= 5 * sd).all(), (freq, p)


# ------------------------------------------------------------------------------------- commit
def _commit_case(layers, counts, lens, page, hkv, d, dt, seed, es=None):
    rng = np.random.default_rng(seed)
    B = len(counts)
    ptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    per = max(-(-(n + c) // page) for n, c in zip(lens, counts)) + 1
    table = torch.from_numpy(rng.permutation(B * per).astype(np.int32).reshape(B, per))
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    D = max(1, max(counts))
    acc = np.array([rng.integers(0, c + 1) for c in counts], dtype=np.int32)
    path = np.full((B, D), -1, dtype=np.int32)
    for b in range(B):
        path[b, :acc[b]] = np.sort(rng.permutation(counts[b])[:acc[b]])
    return dict(k=rnd(layers, B * per, page, hkv, d), v=rnd(layers, B * per, page, hkv, d), table=table,
                lens=torch.tensor(lens, dtype=torch.int32), kb=rnd(layers, int(ptr[-1]), hkv, d),
                vb=rnd(layers, int(ptr[-1]), hkv, d), ptr=torch.from_numpy(ptr), path=torch.from_numpy(path),
                count=torch.from_numpy(acc)), page


def _commit_ref(a, page, whole=False):
    k, v = a["k"].clone(), a["v"].clone()
    for b in range(len(a["lens"])):
        n0 = int(a["ptr"][b])
        nodes = range(int(a["ptr"][b + 1]) - n0) if whole else a["path"][b, :int(a["count"][b])].tolist()
        for i, node in enumerate(nodes):
            t = int(a["lens"][b]) + i
            at = int(a["table"][b, t // page]), t % page
            k[:, at[0], at[1]], v[:, at[0], at[1]] = a["kb"][:, n0 + node], a["vb"][:, n0 + node]
    return k, v


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("layers,counts,lens,page,hkv,d", [
    (1, [1], [0], 16, 1, 64), (3, [5, 9, 2], [15, 16, 17], 16, 2, 128), (2, [40, 1], [0, 1000], 64, 8, 128),
    (1, [200], [3], 1, 3, 64), (4, [16] * 20, list(range(20)), 32, 4, 64)])
def test_commit(splitkv, layers, counts, lens, page, hkv, d, dt):
    from context_block_sparse_b200.draft_tree import commit_draft
    for whole in (False, True):
        a, page = _commit_case(layers, counts, lens, page, hkv, d, DT[dt], len(counts))
        c = {n: x.cuda() for n, x in a.items()}
        args = dict(max_nodes=max(counts)) if whole else dict(path=c["path"], count=c["count"])
        if layers == 1:
            commit_draft(c["k"][0], c["v"][0], c["table"], c["lens"], c["kb"][0], c["vb"][0], c["ptr"], **args)
        else:
            commit_draft(c["k"], c["v"], c["table"], c["lens"], c["kb"], c["vb"], c["ptr"], **args)
        k, v = _commit_ref(a, page, whole)
        assert torch.equal(c["k"].cpu(), k) and torch.equal(c["v"].cpu(), v)


def test_commit_strides_and_bad_entries(splitkv):
    from context_block_sparse_b200.draft_tree import check_status, commit_draft, new_status
    a, page = _commit_case(2, [6, 7], [10, 3], 16, 2, 64, torch.bfloat16, 1)
    a["count"][:] = 5
    a["path"][:, :5] = torch.arange(5).int()
    both = torch.stack([a["k"], a["v"]], 2).cuda()                 # [layers, pages, 2, page, heads, d]
    new = torch.cat([a["kb"], a["vb"]], 2).cuda()                  # [layers, nodes, 2 heads, d]
    c = {n: x.cuda() for n, x in a.items()}
    status = new_status()
    commit_draft(both[:, :, 0], both[:, :, 1], c["table"], c["lens"], new[:, :, :2], new[:, :, 2:], c["ptr"], c["path"],
                 c["count"], status=status)
    k, v = _commit_ref(a, page)
    assert torch.equal(both[:, :, 0].cpu(), k) and torch.equal(both[:, :, 1].cpu(), v)
    check_status(status)

    def bad(**over):
        x = {**c, **{n: t.cuda() for n, t in over.items()}, "k": a["k"].cuda(), "v": a["v"].cuda()}
        commit_draft(x["k"], x["v"], x["table"], x["lens"], x["kb"], x["vb"], x["ptr"], x["path"], x["count"], status=status)
        with pytest.raises(splitkv.SplitKVError):
            check_status(status)
        return x["k"].cpu(), x["v"].cpu()

    path = a["path"].clone()
    path[0, 2] = 6                                                 # not a node of sequence 0
    path[1, 1] = -1
    got = bad(path=path)
    k, v = _commit_ref(a, page)
    for b, i in ((0, 2), (1, 1)):                                  # those rows are left as they were
        t = int(a["lens"][b]) + i
        at = int(a["table"][b, t // page]), t % page
        k[:, at[0], at[1]], v[:, at[0], at[1]] = a["k"][:, at[0], at[1]], a["v"][:, at[0], at[1]]
    assert torch.equal(got[0], k) and torch.equal(got[1], v)
    table = a["table"].clone()
    table[:, :2] = torch.tensor([[-1, 10 ** 6], [2 ** 31 - 1, -2 ** 31]]).int()
    assert torch.equal(bad(table=table)[0], a["k"])
    assert torch.equal(bad(lens=torch.tensor([10 ** 6, 2 ** 31 - 1]).int())[0], a["k"])
    assert torch.equal(bad(lens=torch.tensor([-1, -2 ** 31]).int())[0], a["k"])
    assert torch.equal(bad(count=torch.tensor([8, -1]).int())[0], a["k"])
    assert torch.equal(bad(ptr=torch.tensor([-2, 30, 20]).int())[0], a["k"])
    with pytest.raises(ValueError, match="share memory"):
        commit_draft(c["k"][:1].expand(2, -1, -1, -1, -1), c["v"], c["table"], c["lens"], c["kb"], c["vb"], c["ptr"],
                     c["path"], c["count"])


# ----------------------------------------------------------------------------- a run of them
@pytest.mark.parametrize("captured", [False, True])
def test_speculative_steps(splitkv, captured):
    """Three steps of a two-layer toy target: rotary positions, tree attention, verification, commit and the lengths'
    advance, eagerly and as one captured graph; every step against the plain forms on the state that it started from."""
    from context_block_sparse_b200.draft_tree import (SplitKVTreeAttention, commit_draft, tree_mask, verify_draft)
    from context_block_sparse_b200.rotary import Rotary
    L, B, T, hq, hkv, d, page, V = 2, 3, 7, 4, 2, 64, 16, 50
    rng = np.random.default_rng(0)
    ptr = np.arange(0, B * T + 1, T).astype(np.int32)
    parents = np.concatenate([random_parents(rng, T, "tree") for _ in range(B)]).astype(np.int32)
    depth = np.zeros(B * T, dtype=np.int32)
    for i, p in enumerate(parents):
        depth[i] = 0 if p < 0 else depth[i - i % T + p] + 1
    mask = torch.from_numpy(tree_mask(parents, ptr, T)).cuda()
    rot, tree = Rotary(d, base=1000.0), SplitKVTreeAttention(hq, hkv, d, T)
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    kc, vc = (rnd(L, 12, page, hkv, d).bfloat16() for _ in range(2))
    table = torch.from_numpy(rng.permutation(12).astype(np.int32).reshape(B, 4)).cuda()
    lens = torch.tensor([5, 16, 30], dtype=torch.int32, device="cuda")
    nptr, par = torch.from_numpy(ptr).cuda(), torch.from_numpy(parents).cuda()
    dep, seq = torch.from_numpy(depth).cuda(), torch.arange(B * T, device="cuda") // T
    x = dict(q=rnd(L, B * T, hq, d).bfloat16(), kb=rnd(L, B * T, hkv, d).bfloat16(), vb=rnd(L, B * T, hkv, d).bfloat16(),
             p=torch.softmax(rnd(B * T, V), -1), qd=torch.softmax(rnd(B * T, V), -1),
             tok=torch.randint(0, V, (B * T,), generator=g, device="cuda").int(),
             ua=torch.rand(B * T, generator=g, device="cuda"), us=torch.rand(B, generator=g, device="cuda"))
    out = {}

    def step():
        pos = lens[seq] + dep
        kbs, outs = [], []
        for layer in range(L):
            q, kb = rot.forward(pos, x["q"][layer], x["kb"][layer])
            outs.append(tree.forward(q, kb, x["vb"][layer], nptr, mask, kc[layer], vc[layer], table, lens, d ** -0.5) + (q,))
            kbs.append(kb)
        out["kb"] = torch.stack(kbs)
        out["att"] = outs
        out["v"] = verify_draft(x["p"], x["qd"], x["tok"], par, nptr, x["ua"], x["us"], max_nodes=T)
        commit_draft(kc, vc, table, lens, out["kb"], x["vb"], nptr, out["v"][0], out["v"][1])
        lens.add_(out["v"][1])

    state = [kc.clone(), vc.clone(), lens.clone()]
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()                       # warm up
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, was in zip((kc, vc, lens), state):
            t.copy_(was)
    for _ in range(3):
        for n in ("q", "kb", "vb"):
            x[n].copy_(rnd(*x[n].shape).bfloat16())
        for n in ("ua", "us"):
            x[n].copy_(torch.rand(x[n].shape, generator=g, device="cuda"))
        before = [t.cpu().clone() for t in (kc, vc, lens)]
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        for layer in range(L):
            o, lse, q = out["att"][layer]
            ro, rl, to, tl = tree_ref(q.cpu(), out["kb"][layer].cpu(), x["vb"][layer].cpu(), ptr, mask.cpu(),
                                      before[0][layer], before[1][layer], table.cpu(), before[2], d ** -0.5)
            assert_within("o", o, ro, to, torch.bfloat16)
            assert_within("lse", lse, rl, tl, torch.float32)
        a = dict(target=x["p"].cpu(), draft=x["qd"].cpu(), tokens=x["tok"].cpu(), parents=par.cpu(), node_ptr=nptr.cpu(),
                 u_accept=x["ua"].cpu(), u_sample=x["us"].cpu())
        _same(out["v"], a, T)
        ref = _commit_ref(dict(k=before[0], v=before[1], lens=before[2], ptr=nptr.cpu(), path=out["v"][0].cpu(),
                               count=out["v"][1].cpu(), table=table.cpu(), kb=out["kb"].cpu(), vb=x["vb"].cpu()), page)
        assert torch.equal(kc.cpu(), ref[0]) and torch.equal(vc.cpu(), ref[1])
        assert torch.equal(lens.cpu(), before[2] + out["v"][1].cpu())
    tree.check()
