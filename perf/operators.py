"""The speculative-decoding operators as measured work: rotary positions, attention of a draft
tree over a paged cache, verification of drafted tokens, and the commit of the accepted nodes'
keys and values to the cache.

Each case is one call a serving (or, for the rotary backward, a training) step makes.  `run`
computes it in plain torch operations, or, where `own` is true, through this package.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of four sequences with 16 drafted nodes each, far into a long context
        dict(name="rope_step", op="rope", tokens=64, hq=32, hkv=8, d=128, rd=128, interleaved=False,
             scaling="parts", factor=8.0, dtype="bf16", backward=False, far=131072),
        # the queries and keys of a whole 64k-token packed context
        dict(name="rope_context", op="rope", tokens=65536, hq=32, hkv=8, d=128, rd=128, interleaved=False,
             scaling="none", factor=1.0, dtype="bf16", backward=False, far=16384),
        # float32 gradients of 8192 draft queries and their block keys; a quarter-odd number of tokens
        dict(name="rope_grad", op="rope", tokens=8191, hq=32, hkv=8, d=128, rd=64, interleaved=True,
             scaling="linear", factor=4.0, dtype="fp32", backward=True, far=65536),
        # a single token of a single sequence: no draft at all, latency only
        dict(name="tree_token", op="tree", seqs=1, nodes=1, fixed=True, lo=1001, hi=1001, hq=32, hkv=8, d=128,
             page=16, dtype="bf16", kind="chain"),
        # an ordinary batch: 16 sequences, up to 16 nodes each, 1k to 8k of context
        dict(name="tree_batch", op="tree", seqs=16, nodes=16, fixed=False, lo=1024, hi=8192, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", kind="tree"),
        # few long sequences with wide trees: 64 nodes over 64k to 128k of context
        dict(name="tree_long", op="tree", seqs=4, nodes=64, fixed=True, lo=65536, hi=131072, hq=32, hkv=8, d=128,
             page=128, dtype="bf16", kind="tree"),
        # a drafter's own block of 8 bidirectional queries: small heads, many short sequences, ragged
        dict(name="tree_block_d64", op="tree", seqs=130, nodes=8, fixed=True, lo=0, hi=3001, hq=16, hkv=2, d=64,
             page=32, dtype="fp16", kind="block"),
        # one sequence, 15 drafted tokens in a row
        dict(name="verify_one", op="verify", seqs=1, nodes=16, vocab=32000, kind="chain", dtype="fp32", probs=True),
        # 64 sequences of 15 drafted tokens, a large vocabulary
        dict(name="verify_batch", op="verify", seqs=64, nodes=16, vocab=131072, kind="chain", dtype="fp32", probs=True),
        # trees with several candidates a level: rejected siblings change the target's distribution
        dict(name="verify_tree", op="verify", seqs=24, nodes=40, vocab=50001, kind="tree", dtype="fp32", probs=True),
        # accepted nodes of one sequence into a single layer's cache
        dict(name="commit_one", op="commit", layers=1, seqs=1, nodes=16, depth=6, hkv=8, d=128, page=16, dtype="bf16"),
        # accepted nodes of 48 sequences into the caches of 24 layers at once
        dict(name="commit_layers", op="commit", layers=24, seqs=48, nodes=32, depth=8, hkv=8, d=128, page=32,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "tree", "verify", "verify", "commit"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 40000), hq=hkv * group, hkv=hkv, d=d,
                    rd=rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "parts"]),
                    factor=rng.choice([1.0, 2.0, 4.0, 16.0]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    backward=rng.random() < 0.4, far=_log(rng, 64, 1 << 20))
    if op == "tree":
        seqs = _log(rng, 1, 128)
        hi = _log(rng, 64, max(128, min(131072, 400000 // seqs)))
        lo = rng.choice([0, hi, hi // 3])
        cap = max(1, min(192, 700000000 // (seqs * hkv * group * hi)))
        return dict(op=op, seqs=seqs, nodes=_log(rng, 1, cap), fixed=rng.random() < 0.3, lo=lo, hi=hi,
                    hq=hkv * group, hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128, 256]),
                    dtype=rng.choice(["bf16", "fp16"]), kind=rng.choice(["chain", "tree", "block"]))
    if op == "verify":
        seqs, nodes = _log(rng, 1, 64), _log(rng, 1, 48)
        return dict(op=op, seqs=seqs, nodes=nodes, vocab=_log(rng, 100, min(200000, 64 * 16 * 131072 // (seqs * nodes))),
                    kind=rng.choice(["chain", "tree"]), dtype=rng.choice(["fp32", "fp32", "bf16"]),
                    probs=rng.random() < 0.7)
    nodes = _log(rng, 1, 64)
    return dict(op=op, layers=_log(rng, 1, 16), seqs=_log(rng, 1, 64), nodes=nodes, depth=rng.randint(1, min(nodes, 12)),
                hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]))


# ---------------------------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _counts(case):
    """Nodes of each sequence: all of them `nodes`, or ragged from half of that up (the same for every seed: the
    outputs' shape goes by their sum)."""
    n = case["nodes"]
    if case.get("fixed", case["op"] != "tree"):
        return np.full(case["seqs"], n, dtype=np.int64)
    return np.random.default_rng(n).integers(max(1, n // 2), n + 1, size=case["seqs"])


def _parents(kind, counts, host):
    """Local parent of each node, parents first; node 0 of a sequence is its root (-1)."""
    out = []
    for n in counts:
        p = np.arange(-1, n - 1)
        if kind == "tree":        # up to three candidates below a node, in breadth-first order
            p = np.maximum.accumulate(np.concatenate([[-1], np.sort(host.integers(0, 1 + np.arange(n - 1) // 2 + 1))]))
            p = np.minimum(p, np.arange(-1, n - 1))
        out.append(p)
    return np.concatenate(out).astype(np.int32)


def _tree_mask(kind, parents, counts, width):
    """mask[i, j]: node i sees node j of its own sequence (itself and its ancestors; a block sees all)."""
    mask = np.zeros((len(parents), width), dtype=bool)
    at = 0
    for n in counts:
        if kind == "block":
            mask[at:at + n, :n] = True
        else:
            for i in range(n):
                if parents[at + i] >= 0:
                    mask[at + i] = mask[at + parents[at + i]]
                mask[at + i, i] = True
        at += n
    return mask


def _pages(host, seqs, per_seq):
    """A cache's page table: every sequence's pages scattered over the whole cache."""
    return host.permutation(seqs * per_seq).astype(np.int32).reshape(seqs, per_seq)


def prepare(case, seed):
    g, host = _gen(seed), np.random.default_rng(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    s = {"case": case, "handle": None}
    if op == "rope":
        n = case["tokens"]
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["q"] = torch.randn(n, case["hq"], case["d"], generator=g, device="cuda", dtype=dt)
        s["k"] = torch.randn(n, case["hkv"], case["d"], generator=g, device="cuda", dtype=dt)
        return s
    counts = _counts(case)
    ptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total, width = int(ptr[-1]), int(case["nodes"])
    s["node_ptr"] = dev(ptr)
    if op == "commit":
        per_seq = -(-(4 * case["page"] + 64) // case["page"])
        shape = (case["layers"], case["seqs"] * per_seq, case["page"], case["hkv"], case["d"])
        s["lens"] = dev(host.integers(0, per_seq * case["page"] - case["nodes"], size=case["seqs"]).astype(np.int32))
        accepted = host.integers(1, case["depth"] + 1, size=case["seqs"]).astype(np.int32)
        path = np.full((case["seqs"], case["depth"]), -1, dtype=np.int32)
        for b in range(case["seqs"]):
            path[b, :accepted[b]] = np.sort(host.permutation(case["nodes"])[:accepted[b]])
        s["path"], s["accepted"] = dev(path), dev(accepted)
        s["page_table"] = dev(_pages(host, case["seqs"], per_seq))
        s["k_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        s["v_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        s["kb"] = torch.randn(case["layers"], total, case["hkv"], case["d"], generator=g, device="cuda", dtype=dt)
        s["vb"] = torch.randn(case["layers"], total, case["hkv"], case["d"], generator=g, device="cuda", dtype=dt)
        return s
    parents = _parents(case["kind"], counts, host)
    if op == "tree":
        lens = host.integers(case["lo"], case["hi"] + 1, size=case["seqs"]).astype(np.int32)
        per_seq = max(1, -(-int(case["hi"]) // case["page"]))
        shape = (case["seqs"] * per_seq, case["page"], case["hkv"], case["d"])
        s["lens"], s["page_table"] = dev(lens), dev(_pages(host, case["seqs"], per_seq))
        s["mask"] = dev(_tree_mask(case["kind"], parents, counts, width))
        s["q"] = torch.randn(total, case["hq"], case["d"], generator=g, device="cuda", dtype=dt)
        s["kb"] = torch.randn(total, case["hkv"], case["d"], generator=g, device="cuda", dtype=dt)
        s["vb"] = torch.randn(total, case["hkv"], case["d"], generator=g, device="cuda", dtype=dt)
        s["k_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        s["v_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        return s
    # verification: the target's distributions, the drafter's (near them), tokens drawn from the drafter's
    parent_row = dev((parents + np.repeat(ptr[:-1], counts)).clip(0)).long()
    logits = torch.randn(total, case["vocab"], generator=g, device="cuda") * 2.0
    target = torch.softmax(logits, -1).to(dt)
    draft = torch.softmax(logits + 0.5 * torch.randn(total, case["vocab"], generator=g, device="cuda"), -1).to(dt)
    picks = torch.empty(total, dtype=torch.int64, device="cuda")
    for at in range(0, total, 256):
        noise = torch.empty(min(256, total - at), case["vocab"], device="cuda").exponential_(generator=g)
        picks[at:at + 256] = (draft[parent_row[at:at + 256]].float() / noise).argmax(-1)
    s["tokens"], s["parents"] = picks.int(), dev(parents)
    s["target"], s["draft"] = target, draft if case["probs"] else None
    s["u_accept"] = torch.rand(total, generator=g, device="cuda")
    s["u_sample"] = torch.rand(case["seqs"], generator=g, device="cuda")
    return s


# ---------------------------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    case = s["case"]
    if case["op"] == "rope":
        from context_block_sparse_b200.rotary import Rotary
        if s["handle"] is None:
            s["handle"] = Rotary(case["d"], rotary_dim=case["rd"], base=10000.0, interleaved=case["interleaved"],
                                 scaling=case["scaling"], factor=case["factor"], original_len=4096)
        turn = s["handle"].backward if case["backward"] else s["handle"].forward
        return turn(s["positions"], s["q"], s["k"])
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention, commit_draft, verify_draft
    if case["op"] == "tree":
        if s["handle"] is None:
            s["handle"] = SplitKVTreeAttention(case["hq"], case["hkv"], case["d"], case["nodes"])
        return s["handle"].forward(s["q"], s["kb"], s["vb"], s["node_ptr"], s["mask"], s["k_cache"], s["v_cache"],
                                   s["page_table"], s["lens"], case["d"] ** -0.5)
    if case["op"] == "verify":
        return verify_draft(s["target"], s["draft"], s["tokens"], s["parents"], s["node_ptr"], s["u_accept"],
                            s["u_sample"], max_nodes=case["nodes"])
    commit_draft(s["k_cache"], s["v_cache"], s["page_table"], s["lens"], s["kb"], s["vb"], s["node_ptr"],
                 s["path"], s["accepted"])
    return s["k_cache"], s["v_cache"]


# -------------------------------------------------------------------------- rotary, plain form
def _freqs(case):
    """Radians per position of each pair, and the factor on the rotated vector."""
    rd, f = case["rd"], case["factor"]
    i = torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd
    base, scale = 10000.0, 1.0
    if case["scaling"] == "base" and rd > 2:
        base *= f ** (rd / (rd - 2))
    w = base ** -i
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "parts":   # keep pairs that turn over 32 times in 4096 positions, stretch those below one
        keep = ((4096 * w / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        w = w / f * (1 - keep) + w * keep
        scale = 0.1 * math.log(f) + 1.0
    return w, scale


def _plain_rope(s):
    case = s["case"]
    rd, h = case["rd"], case["rd"] // 2
    w, scale = _freqs(case)
    angle = s["positions"].double()[:, None, None] * w      # far positions: the angle needs 64 bits
    c, sn = (torch.cos(angle) * scale).float(), (torch.sin(angle) * scale).float()
    if case["backward"]:
        sn = -sn

    def turn(x):
        y = x.float()
        if case["interleaved"]:
            a, b = y[..., 0:rd:2], y[..., 1:rd:2]
            r = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
        else:
            a, b = y[..., :h], y[..., h:rd]
            r = torch.cat([a * c - b * sn, b * c + a * sn], -1)
        return torch.cat([r, y[..., rd:]], -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


# ------------------------------------------------------------------------ attention, plain form
def _plain_tree(s):
    case = s["case"]
    B, T, hkv, d, page = case["seqs"], case["nodes"], case["hkv"], case["d"], case["page"]
    G, L = case["hq"] // hkv, max(1, case["hi"])
    total = s["q"].shape[0]
    ptr, lens = s["node_ptr"].long(), s["lens"].long()
    t = torch.arange(T, device="cuda")
    there = t < (ptr[1:] - ptr[:-1])[:, None]                              # [B, T]
    row = torch.clamp(ptr[:-1, None] + t, max=total - 1)
    q = s["q"][row].float().view(B, T, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * T, d)
    at = torch.arange(L, device="cuda")
    keys = s["page_table"].long()[:, at // page], at % page
    k, v = s["k_cache"][keys].float(), s["v_cache"][keys].float()          # [B, L, hkv, d]
    low = float("-inf")
    ctx = (q @ k.permute(0, 2, 3, 1)).mul_(d ** -0.5).masked_fill_((at >= lens[:, None])[:, None, None], low)
    kb, vb = s["kb"][row].float(), s["vb"][row].float()                    # [B, T, hkv, d]
    see = s["mask"][row] & there[:, None] & there[:, :, None]              # [B, T, T]
    see = see[:, None, None].expand(B, 1, G, T, T).reshape(B, 1, G * T, T)
    tree = (q @ kb.permute(0, 2, 3, 1) * d ** -0.5).masked_fill(~see, low)
    m = torch.maximum(ctx.amax(-1, True), tree.amax(-1, True))
    ref = m.masked_fill(m == low, 0.0)                                     # a row that sees nothing
    ctx, tree = ctx.sub_(ref).exp_(), (tree - ref).exp()
    l = ctx.sum(-1, True) + tree.sum(-1, True)
    o = (ctx @ v.transpose(1, 2) + tree @ vb.transpose(1, 2)) / l.masked_fill(l == 0, 1.0)
    lse = m + l.log().masked_fill(m == low, 0.0)
    seq = torch.bucketize(torch.arange(total, device="cuda"), ptr[1:], right=True)
    node = torch.arange(total, device="cuda") - ptr[seq]
    o = o.view(B, hkv, G, T, d)[seq, :, :, node].reshape(total, case["hq"], d)
    lse = lse.view(B, hkv, G, T)[seq, :, :, node].reshape(total, case["hq"])
    return o.to(s["q"].dtype), lse


# --------------------------------------------------------------------- verification, plain form
def _plain_verify(s):
    """Sums and comparisons of probabilities in 64 bits: the outputs are whole numbers decided at borders."""
    case = s["case"]
    B, T, V = case["seqs"], case["nodes"], case["vocab"]
    p_all = s["target"].view(B, T, V)
    q_all = None if s["draft"] is None else s["draft"].view(B, T, V)
    x = s["tokens"].long().view(B, T)
    parent, u = s["parents"].long().view(B, T), s["u_accept"].double().view(B, T)
    b = torch.arange(B, device="cuda")
    path, n, cur, cut = (_walk_chain if case["kind"] == "chain" else _walk_tree)(p_all, q_all, x, parent, u, b)
    p = p_all[b, cur].double()
    left = p.clone()
    if q_all is not None:
        left = (p - cut[0][:, None] * q_all[b, cur].double()).clamp_(min=0)
    else:
        left.masked_fill_(cut[1], 0.0)
    cum = left.cumsum_(-1)
    total = cum[:, -1:]
    empty = total <= 0
    cum = torch.where(empty, p.cumsum_(-1), cum)
    goal = s["u_sample"].double()[:, None] * cum[:, -1:]
    goal = torch.minimum(goal, torch.nextafter(cum[:, -1:], torch.zeros_like(goal)))
    token = (cum <= goal).sum(-1)
    return path.int(), n.int(), token.int()


def _walk_chain(p, q, x, parent, u, b):
    B, T, V = p.shape
    t = torch.arange(T, device="cuda")
    px = p[:, :-1].gather(2, x[:, 1:, None]).squeeze(2).double()
    qx = torch.ones_like(px) if q is None else q[:, :-1].gather(2, x[:, 1:, None]).squeeze(2).double()
    n = 1 + (u[:, 1:] * qx < px).long().cumprod(1).sum(1)
    cur, stopped = n - 1, n < T
    path = torch.where(t < n[:, None], t, -1)
    wrong = x[b, n.clamp(max=T - 1)]
    removed = (torch.arange(V, device="cuda") == wrong[:, None]) & stopped[:, None]
    return path, n, cur, (stopped.double(), removed)


def _walk_tree(p, q, x, parent, u, b):
    """The candidates of a level are tried in order, each against what its rejected elders left of the target's
    distribution: max(p - c q, 0) with c growing by that distribution's mass at each rejection."""
    B, T, V = p.shape
    cur, n = torch.zeros_like(b), torch.ones_like(b)
    path = torch.full((B, T), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    c, mass = torch.zeros(B, dtype=torch.float64, device="cuda"), torch.ones(B, dtype=torch.float64, device="cuda")
    removed = torch.zeros(B, V, dtype=torch.bool, device="cuda")
    for i in range(1, T):
        xi, tried = x[:, i], parent[:, i] == cur
        px = p[b, cur, xi].double()
        if q is None:
            qx = 1.0
            r = torch.where(removed[b, xi], 0.0, px)
        else:
            qx = q[b, cur, xi].double()
            r = (px - c * qx).clamp(min=0)
        taken = tried & (u[:, i] * mass * qx < r)
        missed = tried & ~taken
        if q is None:
            mass = torch.where(missed, (mass - r).clamp(min=0), mass)
            removed = removed & ~taken[:, None]
            removed[b, xi] |= missed
        else:
            c = torch.where(missed, c + mass, torch.where(taken, 0.0, c))
            rest = (p[b, cur].double() - c[:, None] * q[b, cur].double()).clamp_(min=0).sum(-1)
            mass = torch.where(missed, rest, mass)
        mass = torch.where(taken, 1.0, mass)
        path[b, torch.where(taken, n, T - 1)] = torch.where(taken, i, path[:, T - 1])
        n, cur = n + taken, torch.where(taken, i, cur)
    return path, n, cur, (c, removed)


# --------------------------------------------------------------------------- commit, plain form
def _plain_commit(s):
    case = s["case"]
    D, page = case["depth"], case["page"]
    i = torch.arange(D, device="cuda")
    i = torch.where(i < s["accepted"][:, None], i, 0)                      # beyond the path: its first node again
    row = s["node_ptr"][:-1, None].long() + s["path"].gather(1, i).long()
    at = s["lens"][:, None].long() + i
    where = s["page_table"].gather(1, at // page).long(), at % page
    s["k_cache"][:, where[0], where[1]] = s["kb"][:, row]
    s["v_cache"][:, where[0], where[1]] = s["vb"][:, row]
    return s["k_cache"], s["v_cache"]


_PLAIN = {"rope": _plain_rope, "tree": _plain_tree, "verify": _plain_verify, "commit": _plain_commit}


# ------------------------------------------------------------------------------------- the work
def work(case):
    op, e = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "rope":
        rows = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * rows * case["d"] * e + 4 * case["tokens"], "flops": 3 * rows * case["rd"]}
    if op == "commit":
        mean = (1 + case["depth"]) / 2
        return {"bytes": 4 * case["layers"] * case["seqs"] * mean * case["hkv"] * case["d"] * e, "flops": 0}
    if op == "verify":   # the distributions of the node where the walk stops, read once
        rows = 2 if case["probs"] else 1
        return {"bytes": case["seqs"] * (rows * case["vocab"] * e + 24 * case["nodes"]), "flops": 3 * case["seqs"] * case["vocab"]}
    n = int(_counts(case).sum())
    ctx = case["seqs"] * (case["lo"] + case["hi"]) / 2
    per_seq = n / case["seqs"]
    kv = 2 * (ctx + n) * case["hkv"] * case["d"] * e
    qo = n * case["hq"] * (2 * case["d"] * e + 4)
    return {"bytes": kv + qo, "flops": 4 * case["hq"] * case["d"] * per_seq * (ctx + n / 2)}


# ---------------------------------------------------------------------- 64 bits, from the definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "verify": _exact_verify, "commit": _exact_commit}[case["op"]](s)


def _exact_rope(s):
    """Each pair (a, b) as the complex number a + ib, times scale e^(i position w) (its conjugate backward)."""
    case = s["case"]
    rd, f = case["rd"], case["factor"]
    w = []
    for j in range(rd // 2):
        base = 10000.0 * (f ** (rd / (rd - 2.0)) if case["scaling"] == "base" and rd > 2 else 1.0)
        wj = 1.0 / base ** (2.0 * j / rd)
        if case["scaling"] == "linear":
            wj /= f
        if case["scaling"] == "parts":
            keep = min(1.0, max(0.0, (4096 * wj / (2 * math.pi) - 1.0) / 31.0))
            wj = keep * wj + (1 - keep) * wj / f
        w.append(wj)
    scale = 0.1 * math.log(f) + 1.0 if case["scaling"] == "parts" else 1.0
    sign = -1.0 if case["backward"] else 1.0
    turn = torch.polar(torch.full((len(s["positions"]), rd // 2), scale, dtype=torch.float64, device="cuda"),
                       sign * s["positions"].double()[:, None] * torch.tensor(w, dtype=torch.float64, device="cuda"))
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        for h in range(x.shape[1]):
            first = y[:, h, 0:rd:2] if case["interleaved"] else y[:, h, :rd // 2]
            second = y[:, h, 1:rd:2] if case["interleaved"] else y[:, h, rd // 2:rd]
            z = torch.complex(first, second) * turn
            first.copy_(z.real)
            second.copy_(z.imag)
        out.append(y)
    return tuple(out)


def _exact_tree(s):
    """One sequence and one KV head at a time: softmax over the context's keys and the visible nodes."""
    case = s["case"]
    G, page = case["hq"] // case["hkv"], case["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    ptr, lens = s["node_ptr"].tolist(), s["lens"].tolist()
    for b in range(case["seqs"]):
        i0, i1, n = ptr[b], ptr[b + 1], lens[b]
        pages = s["page_table"][b, :-(-n // page)].long()
        kc = s["k_cache"][pages].flatten(0, 1)[:n]
        vc = s["v_cache"][pages].flatten(0, 1)[:n]
        mask = torch.cat([torch.ones(i1 - i0, n, dtype=torch.bool, device="cuda"), s["mask"][i0:i1, :i1 - i0]], 1)
        for h in range(case["hkv"]):
            k = torch.cat([kc[:, h], s["kb"][i0:i1, h]]).double()
            v = torch.cat([vc[:, h], s["vb"][i0:i1, h]]).double()
            for g in range(h * G, h * G + G):
                sc = torch.where(mask, s["q"][i0:i1, g].double() @ k.T / math.sqrt(case["d"]), -math.inf)
                lse[i0:i1, g] = torch.logsumexp(sc, 1)
                o[i0:i1, g] = torch.nan_to_num(torch.softmax(sc, 1)) @ v
    return o, lse


def _exact_verify(s):
    """The walk itself, one sequence at a time on the host: residual distributions are formed and normalised."""
    case = s["case"]
    T = case["nodes"]
    path = np.full((case["seqs"], T), -1, dtype=np.int32)
    count = np.zeros(case["seqs"], dtype=np.int32)
    token = np.zeros(case["seqs"], dtype=np.int32)
    x, parents = s["tokens"].cpu().numpy(), s["parents"].cpu().numpy()
    u, us = s["u_accept"].cpu().numpy().astype(np.float64), s["u_sample"].cpu().numpy().astype(np.float64)
    for b in range(case["seqs"]):
        at, cur, n = b * T, 0, 1
        path[b, 0] = 0
        while True:
            p = s["target"][at + cur].double().cpu().numpy()
            r, moved = p.copy(), False
            q = None if s["draft"] is None else s["draft"][at + cur].double().cpu().numpy()
            mass = 1.0                                                     # rows are taken as normalised
            for i in range(cur + 1, T):
                if parents[at + i] != cur:
                    continue
                xi = x[at + i]
                if u[at + i] * mass * (1.0 if q is None else q[xi]) < r[xi]:
                    cur, moved = i, True
                    path[b, n] = i
                    n += 1
                    break
                if q is None:
                    mass, r[xi] = max(mass - r[xi], 0.0), 0.0
                else:
                    r = np.maximum(r - mass * q, 0.0)
                    mass = r.sum()
            if not moved:
                break
        if r.sum() <= 0:
            r = p
        cum = np.cumsum(r)
        token[b] = min(int(np.searchsorted(cum, us[b] * cum[-1], side="right")), int(np.flatnonzero(r > 0)[-1]))
        count[b] = n
    return path, count, token


def _exact_commit(s):
    case = s["case"]
    k, v = s["k_cache"].double(), s["v_cache"].double()
    ptr, lens, path = s["node_ptr"].tolist(), s["lens"].tolist(), s["path"].tolist()
    table, accepted = s["page_table"].tolist(), s["accepted"].tolist()
    for b in range(case["seqs"]):
        for i in range(accepted[b]):
            page, slot = table[b][(lens[b] + i) // case["page"]], (lens[b] + i) % case["page"]
            k[:, page, slot] = s["kb"][:, ptr[b] + path[b][i]].double()
            v[:, page, slot] = s["vb"][:, ptr[b] + path[b][i]].double()
    return k, v
