"""Host side of the rotary and draft-tree calls (CPU): struct layouts, refusals before any launch, frequency tables,
the mask helper, and the walk's oracle against closed forms."""

import ctypes

import numpy as np
import pytest
import torch

from draft_util import random_parents, verify_ref
from test_abi import _c_layout

BAD, UNSUP = -1, -2


def test_struct_layouts_match_header(splitkv, tmp_path):
    abi = splitkv._abi
    for struct, cls in (("splitkv_rope_args", abi.RopeArgs), ("splitkv_tree_args", abi.TreeArgs),
                        ("splitkv_verify_args", abi.VerifyArgs), ("splitkv_commit_args", abi.CommitArgs)):
        fields = [f for f, _ in cls._fields_]
        size, offs = _c_layout(struct, fields, tmp_path)
        assert ctypes.sizeof(cls) == size, struct
        assert [getattr(cls, f).offset for f in fields] == offs, struct


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
@pytest.mark.parametrize("rd", [2, 6, 64, 128])
def test_frequencies(splitkv, scaling, rd):
    from context_block_sparse_b200.rotary import SCALINGS
    f, scale = splitkv.splitkv_rope_freqs(rd, 5000.0, SCALINGS[scaling], 8.0, 2048, 1.0, 32.0)
    i = np.arange(rd // 2)
    base = 5000.0 * (8.0 ** (rd / (rd - 2)) if scaling == "base" and rd > 2 else 1.0)
    w = base ** (-2.0 * i / rd)
    if scaling == "linear":
        w = w / 8
    if scaling == "parts":
        turns = 2048 * w / (2 * np.pi)
        keep = np.clip((turns - 1) / 31, 0, 1)
        w = keep * w + (1 - keep) * w / 8
    np.testing.assert_allclose(f, w, rtol=1e-14)
    assert scale == pytest.approx(1 + 0.1 * np.log(8.0) if scaling == "parts" else 1.0, rel=1e-15)
    if scaling == "base" and rd > 2:     # the slowest pair stretched by the factor, the fastest kept
        assert f[0] == 1.0 and f[-1] == pytest.approx(5000.0 ** (-(rd - 2) / rd) / 8, rel=1e-12)


def test_frequency_refusals(splitkv):
    for rd, base, kind, factor, length in ((3, 1e4, 0, 1, 0), (0, 1e4, 0, 1, 0), (8, -1, 0, 1, 0), (8, 1e4, 9, 1, 0),
                                           (8, 1e4, 1, 0, 0), (8, 1e4, 3, 2, 0), (8, float("nan"), 0, 1, 0)):
        with pytest.raises(splitkv.SplitKVError):
            splitkv.splitkv_rope_freqs(rd, base, kind, factor, length)
    from context_block_sparse_b200.rotary import Rotary
    for kw in (dict(rotary_dim=63), dict(rotary_dim=130), dict(scaling="other"), dict(rotary_dim=0)):
        with pytest.raises(ValueError):
            Rotary(128, **kw)


def _rope(abi, **kw):
    a = abi.RopeArgs(10, 4, 2, 64, 64, abi.DTYPE_BF16, 0, 1.0, 4096, 8192, 1 << 20, 2 << 20, 3 << 20, 4 << 20,
                     (256, 64), (256, 64), (128, 64), (128, 64))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _pair(x, y):
    return (ctypes.c_int64 * 2)(x, y)


@pytest.mark.parametrize("kw", [dict(rotary_dim=65), dict(rotary_dim=66), dict(rotary_dim=0), dict(num_tokens=-1),
                                dict(dtype=7), dict(flags=64), dict(positions=None), dict(freqs=None), dict(q=None),
                                dict(k_out=None), dict(q_out=(1 << 20) + 128), dict(positions=4097),
                                dict(q_out_stride=_pair(256, 32)), dict(q_out_stride=_pair(0, 64)),
                                dict(q_stride=_pair(-256, 64)), dict(k_out=(3 << 20) + 1)])
def test_rope_refuses(splitkv, kw):
    assert splitkv._lib.splitkv_rope(ctypes.byref(_rope(splitkv._abi, **kw)), None) == BAD
    assert splitkv._lib.splitkv_rope(None, None) == BAD


def test_rope_without_work(splitkv):
    lib, abi = splitkv._lib, splitkv._abi
    assert lib.splitkv_rope(ctypes.byref(_rope(abi, num_tokens=0, q=None)), None) == 0
    assert lib.splitkv_rope(ctypes.byref(_rope(abi, q_heads=0, k_heads=0)), None) == 0


def _tree(abi, **kw):
    a = abi.TreeArgs(2, 8, 4, 8, 2, 128, abi.DTYPE_BF16, abi.DTYPE_BF16, 16, 10, 5, 1.0, 4096, 4096, 4096, 4096, 4096,
                     None, 4096, 4096, 4096, 4096, 4096, None, (1024, 128), (256, 128), (256, 128), (4096, 256, 128),
                     (4096, 256, 128), 0, 5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(num_q_heads=7), BAD), (dict(num_kv_heads=0), BAD), (dict(page_size=0), BAD), (dict(page_size=24), BAD),
    (dict(dtype=0, o_dtype=0), BAD), (dict(o_dtype=2), BAD), (dict(max_nodes=0), BAD), (dict(head_dim=96), UNSUP),
    (dict(max_nodes=257), UNSUP), (dict(num_seqs=-1), BAD), (dict(num_seqs=70000), UNSUP), (dict(q=None), BAD),
    (dict(q=4098), BAD), (dict(lse=None), BAD), (dict(o=None), BAD), (dict(k_cache=None), BAD),
    (dict(page_table=None), BAD), (dict(context_lens=None), BAD), (dict(node_ptr=None), BAD),
    (dict(q_stride=_pair(1020, 128)), BAD), (dict(q_stride=_pair(1024, -128)), BAD),
    (dict(max_pages=0x7fffffff), UNSUP), (dict(page_table=None, num_pages=0), BAD), (dict(page_table=4098), BAD)])
def test_tree_attn_refuses(splitkv, kw, code):
    lib, a = splitkv._lib, _tree(splitkv._abi, **kw)
    assert lib.splitkv_tree_attn(ctypes.byref(a), 4096, 1 << 40, None) == code


def test_tree_attn_workspace(splitkv):
    lib, abi = splitkv._lib, splitkv._abi
    n = ctypes.c_size_t()
    assert lib.splitkv_tree_workspace_size(ctypes.byref(_tree(abi)), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.splitkv_tree_attn(ctypes.byref(_tree(abi)), 4096, n.value - 1, None) == -3
    assert lib.splitkv_tree_attn(ctypes.byref(_tree(abi)), None, n.value, None) == BAD
    assert lib.splitkv_tree_attn(ctypes.byref(_tree(abi)), 4104, n.value, None) == BAD
    assert lib.splitkv_tree_attn(None, 4096, n.value, None) == BAD
    for kw in (dict(num_seqs=0), dict(num_nodes=0)):    # nothing to do
        assert lib.splitkv_tree_attn(ctypes.byref(_tree(abi, **kw)), None, 0, None) in (0, -3)


def _verify(abi, **kw):
    a = abi.VerifyArgs(2, 8, 4, 100, abi.DTYPE_F32, 0, 4, 0, 4096, 4096, 4096, 4096, 4096, 4096, 4096, 4096, 4096, 4096,
                       None, 100, 100, 4)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), BAD), (dict(vocab=(1 << 21) + 1), UNSUP), (dict(max_nodes=1025), UNSUP), (dict(max_nodes=0), BAD),
    (dict(max_path=0), BAD), (dict(dtype=9), BAD), (dict(target=None), BAD), (dict(target=4098), BAD),
    (dict(draft=4097), BAD), (dict(u_sample=None), BAD), (dict(path=None), BAD), (dict(target_stride=-1), BAD),
    (dict(tokens=None), BAD), (dict(num_seqs=-1), BAD), (dict(path_stride=3), BAD), (dict(path_stride=-4), BAD)])
def test_verify_refuses(splitkv, kw, code):
    assert splitkv._lib.splitkv_tree_verify(ctypes.byref(_verify(splitkv._abi, **kw)), None) == code
    assert splitkv._lib.splitkv_tree_verify(ctypes.byref(_verify(splitkv._abi, num_seqs=0)), None) == 0


def _commit(abi, **kw):
    a = abi.CommitArgs(1, 2, 8, 4, 2, 64, 2, 16, 10, 5, 4096, 4096, 4096, 4096, 4096, 4096, 4096, 4096, 4096, None,
                       (1024, 128, 64), (1024, 128, 64), (20480, 2048, 128, 64), (20480, 2048, 128, 64), 4, 5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=12), BAD), (dict(elem_bytes=3), BAD), (dict(head_dim=4), UNSUP), (dict(num_layers=-1), BAD),
    (dict(num_layers=70000), UNSUP), (dict(kb=None), BAD), (dict(k_cache=4097), BAD), (dict(count=None), BAD),
    (dict(node_ptr=None), BAD), (dict(page_table=None), BAD), (dict(kb_stride=(ctypes.c_int64 * 3)(1024, 130, 64)), BAD)])
def test_commit_refuses(splitkv, kw, code):
    assert splitkv._lib.splitkv_tree_commit(ctypes.byref(_commit(splitkv._abi, **kw)), None) == code
    assert splitkv._lib.splitkv_tree_commit(ctypes.byref(_commit(splitkv._abi, max_rows=0)), None) == 0


def test_bindings_refuse_host_tensors_and_wrong_shapes(splitkv):
    from context_block_sparse_b200.draft_tree import SplitKVTreeAttention, commit_draft, tree_mask, verify_draft
    from context_block_sparse_b200.rotary import Rotary
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        Rotary(64).forward(z(3, dtype=torch.int32), z(3, 2, 64))
    with pytest.raises(ValueError, match=r"\[n, heads, 64\]"):
        Rotary(64).forward(z(3, dtype=torch.int32), z(3, 2, 32))
    i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        verify_draft(z(3, 5), None, i(3), i(3), i(2), z(3), z(1), max_nodes=3)
    cache, new = z(4, 16, 2, 64), z(3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        commit_draft(cache, cache, i(1, 4), i(1), new, new, i(2), i(1, 3), i(1))
    with pytest.raises(ValueError, match="max_nodes"):
        commit_draft(cache, cache, i(1, 4), i(1), new, new, i(2))
    with pytest.raises(ValueError, match="count"):
        commit_draft(cache, cache, i(1, 4), i(1), new, new, i(2), i(1, 3))
    with pytest.raises(ValueError, match="multiple"):
        SplitKVTreeAttention(7, 2, 64, 4, device="cpu")
    tree = SplitKVTreeAttention(4, 2, 64, 4, device="cpu")
    with pytest.raises(ValueError, match="q must be"):
        tree.forward(z(3, 2, 64), new, new, i(2), None, cache, cache, i(1, 4), i(1), 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        tree.forward(z(3, 4, 64), new, new, i(2), None, cache, cache, i(1, 4), i(1), 1.0)
    with pytest.raises(ValueError, match="earlier"):
        tree_mask([-1, 1], [0, 2], 4)
    with pytest.raises(ValueError, match="max_nodes"):
        tree_mask([-1, 0], [0, 2], 1)


def test_tree_mask_is_ancestry(splitkv):
    from context_block_sparse_b200.draft_tree import tree_mask
    m = tree_mask([-1, 0, 0, 1, 3, -1, 0], [0, 5, 7], 6)
    want = [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [0], [0, 1]]
    assert m.shape == (7, 6)
    for row, cols in zip(m, want):
        assert list(np.flatnonzero(row)) == cols


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("siblings", [1, 2, 3])
def test_walk_oracle_keeps_the_targets_distribution(siblings, certain):
    """The oracle's first token (an accepted child's, or the next token) is distributed as the target's row: its
    probability, with the acceptance numbers integrated exactly, against p.  Root with k children."""
    rng = np.random.default_rng(siblings)
    V = 4
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    got = np.zeros(V)

    def follow(r, S, k, weight, tried):
        """Adds the law of the first token from residual r (S its mass as tracked) with k children left."""
        if k == 0:
            got[:] += weight * r / r.sum()
            return
        # certain children: fixed distinct tokens; drawn ones: each x with probability q(x)
        options = [(tried, 1.0)] if certain else [(x, q[x]) for x in range(V)]
        for x, w in options:
            a = min(1.0, r[x] / (S * (1.0 if certain else q[x])))
            got[x] += weight * w * a
            if a < 1.0:
                if certain:
                    r2 = r.copy()
                    r2[x] = 0.0
                    follow(r2, S - r[x], k - 1, weight * w * (1 - a), tried + 1)
                else:
                    r2 = np.maximum(r - S * q, 0.0)
                    follow(r2, r2.sum(), k - 1, weight * w * (1 - a), tried)

    follow(p, 1.0, siblings, 1.0, 0)
    np.testing.assert_allclose(got, p, atol=1e-12)
    # and the oracle takes those decisions: acceptance just below and just above the threshold
    tok = np.array([0] + list(range(siblings)))
    par = np.array([-1] + [0] * siblings)
    t, d = np.tile(p, (siblings + 1, 1)), np.tile(q, (siblings + 1, 1))
    edge = p[0] / (1.0 if certain else q[0])
    for u, accepted in ((edge * (1 - 1e-9), True), (edge * (1 + 1e-9), False)):
        if u >= 1:
            continue
        ua = np.array([0.0, u] + [1 - 1e-12] * (siblings - 1))
        path, count, nxt = verify_ref(t, None if certain else d, tok, par, [0, siblings + 1], ua, [0.5], 4)
        assert (path[0, 1] == 1) == accepted


def test_random_parents_come_first():
    rng = np.random.default_rng(0)
    for kind in ("chain", "tree"):
        p = random_parents(rng, 50, kind)
        assert p[0] == -1 and all(0 <= p[i] < i for i in range(1, 50))
