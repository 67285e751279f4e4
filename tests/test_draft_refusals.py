"""Refusals of the rotary and draft-tree calls that go by where their arrays lie (host only: nothing is launched)."""

import ctypes

import pytest

BAD, UNSUP = -1, -2
M = 1 << 20


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def _rope(abi, **kw):
    """10 tokens, 4 + 2 heads of 64 in 16 bits: q 5120 bytes, k 2560."""
    a = abi.RopeArgs(10, 4, 2, 64, 64, abi.DTYPE_BF16, 0, 1.0, 4096, 8192, M, 2 * M, 3 * M, 4 * M,
                     (256, 64), (256, 64), (128, 64), (128, 64))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(q_out=3 * M),                                   # q' over k
    dict(q_out=3 * M - 4096),                            # its last tokens over k's first
    dict(k_out=M),                                       # k' over q
    dict(k_out=M + 5120 - 16),                           # over q's last elements
    dict(k_out=2 * M),                                   # k' over q'
    dict(k_out=2 * M + 2560),
    dict(q_out=M, k=M, k_out=M),                         # one array in place as both
    dict(q_out=M, k=M),                                  # q in place, and k reads it
    dict(q_out=3 * M, k_out=M),                          # swapped
    # q in place in a fused buffer of 6 heads a token, k' at its last head: one head of k' would be the next token's
    dict(q_out=M, q_stride=i64(384, 64), q_out_stride=i64(384, 64), k_out=M + 640, k_out_stride=i64(384, 64)),
])
def test_rotary_outputs_over_the_other_side(splitkv, kw):
    assert splitkv._lib.splitkv_rope(ctypes.byref(_rope(splitkv._abi, **kw)), None) == BAD


HARNESS = r"""
#include <cstdio>
#include <vector>
#include "strided.h"
using splitkv::Strided;
int main() {
  Strided a[2];
  long long p;
  while (std::scanf("%lld", &p) == 1) {
    for (int k = 0; k < 2; ++k) {
      if (k) std::scanf("%lld", &p);
      long long row, n, s, t;
      std::scanf("%lld %lld", &row, &n);
      a[k] = {reinterpret_cast<const void*>(p), row, int(n), {}, {}};
      for (int i = 0; i < n; ++i) {
        std::scanf("%lld %lld", &s, &t);
        a[k].size[i] = s;
        a[k].stride[i] = t;
      }
    }
    std::printf("%d %d\n", int(splitkv::apart(a[0], a[1])), int(splitkv::apart(a[1], a[0])));
  }
}
"""


def _bytes(ptr, row, dims):
    at = {ptr}
    for n, s in dims:
        at = {a + i * s for a in at for i in range(n)}
    return {a + i for a in at for i in range(row)}


def test_apart_arrays(splitkv, tmp_path):
    """apart() against the bytes themselves: never true for arrays that meet, true for extents that do not and for the
    woven views that callers have."""
    import os
    import random
    import subprocess
    from conftest import ROOT
    src, exe = tmp_path / "apart.cpp", tmp_path / "apart"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "context_block_sparse_b200", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    rng = random.Random(1)
    woven = [((0, 8, [(5, 48), (2, 8)]), (16, 8, [(5, 48), (4, 8)])),        # heads of a fused projection
             ((0, 8, [(5, 48), (2, 24)]), (8, 8, [(5, 48), (2, 24)])),       # q and k of one head side by side
             ((0, 8, [(2, 240), (5, 48)]), (24, 8, [(7, 48)])),
             ((0, 4, [(3, 64), (4, 8)]), (32, 4, [(3, 64), (4, 8)])),        # keys beside values in a page
             ((0, 4, [(2, 192), (3, 64), (4, 8)]), (32, 4, [(3, 64), (2, 192), (4, 8)])),
             ((0, 4, [(1, 7), (4, 8)]), (4, 4, [(4, 8)]))]
    cases = list(woven)
    for _ in range(4000):
        mk = lambda: (rng.randrange(60), rng.randint(1, 6), [(rng.randint(1, 4), rng.choice([0, 4, 6, 8, 12, 24, 30, 48]))
                                                             for _ in range(rng.randint(0, 4))])  # noqa: E731
        cases.append((mk(), mk()))
    text = "\n".join(" ".join(f"{4096 + p} {row} {len(dims)} " + " ".join(f"{n} {s}" for n, s in dims)
                              for p, row, dims in pair) for pair in cases)
    out = subprocess.run([str(exe)], input=text + "\n", capture_output=True, text=True, check=True).stdout.split()
    said = list(zip(out[::2], out[1::2]))
    assert len(said) == len(cases)
    for i, (pair, (xy, yx)) in enumerate(zip(cases, said)):
        x, y = (_bytes(*p) for p in pair)
        assert xy == yx
        if xy == "1":
            assert not x & y, pair
        if i < len(woven) or max(x) < min(y) or max(y) < min(x):
            assert xy == "1", pair
    assert sum(xy == "1" for xy, _ in said) > 500


def _commit(abi, **kw):
    """2 layers, 10 pages of 16 tokens, 2 heads of 64 in 16 bits (81920 bytes a cache); 8 new nodes (4096 bytes)."""
    a = abi.CommitArgs(2, 2, 8, 4, 2, 64, 2, 16, 10, 5, M, 2 * M, 3 * M, 4 * M, 4096, 4096, 4096, 4096, 4096, None,
                       (1024, 128, 64), (1024, 128, 64), (20480, 2048, 128, 64), (20480, 2048, 128, 64), 4, 5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(kb=3 * M),                                                 # new keys that view the first page
    dict(kb=3 * M + 40960, kb_stride=i64(20480, 128, 64)),          # a page of every layer
    dict(vb=3 * M + 81920 - 16),                                    # new values over the cache of keys
    dict(kb=4 * M - 2048),
    dict(kb=4 * M + 4096, vb=4 * M),
    dict(v_cache=3 * M), dict(v_cache=3 * M + 128),                 # one cache for both
    dict(num_pages=2 ** 31 - 1, k_stride=i64(20480, 1 << 44, 128, 64), kb=5 * M),   # an extent past 64 bits
])
def test_commit_from_inside_a_cache(splitkv, kw):
    assert splitkv._lib.splitkv_tree_commit(ctypes.byref(_commit(splitkv._abi, **kw)), None) == BAD


@pytest.mark.parametrize("kw,code", [
    (dict(num_kv_heads=65536, head_dim=65536, elem_bytes=4), UNSUP),    # a token of 2^30 vectors: 32 rows pass 2^31
    (dict(num_kv_heads=4096, head_dim=65536, elem_bytes=4), UNSUP),     # 2^26 of them: just past
])
def test_commit_of_tokens_past_the_index_range(splitkv, kw, code):
    z4, z3 = i64(0, 0, 0, 0), i64(0, 0, 0)
    a = _commit(splitkv._abi, kb=1 << 50, vb=1 << 51, k_cache=1 << 52, v_cache=1 << 53, kb_stride=z3, vb_stride=z3,
                k_stride=z4, v_stride=z4, **kw)
    assert splitkv._lib.splitkv_tree_commit(ctypes.byref(a), None) == code


def _verify(abi, **kw):
    a = abi.VerifyArgs(2, 8, 4, 100, abi.DTYPE_F32, 0, 4, 0, *(i * M for i in range(1, 11)), None, 100, 100, 4)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _tree(abi, **kw):
    a = abi.TreeArgs(2, 8, 4, 8, 2, 128, abi.DTYPE_BF16, abi.DTYPE_BF16, 16, 10, 5, 1.0, *(i * M for i in range(1, 6)),
                     6 * M, 7 * M, 8 * M, 9 * M, 10 * M, 11 * M, None, (1024, 128), (256, 128), (256, 128),
                     (4096, 256, 128), (4096, 256, 128), 4, 5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("call,make,kw", [
    *(("splitkv_tree_commit", _commit, kw) for kw in (
        dict(node_ptr=4098), dict(context_lens=4097), dict(page_table=4098), dict(path=4098), dict(count=4098),
        dict(status=4098), dict(table_stride=-5), dict(path_stride=-4))),
    *(("splitkv_tree_verify", _verify, kw) for kw in (
        dict(tokens=4098), dict(tokens=4100, token_int64=1), dict(parents=4098), dict(node_ptr=4097),
        dict(u_accept=4098), dict(u_sample=4098), dict(path=4098), dict(count=4098), dict(next=4098),
        dict(next=4100, token_int64=1), dict(status=4098))),
    *(("splitkv_tree_attn", _tree, kw) for kw in (dict(node_ptr=4098), dict(context_lens=4097), dict(status=4098))),
])
def test_misaligned_words_and_negative_strides(splitkv, call, make, kw):
    """A word off its boundary would fault the GPU, and a stride below zero leave the array."""
    a = ctypes.byref(make(splitkv._abi, **kw))
    args = (a, 64 * M, 1 << 40, None) if call == "splitkv_tree_attn" else (a, None)
    assert getattr(splitkv._lib, call)(*args) == BAD


@pytest.mark.parametrize("call,make,kw", [
    *(("splitkv_tree_attn", _tree, kw) for kw in (dict(num_seqs=0), dict(num_nodes=0), dict(num_nodes=0, q=None, o=None))),
    *(("splitkv_tree_verify", _verify, kw) for kw in (dict(num_seqs=0), dict(num_seqs=0, num_nodes=0, target=None))),
    *(("splitkv_tree_commit", _commit, kw) for kw in (dict(num_seqs=0), dict(num_layers=0), dict(num_nodes=0, kb=None),
                                                     dict(max_rows=0))),
    *(("splitkv_rope", _rope, kw) for kw in (dict(num_tokens=0), dict(q_heads=0, k_heads=0, q=None, k=None))),
])
def test_calls_without_work_succeed(splitkv, call, make, kw):
    """Before anything else is asked for: no workspace, no arrays."""
    a = ctypes.byref(make(splitkv._abi, **kw))
    args = (a, None, 0, None) if call == "splitkv_tree_attn" else (a, None)
    assert getattr(splitkv._lib, call)(*args) == 0


@pytest.mark.parametrize("kw", [
    dict(o=2 * M), dict(o=3 * M), dict(o=4 * M), dict(o=5 * M + 4096), dict(o=2 * M - 16),    # over kb, vb, the caches
    dict(o=M + 256), dict(o=M, o_dtype=0),                            # over q otherwise than in place
    dict(o=M, q_stride=(ctypes.c_int64 * 2)(2048, 128)),
    dict(lse=M), dict(lse=4 * M), dict(lse=10 * M + 64), dict(o=64 * M), dict(lse=64 * M), dict(q=64 * M), dict(k_cache=64 * M),
])
def test_tree_attention_outputs_over_its_inputs(splitkv, kw):
    """Other CTAs still read what an output or the workspace overwrites (o in the place of q itself is taken)."""
    a = ctypes.byref(_tree(splitkv._abi, **kw))
    assert splitkv._lib.splitkv_tree_attn(a, 64 * M, 1 << 40, None) == BAD
