"""Speculative decoding with draft trees over a paged cache: what a trained drafter is for.

One step of B sequences, for a target of L layers (all tensors on one GPU; nothing but check() synchronises):

    tree = SplitKVTreeAttention(num_q_heads, num_kv_heads, head_dim, max_nodes)
    # per layer: nodes packed by sequence, rows node_ptr[b] .. node_ptr[b + 1]
    q, kb = rotary.forward(positions, q, kb)
    o, lse = tree.forward(q, kb, vb, node_ptr, mask, k_cache, v_cache, page_table, context_lens, scale)
    # once, from the target's and the drafter's distributions
    path, count, next_token = verify_draft(target_probs, draft_probs, tokens, parents, node_ptr,
                                           u_accept, u_sample, max_nodes=max_nodes, status=tree.status)
    commit_draft(k_caches, v_caches, page_table, context_lens, kbs, vbs, node_ptr, path, count,
                 status=tree.status)                                                              # all layers
    context_lens += count
    tree.check()       # now and then: raises if any of these calls met a bad device array (synchronises)

The kernels cannot raise: what they find wrong in device arrays (a page, a length, a node range, a parent, a token, a path
row) they leave out, and say so in the status words that the call was given.  Without a status nothing says it, and rows
that a commit left out would be counted as context: give all calls of a step the same words.

Node 0 of a sequence is its last certain token (not yet in the cache), the others are drafted; parents hold
each node's local parent (-1 for node 0), smaller than the node itself.  A drafter's own block of queries that
all see each other is the same call with mask=None, and one node a sequence is ordinary decoding.
"""

from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import SplitKVError, _with_site
from .draft_calls import splitkv_tree_attn, splitkv_tree_commit, splitkv_tree_verify


def new_status(device=None) -> torch.Tensor:
    """Cleared status words: the kernels record an error about the device arrays they were given in them."""
    return torch.zeros(2, dtype=torch.int32, device="cuda" if device is None else device)


def check_status(status: torch.Tensor) -> None:
    """Raise SplitKVError if a call that was given `status` recorded an error; clears it.  Synchronises."""
    code, site = status.tolist()
    if code:
        status.zero_()
        raise _with_site(SplitKVError("draft tree call", code), site)


def tree_mask(parents, node_ptr, max_nodes: int) -> np.ndarray:
    """bool [nodes, max_nodes]: each node sees itself and its ancestors (host arrays; upload the result)."""
    parents, ptr = np.asarray(parents), np.asarray(node_ptr)
    mask = np.zeros((int(ptr[-1]), max_nodes), dtype=bool)
    for b in range(ptr.size - 1):
        n0, n = int(ptr[b]), int(ptr[b + 1] - ptr[b])
        if n > max_nodes:
            raise ValueError(f"sequence {b} has {n} nodes; max_nodes is {max_nodes}")
        for i in range(n):
            par = int(parents[n0 + i])
            if par >= i:
                raise ValueError(f"sequence {b}: the parent of node {i} must be an earlier node")
            if par >= 0:
                mask[n0 + i] = mask[n0 + par]
            mask[n0 + i, i] = True
    return mask


class SplitKVTreeAttention:
    """Attention of draft-tree nodes over their sequences' paged context and their own trees.

    The lengths stay on the device, so the kernel and its row tiles are chosen by bounds that the host knows: max_nodes and
    the width of the page table.  Keep both tight.  A step of one node a sequence takes 12 us over 1k keys through an object
    for 1 to 4 nodes and 21 us through one for 64 (64 sequences: 74 and 106 us); an object holds two words, so make one for
    each kind of step, and pass page_table[:, :w] where w pages are enough for every sequence of the call."""

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, max_nodes: int, device=None):
        if num_kv_heads < 1 or num_q_heads % num_kv_heads:
            raise ValueError("num_q_heads must be a multiple of num_kv_heads")
        self.num_q_heads = int(num_q_heads)
        self.num_kv_heads = int(num_kv_heads)
        self.head_dim = int(head_dim)
        self.max_nodes = int(max_nodes)
        self.status = new_status(device)

    def forward(self, q, kb, vb, node_ptr, mask, k_cache, v_cache, page_table, context_lens, scale: float,
                out_dtype: Optional[torch.dtype] = None, o=None, lse=None):
        """q [nodes, Hq, d], kb, vb [nodes, Hkv, d]; node_ptr int32 [B + 1]; mask bool [nodes, >= max_nodes] or
        None (a node sees every node of its sequence); k_cache, v_cache [pages, page_size, Hkv, d] (page_size a
        power of two); page_table int32 [B, pages]; context_lens int32 [B].  bfloat16 or float16; the last
        dimension contiguous, other strides in multiples of 8 elements.  Returns o [nodes, Hq, d] (out_dtype: q's
        type, or float32) and lse [nodes, Hq]; rows behind the last sequence's nodes are left as they were."""
        shape = q.shape
        if len(shape) != 3 or shape[1] != self.num_q_heads or shape[2] != self.head_dim:
            raise ValueError(f"q must be [nodes, {self.num_q_heads}, {self.head_dim}]")
        if k_cache.dim() != 4 or k_cache.shape[2] != self.num_kv_heads:
            raise ValueError(f"k_cache must be [pages, page_size, {self.num_kv_heads}, {self.head_dim}]")
        return splitkv_tree_attn(q, kb, vb, node_ptr, mask, k_cache, v_cache, page_table, context_lens, scale,
                                 self.max_nodes, out_dtype, o, lse, self.status)

    def check(self) -> None:
        """Raise if a call that was given this object's status words recorded an error about its device arrays (a bad
        page, length or node range; in verify_draft and commit_draft also a bad parent, token or path row)."""
        check_status(self.status)


def verify_draft(target_probs, draft_probs, tokens, parents, node_ptr, u_accept, u_sample, max_nodes: int,
                 max_path: Optional[int] = None, status=None):
    """Verification of drafted tokens: the accepted nodes of each sequence and its next token.

    target_probs [nodes, vocab] the target's distribution after each node, draft_probs alike what the node's
    children were drawn from (None: children proposed with certainty, such as a drafter's best candidates);
    float32, bfloat16 or float16.  tokens [nodes] (int32 or int64), parents int32 [nodes], node_ptr int32 [B + 1],
    u_accept float32 [nodes] and u_sample float32 [B] uniform in [0, 1).
    status: words of new_status(), or a SplitKVTreeAttention's, in which bad nodes are recorded (they are never reached).
    Returns path int32 [B, max_path] (local nodes from node 0 on, -1 behind them; max_path defaults to max_nodes,
    and the walk ends there), count int32 [B], next_token [B] (as tokens; -1 where there is none)."""
    return splitkv_tree_verify(target_probs, draft_probs, tokens, parents, node_ptr, u_accept, u_sample, max_nodes,
                               max_nodes if max_path is None else max_path, status)


def commit_draft(k_cache, v_cache, page_table, context_lens, kb, vb, node_ptr, path=None, count=None,
                 max_nodes: Optional[int] = None, status=None) -> None:
    """Append the accepted nodes' keys and values to the cache, behind each sequence's context.

    Caches [pages, page_size, heads, d] with kb, vb [nodes, heads, d], or all layers at once with one more leading
    dimension on the four.  path, count: as verify_draft returns them; without a path every node is appended in
    order (max_nodes then bounds a sequence's nodes).  status: words of new_status(), or a SplitKVTreeAttention's, in
    which rows that had to be left out are recorded.  context_lens is not advanced: add count once all layers are
    written.  Sequences must not share the pages they write, and kb, vb must lie apart from the caches (nodes that are in
    the cache already are copied out first)."""
    if path is None:
        if max_nodes is None:
            raise ValueError("max_nodes bounds the nodes of a sequence where no path is given")
    elif count is None:
        raise ValueError("path needs count")
    else:
        max_nodes = path.shape[1]
    splitkv_tree_commit(k_cache, v_cache, page_table, context_lens, kb, vb, node_ptr, path, count, max_nodes, status)
