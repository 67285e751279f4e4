"""Bindings of the rotary and draft-tree entry points (include/splitkv.h): argument checks and marshalling only.

Tensors may be strided: the last dimension is contiguous, the others have any stride (in 16-byte steps where the
header says so).  A call runs on its tensors' device and that device's current stream.  The serving calls are short
enough for their host time to count, so arguments are packed into the C structs' bytes directly.
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import SplitKVError, _abi, _lib
from ._abi import DTYPE_F32, ROPE_ADJOINT, ROPE_INTERLEAVED, ROPE_POS64, ROPE_SCALE_NONE

_CODES = {torch.float32: _abi.DTYPE_F32, torch.bfloat16: _abi.DTYPE_BF16, torch.float16: _abi.DTYPE_F16}
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32

_pack_rope = _abi.packer(_abi.RopeArgs)
_pack_tree = _abi.packer(_abi.TreeArgs)
_pack_verify = _abi.packer(_abi.VerifyArgs)
_pack_commit = _abi.packer(_abi.CommitArgs)

try:        # the address alone, without a Stream object around it
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:
    def _raw_stream(dev: int) -> int:
        return torch.cuda.current_stream(dev).cuda_stream


def _code(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    return code


def _device_of(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _refuse(t, name: str, shape, dtype, dev: int):
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the others")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    raise ValueError(f"{name}: its last dimension, or all of it where the call takes no strides, must be contiguous")


def _strided(t, name: str, shape, dtype, dev: int):
    """Address and strides of a tensor of that shape, type and device."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
        st = t.stride()
        if st[-1] == 1 or shape[-1] <= 1:
            return t.data_ptr(), st
    _refuse(t, name, shape, dtype, dev)


def _dense(t, name: str, shape, dtype, dev: int) -> int:
    """Address of a contiguous tensor of that shape, type and device."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, shape, dtype, dev)


def _status(status, dev: int) -> int:
    return 0 if status is None else _dense(status, "status", (2,), _I32, dev)


def _call(fn, name: str, dev: int, *args) -> None:
    """fn(*args, device dev's current stream) with dev as the current device."""
    if torch.cuda.current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        raise SplitKVError(name, status)


def splitkv_rope_freqs(rotary_dim: int, base: float = 10000.0, scaling: int = ROPE_SCALE_NONE, factor: float = 1.0,
                       original_len: float = 0.0, turns_low: float = 1.0, turns_high: float = 32.0):
    """Frequencies (radians per position, float64 [rotary_dim / 2]) and the factor on rotated vectors."""
    out = np.zeros(max(0, int(rotary_dim)) // 2, dtype=np.float64)
    scale = ctypes.c_double()
    status = _lib.splitkv_rope_freqs(
        int(rotary_dim), float(base), int(scaling), float(factor), float(original_len), float(turns_low),
        float(turns_high), out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ctypes.byref(scale))
    if status:
        raise SplitKVError("splitkv_rope_freqs", status)
    return out, scale.value


def splitkv_rope(positions, freqs, scale: float, q, k, q_out, k_out, interleaved: bool = False,
                 adjoint: bool = False) -> None:
    """q_out, k_out = the rotary positions (adjoint: their transpose) of q [n, Hq, d] and k [n, Hk, d]
    (k and k_out may be None) at positions [n] (int32 or int64); rotary_dim = 2 * freqs.numel()."""
    dev = _device_of(q, "q")
    code = _code(q, "q")
    dt = q.dtype
    shape = q.shape
    n, hq, d = shape
    flags = (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_ADJOINT if adjoint else 0)
    if positions.dtype is _I64:
        flags |= ROPE_POS64
    ppos = _dense(positions, "positions", (n,), _I64 if flags & ROPE_POS64 else _I32, dev)
    half = freqs.numel()
    pf = _dense(freqs, "freqs", (half,), torch.float64, dev)
    pq, sq = _strided(q, "q", shape, dt, dev)
    pqo, sqo = _strided(q_out, "q_out", shape, dt, dev)
    if k is None:
        hk, pk, pko, sk, sko = 0, 0, 0, (0, 0), (0, 0)
    else:
        hk = k.shape[1]
        pk, sk = _strided(k, "k", (n, hk, d), dt, dev)
        pko, sko = _strided(k_out, "k_out", (n, hk, d), dt, dev)
    args = _pack_rope(n, hq, hk, d, 2 * half, code, flags, scale, ppos, pf, pq, pqo, pk, pko, sq[0], sq[1], sqo[0],
                      sqo[1], sk[0], sk[1], sko[0], sko[1])
    _call(_lib.splitkv_rope, "splitkv_rope", dev, args)


def splitkv_tree_args(q, kb, vb, node_ptr, mask, k_cache, v_cache, page_table, context_lens, scale: float,
                      max_nodes: int, o, lse, status=None):
    """The checked arguments of splitkv_tree_attn (shapes as in the header) as its struct's bytes, and their device."""
    dev = _device_of(q, "q")
    code = _code(q, "q")
    dt = q.dtype
    if q.dim() != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("q is [nodes, heads, d], the caches [pages, page_size, heads, d], page_table [seqs, pages]")
    qs, cs, ts = q.shape, k_cache.shape, page_table.shape
    nq, hq, d = qs
    pages, page, hkv, _ = cs
    B, max_pages = ts
    new, cs = (nq, hkv, d), (pages, page, hkv, d)
    pq, sq = _strided(q, "q", qs, dt, dev)
    pkb, skb = _strided(kb, "kb", new, dt, dev)
    pvb, svb = _strided(vb, "vb", new, dt, dev)
    pk, sk = _strided(k_cache, "k_cache", cs, dt, dev)
    pv, sv = _strided(v_cache, "v_cache", cs, dt, dev)
    ptab, stab = _strided(page_table, "page_table", ts, _I32, dev)
    pm, sm = 0, 0
    if mask is not None:
        if mask.dtype is not torch.bool and mask.dtype is not torch.uint8:
            raise ValueError("mask must be bool or uint8")
        if mask.dim() != 2 or mask.shape[1] < max_nodes:
            raise ValueError(f"mask must be [nodes, columns] with {max_nodes} (max_nodes) columns or more")
        pm, sm = _strided(mask, "mask", (nq, mask.shape[1]), mask.dtype, dev)
        sm = sm[0]
    o_code = code if o.dtype is dt else DTYPE_F32
    return _pack_tree(
        B, nq, max_nodes, hq, hkv, d, code, o_code, page, pages, max_pages, scale, pq, pkb, pvb, pk, pv, pm,
        _dense(node_ptr, "node_ptr", (B + 1,), _I32, dev), _dense(context_lens, "context_lens", (B,), _I32, dev), ptab,
        _dense(o, "o", qs, dt if o_code == code else _F32, dev), _dense(lse, "lse", (nq, hq), _F32, dev),
        _status(status, dev), sq[0], sq[1], skb[0], skb[1], svb[0], svb[1], sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], sm,
        stab[0]), dev


def splitkv_tree_workspace_size(args, dev: int) -> int:
    """Workspace bytes of splitkv_tree_attn for splitkv_tree_args' result."""
    out = ctypes.c_size_t()
    if torch.cuda.current_device() == dev:
        status = _lib.splitkv_tree_workspace_size(args, ctypes.byref(out))
    else:
        with torch.cuda.device(dev):
            status = _lib.splitkv_tree_workspace_size(args, ctypes.byref(out))
    if status:
        raise SplitKVError("splitkv_tree_workspace_size", status)
    return out.value


def splitkv_tree_attn(args, ws, dev: int) -> None:
    """Attention of draft trees over the cache (args, dev from splitkv_tree_args)."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor on the device of the others")
    _call(_lib.splitkv_tree_attn, "splitkv_tree_attn", dev, args, ws.data_ptr(), ws.numel() * ws.element_size())


def splitkv_tree_verify(target, draft, tokens, parents, node_ptr, u_accept, u_sample, max_nodes: int, path, count,
                        next_token, status=None) -> None:
    """path, count, next_token = the verification of the drafted tokens (see the header)."""
    dev = _device_of(target, "target")
    code = _code(target, "target")
    if target.dim() != 2 or path.dim() != 2:
        raise ValueError("target is [nodes, vocab], path [seqs, max_path]")
    rows, ps = target.shape, path.shape
    nq, vocab = rows
    B, max_path = ps
    dt, tok = target.dtype, tokens.dtype
    pt, st = _strided(target, "target", rows, dt, dev)
    pd, sd = (0, (0, 1)) if draft is None else _strided(draft, "draft", rows, dt, dev)
    if tok is not _I32 and tok is not _I64:
        raise ValueError("tokens must be int32 or int64")
    args = _pack_verify(
        B, nq, max_nodes, vocab, code, 1 if tok is _I64 else 0, max_path, 0, pt, pd,
        _dense(tokens, "tokens", (nq,), tok, dev), _dense(parents, "parents", (nq,), _I32, dev),
        _dense(node_ptr, "node_ptr", (B + 1,), _I32, dev), _dense(u_accept, "u_accept", (nq,), _F32, dev),
        _dense(u_sample, "u_sample", (B,), _F32, dev), _dense(path, "path", ps, _I32, dev),
        _dense(count, "count", (B,), _I32, dev), _dense(next_token, "next_token", (B,), tok, dev), _status(status, dev),
        st[0], sd[0], max_path)
    _call(_lib.splitkv_tree_verify, "splitkv_tree_verify", dev, args)


def _apart(t, name: str, st) -> None:
    if 0 in st and any(n > 1 and s == 0 for n, s in zip(t.shape, st)):
        raise ValueError(f"{name} is written: its elements must not share memory")


def splitkv_tree_commit(k_cache, v_cache, page_table, context_lens, kb, vb, node_ptr, path, count, max_rows: int,
                        status=None) -> None:
    """Copy the path's rows of kb, vb ([layers, nodes, heads, d]) behind each sequence's context in the
    caches ([layers, pages, page_size, heads, d]); path None: every node, in order.  The four may leave the layer
    dimension out together."""
    dev = _device_of(k_cache, "k_cache")
    dt = k_cache.dtype
    cs, ns = k_cache.shape, kb.shape
    one = len(cs) == 4
    if len(cs) not in (4, 5) or len(ns) != len(cs) - 1 or page_table.dim() != 2:
        raise ValueError("the caches are [layers, pages, page_size, heads, d], kb and vb [layers, nodes, heads, d] (or all "
                         "without layers), page_table [seqs, pages]")
    pages, page, hkv, d = cs[-4:]
    layers, nq = 1 if one else cs[0], ns[-3]
    new = (nq, hkv, d) if one else (layers, nq, hkv, d)
    ts = page_table.shape
    B, max_pages = ts
    pk, sk = _strided(k_cache, "k_cache", cs, dt, dev)
    pv, sv = _strided(v_cache, "v_cache", cs, dt, dev)
    _apart(k_cache, "k_cache", sk)
    _apart(v_cache, "v_cache", sv)
    pkb, skb = _strided(kb, "kb", new, dt, dev)
    pvb, svb = _strided(vb, "vb", new, dt, dev)
    if one:
        sk, sv, skb, svb = (0, *sk), (0, *sv), (0, *skb), (0, *svb)
    ptab, stab = _strided(page_table, "page_table", ts, _I32, dev)
    ppath, spath, pcount = 0, (0,), 0
    if path is not None:
        if path.dim() != 2 or path.shape[1] < max_rows:
            raise ValueError(f"path must be [seqs, columns] with {max_rows} (max_rows) columns or more")
        ppath, spath = _strided(path, "path", (B, path.shape[1]), _I32, dev)
        pcount = _dense(count, "count", (B,), _I32, dev)
    args = _pack_commit(
        layers, B, nq, max_rows, hkv, d, k_cache.element_size(), page, pages, max_pages, pkb, pvb, pk, pv, ppath, pcount,
        _dense(node_ptr, "node_ptr", (B + 1,), _I32, dev), _dense(context_lens, "context_lens", (B,), _I32, dev), ptab,
        _status(status, dev), skb[0], skb[1], skb[2], svb[0], svb[1], svb[2], sk[0], sk[1], sk[2], sk[3], sv[0], sv[1],
        sv[2], sv[3], spath[0], stab[0])
    _call(_lib.splitkv_tree_commit, "splitkv_tree_commit", dev, args)
