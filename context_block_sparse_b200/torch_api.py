"""Convenience wrapper over the C entry points for torch users.

Allocates the outputs and workspaces with torch (device memory only) and calls
splitkv_attn_fwd / splitkv_merge / splitkv_attn_bwd in order on the current
stream, with the rotary call around them when a Rotary is given.  No arithmetic happens here.
"""

from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import (
    WS_BWD, WS_FWD, Plan, splitkv_attn_bwd, splitkv_attn_fwd, splitkv_cast_bf16, splitkv_merge, splitkv_plan,
    splitkv_plan_upload, splitkv_workspace_size,
)


class SplitKVAttention:
    """One problem (packed samples + anchors + head layout) bound to a device plan."""

    def __init__(self, sample_lens, anchors, block_size: int, num_q_heads: int, num_kv_heads: int,
                 head_dim: int, kv_chunk: int, num_workers: Optional[int] = None,
                 num_bwd_workers: int = 0, q_slice: int = 0, equal_count: bool = False,
                 device: Optional[torch.device] = None, block_keys_in_context: bool = False,
                 partial_bf16: bool = False, tile_cost: bool = False, fwd_tile_cost: bool = False,
                 dynamic_claim: bool = False, contiguous_schedule: bool = False, rotary=None):
        """block_keys_in_context: reading B of the block keys (the block's own tokens are
        the context positions after its anchor); kb, vb are then unused (pass None)
        and backward() returns no dkb, dvb.  partial_bf16: bf16 partial records.
        tile_cost / fwd_tile_cost: backward / forward LPT items costed by executed tile work.
        dynamic_claim: the CTAs claim the items in LPT order at run time.
        contiguous_schedule: the contiguous baseline schedule instead of LPT.
        rotary: a Rotary applied to q, k and kb inside forward and backward (which take and differentiate the
        unrotated ones): a context token's position is its offset in its sample, row r of block b's is its
        anchor's offset + r (the context positions the block's tokens stand for).  After splitkv_plan_update the next call
        of forward or backward brings the new positions, in place where their numbers stay (that call must not be
        captured)."""
        self.device = torch.device("cuda") if device is None else torch.device(device)
        if num_workers is None:
            num_workers = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.plan: Plan = splitkv_plan(sample_lens, anchors, block_size, num_q_heads, num_kv_heads, head_dim,
                                       kv_chunk, num_workers, num_bwd_workers, q_slice, equal_count,
                                       block_keys_in_context, partial_bf16, tile_cost, fwd_tile_cost,
                                       dynamic_claim, contiguous_schedule)
        self.block_keys_in_context = bool(block_keys_in_context)
        splitkv_plan_upload(self.plan)
        self.block_size = block_size
        self.num_q_heads = num_q_heads
        self.num_kv_heads = num_kv_heads
        self.head_dim = head_dim
        self.ws_fwd = torch.empty(splitkv_workspace_size(self.plan, WS_FWD), dtype=torch.uint8, device=self.device)
        self._ws_bwd = None
        self.rotary = rotary
        if rotary is not None:
            if rotary.head_dim != head_dim:
                raise ValueError(f"rotary is for heads of {rotary.head_dim}, not {head_dim}")
            self._ctx_pos = self._row_pos = None
            self._place()
        self._grad32 = None   # float32 gradients behind bf16 ones (grad_dtype=torch.bfloat16)

    def _place(self):
        """The plan's positions on the device: in the same tensors as long as their sizes stay."""
        p = self.plan.problem
        lens, anc = (np.asarray(x, dtype=np.int64) for x in self.plan._keep)
        starts = np.concatenate([[0], np.cumsum(lens)])
        ctx = np.arange(starts[-1]) - np.repeat(starts[:-1], lens)
        rows = (anc - starts[np.searchsorted(starts, anc, side="right") - 1])[:, None] + np.arange(p.block_size)
        new = [torch.from_numpy(x.astype(np.int32).ravel()) for x in (ctx, rows)]
        if self._ctx_pos is not None and [x.shape for x in new] == [self._ctx_pos.shape, self._row_pos.shape]:
            self._ctx_pos.copy_(new[0])       # (a captured graph holds these)
            self._row_pos.copy_(new[1])
        else:
            self._ctx_pos, self._row_pos = (x.to(self.device) for x in new)
        self._placed = p

    def ws_bwd(self) -> torch.Tensor:
        if self._ws_bwd is None:
            self._ws_bwd = torch.empty(splitkv_workspace_size(self.plan, WS_BWD), dtype=torch.uint8,
                                       device=self.device)
        return self._ws_bwd

    def _rotated(self, q, k, kb):
        """q, k, kb as the attention takes them (the rotated ones are this call's own)."""
        if self.rotary is None:
            return q, k, kb
        if self._placed is not self.plan.problem:   # splitkv_plan_update: new positions (not inside a capture)
            self._place()
        if kb is None:
            q = self.rotary.forward(self._row_pos, q)
        else:
            q, kb = self.rotary.forward(self._row_pos, q, kb)
        return q, self.rotary.forward(self._ctx_pos, k), kb

    def forward(self, q, k, v, kb, vb, scale: float, out_dtype=torch.float32, o=None, lse=None):
        Nq = q.shape[0]
        q, k, kb = self._rotated(q, k, kb)
        if o is None:
            o = torch.empty((Nq, self.num_q_heads, self.head_dim), dtype=out_dtype, device=q.device)
        if lse is None:
            lse = torch.empty((Nq, self.num_q_heads), dtype=torch.float32, device=q.device)
        splitkv_attn_fwd(self.plan, q, k, v, scale, self.ws_fwd)
        splitkv_merge(self.plan, q, kb, vb, scale, self.ws_fwd, o, lse)
        return o, lse

    def _grad_buffers(self, q, k, v, kb, vb, dtype):
        a = dict(dtype=dtype, device=q.device)
        return {
            "dq": torch.empty(q.shape, **a),
            "dk": torch.empty(k.shape, **a),
            "dv": torch.empty(v.shape, **a),
            "dkb": None if self.block_keys_in_context else torch.empty(kb.shape, **a),
            "dvb": None if self.block_keys_in_context else torch.empty(vb.shape, **a),
        }

    def backward(self, q, k, v, kb, vb, o, lse, dout, scale: float, grads=None, grad_dtype=torch.float32):
        """Gradients dq, dk, dv (and dkb, dvb).  grad_dtype=torch.bfloat16 returns them in bf16:
        the kernels still accumulate in fp32 (into buffers kept by this object), and
        splitkv_cast_bf16 rounds the finished arrays."""
        if grad_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("grad_dtype must be torch.float32 or torch.bfloat16")
        if grads is None:
            grads = self._grad_buffers(q, k, v, kb, vb, grad_dtype)
        if grad_dtype == torch.float32:
            g32 = grads
        else:
            if self._grad32 is None or self._grad32["dq"].shape != q.shape or self._grad32["dk"].shape != k.shape:
                self._grad32 = self._grad_buffers(q, k, v, kb, vb, torch.float32)
            g32 = self._grad32
        q, k, kb = self._rotated(q, k, kb)
        splitkv_attn_bwd(self.plan, q, k, v, kb, vb, o, lse, dout, g32["dq"], g32["dk"], g32["dv"],
                         g32["dkb"], g32["dvb"], scale, self.ws_bwd())
        if self.rotary is not None:   # gradients of the unrotated q, k, kb, in place
            dq, dk, dkb = g32["dq"], g32["dk"], g32["dkb"]
            self.rotary.backward(self._row_pos, dq, dkb, out=(dq, dkb))
            self.rotary.backward(self._ctx_pos, dk, out=(dk,))
        if grad_dtype == torch.bfloat16:
            for n, t in grads.items():
                if t is not None:
                    splitkv_cast_bf16(g32[n], t)
        return grads
