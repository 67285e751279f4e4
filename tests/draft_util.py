"""Plain 64-bit forms of the rotary and draft-tree operators (numpy / torch float64, one sequence at a time), and
the error bounds their kernels are held to."""

from __future__ import annotations

import math

import numpy as np
import torch


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------------------------ rotary
def rope_ref(x, positions, freqs, scale, interleaved, adjoint=False):
    """float64 [n, heads, d] of x turned by positions * freqs; and the bound on a kernel's error before the
    output's rounding: scale (|a| + |b|) 2^-21.  (The turn reduced in float64 and rounded to float32 once, off by
    2^-24 of a half turn or 2^-22.3 rad; sine and cosine two float32 steps each; three float32 roundings of the
    products and their sum.)"""
    y = x.detach().double().cpu()
    h = freqs.numel()
    ang = positions.cpu().double()[:, None, None] * freqs.cpu().double()
    c, s = torch.cos(ang) * scale, torch.sin(ang) * scale * (-1 if adjoint else 1)
    out, bound = y.clone(), torch.zeros_like(y)
    ia = torch.arange(0, 2 * h, 2) if interleaved else torch.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    bound[..., ia] = bound[..., ib] = scale * (a.abs() + b.abs()) * 2.0 ** -21
    return out, bound


# --------------------------------------------------------------------------------- attention
def gather_context(cache, table_row, n, page):
    """[n, heads, d] of the first n cached tokens of a sequence (cache [pages, page, heads, d], on the CPU)."""
    t = torch.arange(n)
    return cache[table_row.long()[t // page], t % page]


def tree_ref(q, kb, vb, node_ptr, mask, k_cache, v_cache, table, lens, scale, max_nodes=None):
    """o, lse in float64 and the bounds on a kernel's errors (arrays on the CPU)."""
    nq, hq, d = q.shape
    hkv, page = k_cache.shape[2], k_cache.shape[1]
    G = hq // hkv
    o = torch.zeros(nq, hq, d, dtype=torch.float64)
    lse = torch.full((nq, hq), -math.inf, dtype=torch.float64)
    tol_o, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    u = half_step(q.dtype)
    for b in range(len(lens)):
        i0, i1, n = int(node_ptr[b]), int(node_ptr[b + 1]), int(lens[b])
        T = i1 - i0
        if T == 0:
            continue
        kc, vc = gather_context(k_cache, table[b], n, page), gather_context(v_cache, table[b], n, page)
        see = torch.ones(T, T, dtype=torch.bool) if mask is None else mask[i0:i1, :T].bool()
        see = torch.cat([torch.ones(T, n, dtype=torch.bool), see], 1)
        for h in range(hq):
            k = torch.cat([kc[:, h // G], kb[i0:i1, h // G]]).double()
            v = torch.cat([vc[:, h // G], vb[i0:i1, h // G]]).double()
            qh = q[i0:i1, h].double()
            s = torch.where(see, (qh @ k.T) * scale, -math.inf)
            m = s.amax(1, keepdim=True) if s.shape[1] else torch.full((T, 1), -math.inf, dtype=torch.float64)
            p = torch.where(see, torch.exp(s - torch.where(m == -math.inf, 0.0, m)), 0.0)
            l = p.sum(1, keepdim=True)
            p = p / torch.where(l == 0, 1.0, l)
            # only seen values enter (a product with an unseen infinity or NaN would not be 0)
            vz = torch.where(see[:, :, None], v[None], 0.0)
            o[i0:i1, h] = (p[:, :, None] * vz).sum(1)
            lse[i0:i1, h] = torch.where(l == 0, -math.inf, m + torch.log(torch.where(l == 0, 1.0, l)))[:, 0]
            # Scores: d float32 products summed (each step at most 2^-23 of the terms' magnitude), two roundings of
            # the scaled score; exponentials and sums 2^-21.  P is rounded once to the keys' type.  Sums over n keys
            # in float32 with truncation: n 2^-23.
            mag = torch.where(see, qh.abs() @ k.abs().T, 0.0).nan_to_num(0.0, 0.0, 0.0).amax(1, keepdim=True) * abs(scale)
            ds = mag * (d + 4) * 2.0 ** -23 + 2.0 ** -21
            keys = s.shape[1]
            A = (p[:, :, None] * vz.abs()).sum(1)
            tol_o[i0:i1, h] = A * (1.01 * u + 2 * ds + keys * 2.0 ** -23)
            tol_lse[i0:i1, h] = (ds + keys * 2.0 ** -23)[:, 0] + 2.0 ** -22 * (1 + lse[i0:i1, h].abs().nan_to_num(0, 0, 0))
    return o, lse, tol_o, tol_lse


def assert_within(name, got, ref, tol, out_dtype):
    """|got - ref| <= tol + one rounding of the output; non-finite values in the same places.  Below the type's
    smallest normal number the steps no longer shrink with the value: they are smallest_normal * eps wide, so one
    rounding is off by up to half of that whatever the value (an fp16 result near 5e-6, the exact value rounded, is
    off by 3e-8 = 2^-25, more than 2^-11 of it)."""
    got = got.detach().double().cpu()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{name}: infinities differ"
    err = (got - ref).abs()[fine]
    floor = torch.finfo(out_dtype).smallest_normal * half_step(out_dtype)
    lim = (tol + half_step(out_dtype) * (ref.abs() + tol) + floor + 1e-30)[fine]
    if err.numel():
        worst = float((err / lim).max())
        assert worst <= 1.0, f"{name}: error {float(err.max()):.3e}, {worst:.2f} times its bound"


# ------------------------------------------------------------------------------ verification
def verify_ref(target, draft, tokens, parents, node_ptr, u_accept, u_sample, max_path):
    """The walk by its definition, residual rows formed in float64 (arrays on the CPU as numpy float64 / ints)."""
    B = len(node_ptr) - 1
    clean = lambda r: np.where((r > 0) & np.isfinite(r), r, 0.0)  # noqa: E731
    path = np.full((B, max_path), -1, dtype=np.int64)
    count, nxt = np.zeros(B, dtype=np.int64), np.full(B, -1, dtype=np.int64)
    V = target.shape[1]
    for b in range(B):
        n0, n = int(node_ptr[b]), int(node_ptr[b + 1] - node_ptr[b])
        if n == 0:
            continue
        cur, k = 0, 1
        path[b, 0] = 0
        while True:
            p = clean(target[n0 + cur])
            q = None if draft is None else clean(draft[n0 + cur])
            r, S, moved = p.copy(), 1.0, False
            for i in range(cur + 1, n):
                x = int(tokens[n0 + i])
                if parents[n0 + i] != cur or not 0 <= x < V or k >= max_path:
                    continue
                if u_accept[n0 + i] * S * (1.0 if q is None else q[x]) < r[x]:
                    path[b, k] = i
                    cur, k, moved = i, k + 1, True
                    break
                if q is None:
                    S, r[x] = max(S - r[x], 0.0), 0.0
                else:
                    r = np.maximum(r - S * q, 0.0)
                    S = r.sum()
            if not moved:
                break
        if r.sum() <= 0:
            r = p
        count[b] = k
        if r.sum() > 0:
            cum = np.cumsum(r)
            nxt[b] = min(int(np.searchsorted(cum, min(u_sample[b] * cum[-1], np.nextafter(cum[-1], 0)), side="right")),
                         int(np.flatnonzero(r > 0)[-1]))
    return path, count, nxt


def random_parents(rng, n, kind):
    if kind == "chain":
        return np.arange(-1, n - 1)
    p = np.array([-1] + [int(rng.integers(0, i)) if rng.random() < 0.5 else max(0, (i - 1) // 3) for i in range(1, n)])
    return np.minimum(p, np.arange(-1, n - 1))
