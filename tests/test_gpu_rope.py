"""splitkv_rope / Rotary on the GPU against the 64-bit form, and inside SplitKVAttention."""

import numpy as np
import pytest
import torch

from draft_util import assert_within, half_step, rope_ref
from gpu_util import TOL_LSE, TOL_OUT, assert_close, small, to_dev

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _inputs(n, hq, hk, d, dt, far=1 << 20, seed=0, pos=torch.int32):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(n, hq, d, generator=g).to(dt).cuda()
    k = torch.randn(n, hk, d, generator=g).to(dt).cuda() if hk else None
    p = torch.randint(-far, far, (n,), generator=g).to(pos).cuda()
    return q, k, p


def _check(rot, x, got, pos, adjoint=False):
    ref, tol = rope_ref(x, pos, rot.freqs, rot.scale, rot.interleaved, adjoint)
    assert_within("rope", got, ref, tol, x.dtype)
    rd = rot.rotary_dim
    assert torch.equal(got[..., rd:].cpu(), x[..., rd:].cpu())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("n,hq,hk,d,rd", [(1, 1, 0, 64, 64), (3, 5, 1, 128, 128), (257, 32, 8, 128, 64), (33, 8, 8, 64, 16),
                                          (7, 3, 2, 128, 50), (5, 2, 2, 6, 4), (2, 1, 1, 2, 2), (129, 40, 8, 128, 112)])
def test_rope_matches_64_bits(splitkv, n, hq, hk, d, rd, dt, interleaved):
    from context_block_sparse_b200.rotary import Rotary
    q, k, pos = _inputs(n, hq, hk, d, DT[dt])
    rot = Rotary(d, rotary_dim=rd, interleaved=interleaved, scaling="parts", factor=4.0, original_len=4096)
    for adjoint in (False, True):
        turn = rot.backward if adjoint else rot.forward
        out = turn(pos, q, k)
        _check(rot, q, out if k is None else out[0], pos, adjoint)
        if k is not None:
            _check(rot, k, out[1], pos, adjoint)


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
def test_far_positions_and_int64(splitkv, scaling):
    """Positions up to 2^40 in int64: the angle is formed and reduced in float64 (2^40 * 2^-53 turns off at most)."""
    from context_block_sparse_b200.rotary import Rotary
    q, k, pos = _inputs(64, 2, 1, 64, torch.float32, far=1 << 20, pos=torch.int64)
    rot = Rotary(64, scaling=scaling, factor=16.0, original_len=8192)
    _check(rot, q, rot.forward(pos, q, k)[0], pos)
    far = pos * (1 << 11)                       # up to 2^31: the reference's own angle is off by 2^31 * 2^-53 rad
    _check(rot, q, rot.forward(far, q), far)


def test_strided_in_place_and_broadcast(splitkv):
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(128, rotary_dim=96)
    _, _, pos = _inputs(50, 1, 0, 2, torch.float32)
    for dt in DT.values():
        qkv = torch.randn(50, 4 + 2 + 2, 128, device="cuda").to(dt)      # fused projections
        q, k = qkv[:, :4], qkv[:, 4:6]
        keep = qkv.clone()
        out = rot.forward(pos, q, k)
        _check(rot, keep[:, :4], out[0], pos)
        _check(rot, keep[:, 4:6], out[1], pos)
        assert torch.equal(qkv, keep)
        rot.forward(pos, q, k, out=(q, k))                               # in place
        assert torch.equal(q, out[0]) and torch.equal(k, out[1]) and torch.equal(qkv[:, 6:], keep[:, 6:])
        hm = torch.randn(4, 50, 128, device="cuda").to(dt).transpose(0, 1)   # head-major
        res = torch.empty(4, 50, 128, device="cuda", dtype=dt).transpose(0, 1)
        rot.forward(pos, hm, out=(res,))
        _check(rot, hm, res, pos)
        one = torch.randn(50, 1, 128, device="cuda").to(dt).expand(50, 6, 128)   # one head broadcast
        _check(rot, one, rot.forward(pos, one), pos)
        odd = torch.randn(50 * 2 * 129 + 1, device="cuda").to(dt)[1:].view(50, 2, 129)[..., :128]   # no 16-byte rows
        _check(rot, odd, rot.forward(pos, odd), pos)


def test_gradient_against_differences(splitkv):
    """sum(w * rope(x)) has the gradient backward(w): central differences of the linear map are exact but for float32
    rounding (n values of magnitude ~1 summed in float64 on the host, each output off by 2^-21)."""
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(16, rotary_dim=12, interleaved=True, scaling="parts", factor=2.0, original_len=64)
    x, _, pos = _inputs(3, 2, 0, 16, torch.float32, far=100)
    w = torch.randn_like(x)
    g = rot.backward(pos, w).double().cpu()
    f = lambda y: (rot.forward(pos, y).double() * w.double()).sum().item()  # noqa: E731
    eps = 0.5
    for i in range(0, x.numel(), 7):
        e = torch.zeros_like(x).view(-1)
        e[i] = eps
        e = e.view_as(x)
        diff = (f(x + e) - f(x - e)) / (2 * eps)
        # two evaluations, each with every output of the token's head off by at most 2^-21 * 2 * (|a| + |b| + 1)
        lim = 2 / (2 * eps) * 2.0 ** -20 * 16 * 8
        assert abs(diff - g.view(-1)[i].item()) <= lim


def test_refusals_and_empty(splitkv):
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(64)
    q, k, pos = _inputs(4, 2, 1, 64, torch.bfloat16)
    with pytest.raises(ValueError, match="positions"):
        rot.forward(pos[:3], q)
    with pytest.raises(ValueError, match="positions"):
        rot.forward(pos.float(), q)
    with pytest.raises(ValueError, match="k must be"):
        rot.forward(pos, q, k.float())
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        rot.forward(pos, q.double())
    with pytest.raises(ValueError, match="contiguous"):
        rot.forward(pos, q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(splitkv.SplitKVError):                      # an output that overlaps its input
        big = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
        rot.forward(pos, big[:4], out=(big[1:],))
    empty = rot.forward(pos[:0], q[:0], k[:0])
    assert empty[0].shape == (0, 2, 64) and empty[1].shape == (0, 1, 64)


def test_streams_and_graph(splitkv):
    from context_block_sparse_b200.rotary import Rotary
    rot = Rotary(128)
    q, k, pos = _inputs(300, 8, 2, 128, torch.bfloat16)
    want = rot.forward(pos, q, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = rot.forward(pos, q, k)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rot.forward(pos, q, k)
    pos.add_(5)
    graph.replay()
    again = rot.forward(pos, q, k)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("rb", [False, True])
def test_attention_with_rotary(splitkv, rb):
    """SplitKVAttention(rotary=...) is the attention of the rotated tensors, and its gradients are theirs turned back."""
    from context_block_sparse_b200.rotary import Rotary
    from context_block_sparse_b200.torch_api import SplitKVAttention
    from oracle import attention as oatt
    w = small(Hq=4, Hkv=2, d=64, anchors=20)
    rot = Rotary(64, rotary_dim=32, base=500.0)
    t = {n: to_dev(b) for n, b in w.bits.items()}
    kb, vb = (None, None) if rb else (t["kb"], t["vb"])
    att = SplitKVAttention(w.sample_lens, w.anchors, w.block_size, 4, 2, 64, w.kv_chunk, num_workers=148,
                           block_keys_in_context=rb, rotary=rot)
    o, lse = att.forward(t["q"], t["k"], t["v"], kb, vb, w.scale)
    g = att.backward(t["q"], t["k"], t["v"], kb, vb, o, lse, t["dout"], w.scale)
    g16 = att.backward(t["q"], t["k"], t["v"], kb, vb, o, lse, t["dout"], w.scale, grad_dtype=torch.bfloat16)
    # positions by the definition: offset in the sample; block rows from their anchor on
    starts = np.concatenate([[0], np.cumsum(w.sample_lens)])
    seq = lambda a: int(np.searchsorted(starts, a, side="right")) - 1  # noqa: E731
    cpos = torch.tensor([i - starts[seq(i)] for i in range(int(starts[-1]))])
    rpos = torch.tensor([int(a) - starts[seq(a)] + r for a in w.anchors for r in range(w.block_size)])

    def turned(x, pos):          # what the kernel hands on: the rotated values in bf16
        return rot.forward(pos.int().cuda(), x).double().cpu().numpy()

    q2, k2 = turned(t["q"], rpos), turned(t["k"], cpos)
    kb2 = None if rb else turned(t["kb"], rpos)
    args = (q2, k2, w.f64("v"), kb2 if not rb else w.f64("kb"), w.f64("vb"))
    ro, rl = oatt.attention_fwd(*args, w.sample_lens, w.anchors, w.block_size, w.scale, block_keys_in_context=rb)
    assert_close("o", o.double().cpu().numpy(), ro, TOL_OUT)
    assert_close("lse", lse.double().cpu().numpy(), rl, TOL_LSE)
    rg = oatt.attention_bwd(*args, w.f64("dout"), w.sample_lens, w.anchors, w.block_size, w.scale,
                            block_keys_in_context=rb)
    for name, pos in (("dq", rpos), ("dk", cpos), ("dkb", rpos)):
        if rb and name == "dkb":
            continue
        want, _ = rope_ref(torch.from_numpy(np.asarray(rg[name])), pos, rot.freqs, rot.scale, False, True)
        # the turn keeps a pair's length: an error of TOL_OUT in both elements is sqrt(2) of it in one
        assert_close(name, g[name].double().cpu().numpy(), want.numpy(), TOL_OUT * 2 ** 0.5)
        assert torch.equal(g16[name], g[name].bfloat16())
    assert_close("dv", g["dv"].double().cpu().numpy(), rg["dv"], TOL_OUT)


def test_attention_with_rotary_after_a_plan_update(splitkv):
    """The positions are those of the plan as it is, not as it was made."""
    from context_block_sparse_b200.rotary import Rotary
    from context_block_sparse_b200.torch_api import SplitKVAttention
    rot, made = Rotary(64, base=500.0), [([30, 130], [35, 20, 140]), ([100, 60], [10, 70, 120])]   # (the larger first)
    g = torch.Generator().manual_seed(5)
    t = [torch.randn(*s, generator=g).bfloat16().cuda() for s in
         ((48, 4, 64), (160, 2, 64), (160, 2, 64), (48, 2, 64), (48, 2, 64))]
    att = SplitKVAttention(*made[0], 16, 4, 2, 64, 64, num_workers=148, rotary=rot)
    att.forward(*t, 0.125)
    splitkv.splitkv_plan_update(att.plan, *made[1])
    splitkv.splitkv_plan_upload(att.plan)
    got = att.forward(*t, 0.125)
    want = SplitKVAttention(*made[1], 16, 4, 2, 64, 64, num_workers=148, rotary=rot).forward(*t, 0.125)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_refuses_another_head_size(splitkv):
    from context_block_sparse_b200.rotary import Rotary
    from context_block_sparse_b200.torch_api import SplitKVAttention
    with pytest.raises(ValueError, match="heads of 128"):
        SplitKVAttention([100], [10], 16, 1, 1, 64, 64, rotary=Rotary(128))
