"""The operators around attention together, as a block uses them: every step against its
64-bit form on the inputs that it got, eagerly and in a captured graph; the example."""
import importlib.util
import os

import pytest
import torch

import attention_oracle as ao
import blocks_oracle as bo
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _check, _compare, _randn

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


class Block:
    """x, reference -> x; keeps every step's inputs and outputs when asked."""

    def __init__(self, n, lq, lk, hq, hkv, d, dtype, wide, kept=None):
        c = hq * d
        self.sizes, self.kept = (n, lq, lk, hq, hkv, d), kept
        g = lambda *s, k: _randn(s, dtype, sum(s) + k, 1.5 / s[-1] ** 0.5).cuda()      # noqa: E731
        self.wq, self.wkv, self.wo = g(c, c, k=1), g(2 * hkv * d, c, k=2), g(c, c, k=3)
        self.up, self.down = g(wide, c, k=4), g(c, wide, k=5)
        self.b = 0.1 * _randn((wide,), F32, 6).cuda()
        self.norms = [1 + 0.1 * _randn((s,), F32, 10 + i).cuda() for i, s in enumerate((c, c, c, d, d))]
        self.rotary = isa.Rotary(d)
        self.pre, self.mid = isa.BlockNorm(c, "rms"), isa.BlockNorm(c, "layer", "rms", residual_scale=0.5)
        self.held = isa.HeldStates(n, lk, hkv, d, dtype=dtype)
        self.at = torch.arange(max(lq, lk), dtype=torch.int32, device="cuda")[None, :, None].contiguous()

    def note(self, name, *values):
        if self.kept is not None:
            self.kept[name] = tuple(v.clone() if isinstance(v, torch.Tensor) else v for v in values)

    def __call__(self, x, ref, gate, scale, shift, lengths):
        n, lq, lk, hq, hkv, d = self.sizes
        c = hq * d
        _, r = self.pre.apply(ref, weight=self.norms[0])
        _, z = self.pre.apply(x, weight=self.norms[1])
        self.note("pre", x, self.norms[1], z)
        kv = isa.dense(r, self.wkv)
        self.note("kv", r, self.wkv, kv)
        q, kv = isa.dense(z, self.wq).view(n, lq, hq, d), kv.view(n, lk, 2, hkv, d)
        k, v = kv[:, :, 0], kv[:, :, 1]
        self.note("before rotation", q, k)
        self.rotary.apply_qk_norm(q, k, self.at[:, :lq], self.at[:, :lk], self.norms[3], self.norms[4], q_out=q, k_out=k)
        self.note("rotated", q, k)
        self.held.put(k, v, key_lengths=lengths)
        self.note("put", k, v, lengths)
        y = isa.held_attention(q, self.held, key_lengths=lengths)
        if self.kept is not None:
            self.note("attention", q, *self.held.get(), lengths, y)
        o = isa.dense(y.view(n, lq, c), self.wo)
        self.note("o", y.view(n, lq, c), self.wo, o)
        before = x.clone() if self.kept is not None else None
        x2, z = self.mid.apply(x, o, gate=gate, post_weight=self.norms[2], weight=self.norms[1], scale=scale, shift=shift)
        self.note("mid", before, o, x2, z)
        u = isa.dense(z, self.up, self.b, "gelu")
        self.note("up", z, u)
        self.note("down before", x2, u)
        plan = isa.Dense(u, self.down, out=x2, residual=x2)
        out = plan.forward(u, self.down, None, x2, x2)
        self.note("down", out)
        return out


def _inputs(n, lq, lk, c, dtype, seed):
    return [_randn(s, dtype, seed + i).cuda() for i, s in enumerate(((n, lq, c), (n, lk, c), (n, c), (n, c), (n, c)))]


@pytest.mark.parametrize("n,lq,lk,hq,hkv,d,dtype,wide", [(2, 1, 700, 8, 2, 64, BF16, 1024), (3, 150, 333, 4, 4, 40, F16, 328),
                                                         (1, 5, 64, 6, 2, 96, F16, 2304), (2, 900, 100, 8, 8, 32, BF16, 512)])
def test_a_block_step_by_step(n, lq, lk, hq, hkv, d, dtype, wide):
    say("block", n, lq, lk, hq, hkv, d, dtype)
    kept = {}
    block = Block(n, lq, lk, hq, hkv, d, dtype, wide, kept)
    x, ref, gate, scale, shift = _inputs(n, lq, lk, hq * d, dtype, 40)
    lengths = torch.tensor([lk - 7 * b for b in range(n)], dtype=torch.int32, device="cuda")
    block(x, ref, gate, scale, shift, lengths)
    torch.cuda.synchronize()
    kept = {k: tuple(v.cpu() if isinstance(v, torch.Tensor) else v for v in vs) for k, vs in kept.items()}
    norms = [w.cpu() for w in block.norms]
    a, w, z = kept["pre"]
    _check(z, *bo.block_norm(a, norm="rms", weight=w)[2:], "pre")
    a, w, got = kept["kv"]
    _check(got, *bo.dense(a, w), "kv")
    freqs = ao.frequencies(d, 1)
    for i, (name, length) in enumerate((("q", lq), ("k", lk))):
        t = kept["before rotation"][i].double()
        normed, size = ao.norm(t, norms[3 + i].double(), 1e-6, "rms")
        at = torch.arange(length)[None, :, None].expand(n, -1, 1)
        y, m = ao.rotate(normed, at, d, 1, "half", freqs)
        _, ms = ao.rotate(size, at, d, 1, "half", freqs)
        bound = ao.rotary_bound(y, m, dtype) + 2 * ao.norm_error(d, "rms") * ms
        _check(kept["rotated"][i], y, bound, "rotated " + name)
    k, v, ln = kept["put"]
    see = torch.arange(lk)[None] < ln[:, None]
    q, hk, hv, ln, y = kept["attention"]
    for got, want in ((hk, bo.held(k, see)), (hv, bo.held(v, see))):
        assert torch.equal(got.double(), want)
    _compare(y, None, q, hk, hv, see, None, "attention")
    a, w, got = kept["o"]
    _check(got, *bo.dense(a, w), "o")
    before, o, x2, z = kept["mid"]
    wx, bx, wz, bz = bo.block_norm(before, o, "layer", "rms", residual_scale=0.5, gate=gate.cpu(), post_weight=norms[2],
                                   weight=norms[1], scale=scale.cpu(), shift=shift.cpu())
    _check(x2, wx, bx, "mid x")
    _check(z, wz, bz, "mid z")
    z, u = kept["up"]
    _check(u, *bo.dense(z, block.up.cpu(), block.b.cpu(), "gelu"), "up")
    x2, u = kept["down before"]
    _check(kept["down"][0], *bo.dense(u, block.down.cpu(), None, "none", x2), "down")


def test_a_block_in_a_graph():
    """Captured once, replayed with new inputs between eager passes of another block."""
    say("block graph")
    n, lq, lk, hq, hkv, d = 2, 70, 1000, 4, 2, 64
    block, other = (Block(n, lq, lk, hq, hkv, d, BF16, 512) for _ in range(2))
    still = _inputs(n, lq, lk, hq * d, BF16, 3)
    lengths = torch.tensor([lk, 400], dtype=torch.int32, device="cuda")
    block(*still, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(*still, lengths)
    for seed in range(3):
        for t, v in zip(still, _inputs(n, lq, lk, hq * d, BF16, 100 * seed)):
            t.copy_(v)
        want = other(*still, lengths).clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), seed


def test_the_example_runs():
    say("held reference example")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "held_reference_block.py")
    spec = importlib.util.spec_from_file_location("held_reference_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    n, h, w, hr, wr = 2, 18, 40, 24, 20
    block = m.HeldReferenceBlock(m.weights(), n, h, w, hr, wr)
    frame, ref = _randn((n, h, w), F16, 1).cuda(), _randn((n, hr, wr), F16, 2).cuda()
    condition = _randn((n, 1, 8), F16, 3).cuda()
    block.hold(ref)
    y = block(frame, condition)
    assert y.shape == (n, h, w, m.CHANNELS) and torch.isfinite(y).all()
    block.hold(-ref)
    assert not torch.equal(y, block(frame, condition))     # the reference is attended to
