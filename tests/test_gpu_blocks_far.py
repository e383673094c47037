"""The operators around attention where offsets pass 32 bits: entries, rows and tokens
that lie far apart, and a store of held states of more than 4 GiB."""
import pytest
import torch

import blocks_oracle as bo
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _check, _compare, _randn

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _far(shape, strides, dtype, at=0):
    size = at + 1 + sum((s - 1) * d for s, d in zip(shape, strides))
    return torch.empty(size, dtype=dtype, device="cuda").as_strided(shape, strides, at)


@pytest.mark.parametrize("strides", [(2 ** 31 + 1, 2 ** 29 + 3, 1), (1001, 2 ** 30 + 1, 1)])
def test_norm(strides):
    say("norm far", strides)
    shape, c = (2, 3, 1001), 1001
    x, y = _randn(shape, F16, 1), _randn(shape, F16, 2)
    w = 1.0 + 0.1 * _randn((c,), F32, 3)
    wx, bx, wz, bz = bo.block_norm(x, y, "layer", weight=w)
    far = [_far(shape, strides, F16) for _ in range(4)]
    far[0].copy_(x), far[1].copy_(y)
    isa.BlockNorm(c, "layer").apply(far[0], far[1], weight=w.cuda(), x_out=far[2], out=far[3])
    _check(far[2], wx, bx, "sum")
    _check(far[3], wz, bz, "normed")


@pytest.mark.parametrize("n,rows,k,m", [(3, 5, 72, 50), (3, 600, 72, 130)])
def test_dense(n, rows, k, m):
    say("dense far", rows)
    x, w, r = _randn((n, rows, k), BF16, 1), _randn((m, k), BF16, 2, 1.5 / k ** 0.5), _randn((n, rows, m), BF16, 3)
    xs, rs, out = (_far(t.shape, (2 ** 31 + 64, s, 1), BF16) for t, s in ((x, 80), (r, m + 1), (r, m + 3)))
    xs.copy_(x), rs.copy_(r)
    plan = isa.Dense(xs, w.cuda(), out=out, residual=rs, activation="silu")
    _check(plan.forward(xs, w.cuda(), None, rs, out), *bo.dense(x, w, None, "silu", r), "dense")


@pytest.mark.parametrize("rows,k,m,tile", [(1100, 72, 300, 64), (5001, 520, 3001, 256)])
def test_rows_at_the_largest_stride(rows, k, m, tile):
    """Rows and weights 2^21 elements apart: the last row of a 256-row tile lies 2^30 bytes
    from its first."""
    say("dense far rows", rows)
    x, w = _randn((1, rows, k), F16, 1), _randn((m, k), F16, 2, 1.5 / k ** 0.5)
    xs, ws = _far(x.shape, (0, 2 ** 21, 1), F16), _far(w.shape, (2 ** 21, 1), F16)
    xs.copy_(x), ws.copy_(w)
    plan = isa.Dense(xs, ws)
    assert plan.info()["tile"] == (tile, tile)
    _check(plan.forward(xs, ws), *bo.dense(x, w), "dense")


def test_put_and_get():
    say("held far")
    n, length, heads, d = 2, 70, 2, 40
    k, v = _randn((n, length, heads, d), F16, 1), _randn((n, length, heads, d), F16, 2)
    ks, vs = _far(k.shape, (d, 2 ** 25 + 5, 2 ** 24 + 1, 1), F16), _far(v.shape, (2 ** 31 + 1, 2 * d, d, 1), F16)
    ks.copy_(k), vs.copy_(v)
    h = isa.HeldStates(n, length, heads, d).put(ks, vs)
    assert torch.equal(h.data, isa.HeldStates(n, length, heads, d).put(k.cuda(), v.cuda()).data)
    ks.zero_(), vs.zero_()
    gk, gv = h.get(k_out=ks, v_out=vs)
    assert torch.equal(gk.cpu().double(), bo.held(k)) and torch.equal(gv.cpu().double(), bo.held(v))


@pytest.mark.parametrize("lq,kernel", [(3, "is_k15_held_attention"), (2100, "is_k14_held_load, is_k11_attention")])
def test_attention_over_a_long_store(lq, kernel):
    """1.2 million tokens of 8 heads of 256: 4.9 GB of held bytes, twice that as 16-bit
    numbers. A few visible tokens at both ends."""
    length, heads, d, count = 1200000, 8, 256, 96
    at = length - count
    h = isa.HeldStates(1, length, heads, d, dtype=BF16)
    assert h.bytes > 2 ** 32
    k, v = _randn((1, 2 * count, heads, d), BF16, 1), _randn((1, 2 * count, heads, d), BF16, 2)
    h.put(k[:, :count].cuda(), v[:, :count].cuda()).put(k[:, count:].cuda(), v[:, count:].cuda(), at=at)
    parts = [h.get(a, count) for a in (0, at)]
    hk, hv = (torch.cat([p[i] for p in parts], 1).cpu() for i in range(2))
    assert torch.equal(hk[:, count:].double(), bo.held(k[:, count:]))
    assert torch.equal(hv[:, count:].double(), bo.held(v[:, count:]))
    see = torch.rand(1, 2 * count, generator=torch.Generator().manual_seed(0)) < 0.5
    mask = torch.zeros(1, length, dtype=torch.bool)
    mask[:, :count], mask[:, at:] = see[:, :count], see[:, count:]
    q = _randn((1, lq, heads, d), BF16, 3, 1.5)
    plan, lse = isa.HeldAttention(q, h), torch.empty(1, heads, lq, device="cuda")
    say("held attention far", plan.info())
    assert plan.info()["kernel"] == kernel
    out = plan.forward(q.cuda(), h, key_mask=mask.cuda(), lse=lse)
    _compare(out, lse, q, hk, hv, see, None, "far")
