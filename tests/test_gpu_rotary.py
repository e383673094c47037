"""Rotary positions and the query/key norm on the GPU against the 64-bit forms
of attention_oracle.py, at layouts, sizes, strides and positions where they can
go wrong."""
import pytest
import torch

import attention_oracle as ao
import image_stencil_amd as isa
from gpu_util import say

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _positions(n, length, axes, seed, most=4000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most, (n, length, axes), generator=g, dtype=torch.int32)


def _check(got, want, bound, label):
    got = got.detach().cpu().double()
    err = (got - want).abs()
    ok = err <= bound
    assert ok.all(), "%s: %d of %d off, worst %.3g over its bound" % (
        label, int((~ok).sum()), ok.numel(), float((err / bound.clamp_min(1e-300)).max()))


def _case(x, pos, rot, axes, layout, out=None, **kw):
    """Run x (CPU) through the kernel and check it."""
    plan = isa.Rotary(x.shape[3], rot, axes=axes, layout=layout, **kw)
    y = plan.apply(x.cuda(), pos.cuda())
    f = ao.frequencies(rot, axes, **{k: v for k, v in kw.items() if k != "magnitude"})
    want, m = ao.rotate(x.double(), pos.expand(x.shape[0], -1, -1), rot, axes, layout, f, kw.get("magnitude", 1.0))
    bound = ao.rotary_bound(want, m, x.dtype)
    bound[..., rot:] = 0       # elements that do not turn pass through as they are
    _check(y, want, bound, "rotary")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,axes", [(64, 64, 1), (128, 128, 2), (128, 64, 1), (80, 40, 1), (96, 96, 3), (40, 8, 2),
                                        (256, 256, 1), (24, 24, 1), (7, 4, 1), (250, 246, 3), (2, 2, 1), (1, 0, 1),
                                        (72, 0, 1), (200, 198, 1)])
def test_rotary_heads(dtype, layout, d, rot, axes):
    """Head sizes and turned parts: 16-byte chunks, 8-byte chunks, single
    elements, odd numbers of chunks that pass through."""
    say("rotary", dtype, layout, d, rot, axes)
    _case(_randn((2, 5, 3, d), dtype, d + rot), _positions(2, 5, axes, d), rot, axes, layout)


@pytest.mark.parametrize("n,length,heads", [(1, 1, 1), (1, 1, 32), (3, 1, 5), (16, 1, 16), (1, 257, 1), (2, 1000, 6),
                                            (1, 7, 33), (65, 3, 2)])
def test_rotary_sizes(n, length, heads):
    say("rotary sizes", n, length, heads)
    for dtype in (F16, F32):
        _case(_randn((n, length, heads, 64), dtype, n + length), _positions(n, length, 2, heads), 64, 2, "half")


def test_rotary_many_tokens_walk_several_heads():
    """Enough threads that each walks several heads with one set of sines."""
    for heads, layout in ((16, "half"), (13, "interleaved")):
        n, length = 2, 9001
        x = _randn((n, length, heads, 128), BF16, heads)
        pos = torch.arange(length, dtype=torch.int32)[None, :, None]
        say("rotary many", heads, layout)
        _case(x, pos, 128, 1, layout)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "ramp"])
def test_rotary_scaled_far_positions(scaling):
    """Positions up to 2^31: the angle keeps its whole precision."""
    pos = torch.tensor([[[2 ** 31 - 1], [-2 ** 31], [2 ** 30 + 1], [1234567], [0]]], dtype=torch.int32)
    for dtype in (F32, F16):
        _case(_randn((1, 5, 4, 64), dtype, 5), pos, 48, 1, "half", scaling=scaling, factor=8.0, original_len=2048,
              ramp=(1.0, 32.0), magnitude=1.2079441541679836)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_rotary_strides_in_place_and_slices(dtype):
    """A slice of a packed projection, heads before tokens, an offset base, odd
    strides, one entry repeated over the batch, and in place."""
    n, length, heads, d = 2, 33, 4, 64
    pos = _positions(n, length, 1, 3)
    plan, f = isa.Rotary(d), ao.frequencies(d, 1)

    def check(x, out, label):
        want, m = ao.rotate(x.detach().cpu().double(), pos, d, 1, "half", f)
        got = plan.apply(x, pos.cuda(), out=out)
        _check(got, want, ao.rotary_bound(want, m, dtype), label)

    packed = _randn((n, length, 3 * heads, d), dtype, 1).cuda()
    before = packed.clone()
    check(packed[:, :, heads:2 * heads], None, "packed slice")
    assert torch.equal(packed, before)
    other = _randn((n, heads, length, d), dtype, 2).cuda().permute(0, 2, 1, 3)
    out = torch.zeros((n, heads, length, d), dtype=dtype, device="cuda").permute(0, 2, 1, 3)
    check(other, out, "heads before tokens")
    odd = _randn((n, length, heads, d + 3), dtype, 4).cuda()[..., :d]
    check(odd, None, "odd strides")
    shared = _randn((1, length, heads, d), dtype, 6).cuda().expand(n, -1, -1, -1)
    check(shared, None, "one entry for the batch")
    x = packed[:, :, heads:2 * heads]
    want, m = ao.rotate(x.cpu().double(), pos, d, 1, "half", f)
    plan.apply(x, pos.cuda(), out=x)
    _check(x, want, ao.rotary_bound(want, m, dtype), "in place")
    assert torch.equal(packed[:, :, :heads], before[:, :, :heads])
    assert torch.equal(packed[:, :, 2 * heads:], before[:, :, 2 * heads:])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d,rot,layout", [(64, 64, "half"), (128, 96, "interleaved"), (80, 40, "half"),
                                          (40, 40, "half"), (256, 64, "interleaved"), (7, 4, "half"),
                                          (251, 250, "half"), (96, 0, "half")])
def test_qk_norm(dtype, kind, d, rot, layout):
    """q and k of different lengths and head counts, weights on q only."""
    say("qk", dtype, kind, d, rot, layout)
    q, k = _randn((2, 19, 6, d), dtype, 1, 3.0), _randn((2, 5, 2, d), dtype, 2, 0.3)
    w = 1 + 0.3 * _randn((d,), F32, 3)
    pq, pk = _positions(2, 19, 1, 4), _positions(1, 5, 1, 5)
    eps = 1e-5
    plan, f = isa.Rotary(d, rot, layout=layout), ao.frequencies(rot, 1)
    yq, yk = plan.apply_qk_norm(q.cuda(), k.cuda(), pq.cuda(), pk.cuda(), w.cuda(), None, eps=eps, norm=kind)
    for got, x, weight, pos in ((yq, q, w, pq), (yk, k, torch.ones(d), pk.expand(2, -1, -1))):
        z, size = ao.norm(x.double(), weight.double(), eps, kind)
        want, _ = ao.rotate(z, pos, rot, 1, layout, f)
        _, m = ao.rotate(size, pos, rot, 1, layout, f)
        _check(got, want, ao.rotary_bound(want, m, dtype) + ao.norm_error(d, kind) * (1 + ao.half(dtype)) * m, "qk")


def test_qk_norm_packed_in_place_and_empty():
    """Queries and keys of one packed projection normed in place; an empty k."""
    n, length, h, d = 2, 50, 4, 64
    qkv = _randn((n, length, 3 * h, d), F16, 7).cuda()
    before = qkv.clone()
    pos = _positions(1, length, 2, 8)
    plan, f = isa.Rotary(d, axes=2), ao.frequencies(d, 2)
    plan.apply_qk_norm(qkv[:, :, :h], qkv[:, :, h:2 * h], pos.cuda(), q_out=qkv[:, :, :h], k_out=qkv[:, :, h:2 * h])
    z, size = ao.norm(before[:, :, :2 * h].cpu().double(), torch.ones(d).double(), 1e-6, "rms")
    want, _ = ao.rotate(z, pos.expand(n, -1, -1), d, 2, "half", f)
    _, m = ao.rotate(size, pos.expand(n, -1, -1), d, 2, "half", f)
    _check(qkv[:, :, :2 * h], want, ao.rotary_bound(want, m, F16) + ao.norm_error(d, "rms") * (1 + 2 ** -11) * m, "qk")
    assert torch.equal(qkv[:, :, 2 * h:], before[:, :, 2 * h:])
    q, k = _randn((n, 3, h, d), F16, 9).cuda(), torch.empty(n, 0, h, d, dtype=F16, device="cuda")
    yq, yk = plan.apply_qk_norm(q, k, pos[:, :3].cuda(), torch.empty(1, 0, 2, dtype=torch.int32, device="cuda"))
    z, size = ao.norm(q.cpu().double(), torch.ones(d).double(), 1e-6, "rms")
    want, m = ao.rotate(z, pos[:, :3].expand(n, -1, -1), d, 2, "half", f)
    _, m = ao.rotate(size, pos[:, :3].expand(n, -1, -1), d, 2, "half", f)
    _check(yq, want, ao.rotary_bound(want, m, F16) + ao.norm_error(d, "rms") * (1 + 2 ** -11) * m, "empty k")
    assert yk.shape == k.shape


def test_qk_norm_zero_rows_and_streams():
    """A head of zeros gives zeros (eps keeps the root), and a side stream's call
    gives the same bits."""
    plan = isa.Rotary(64)
    q = _randn((1, 40, 4, 64), BF16, 1).cuda()
    q[:, 3] = 0
    pos = _positions(1, 40, 1, 2).cuda()
    yq, yk = plan.apply_qk_norm(q, q[:, :, :2], pos)
    assert (yq[:, 3] == 0).all() and torch.isfinite(yq.float()).all()
    assert torch.equal(yq[:, :, :2], yk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        zq, _ = plan.apply_qk_norm(q, q[:, :, :2], pos)
    torch.cuda.synchronize()
    assert torch.equal(zq, yq)
