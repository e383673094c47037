"""The sum and norm between blocks on the GPU against the 64-bit form: channel counts
around every shape of the kernel, odd ones, all types, strides, in place, vectors
shared or per entry, rows of zeros, infinities and NaN, graphs and streams."""
import itertools

import pytest
import torch

import blocks_oracle as bo
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _check, _randn

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _case(n, length, c, dtype, norm="rms", post=None, modulated=True, seed=0):
    kw = {"y": _randn((n, length, c), dtype, 2 * seed + 1, 0.7), "residual_scale": 0.5}
    if norm:
        kw.update(weight=1 + 0.1 * _randn((c,), F32, seed + 5), bias=0.1 * _randn((c,), F32, seed + 6))
    if post:
        kw["post_weight"] = 1 + 0.1 * _randn((c,), F32, seed + 7)
    if modulated:
        kw["gate"] = _randn((n, c), dtype, seed + 8)
        if norm:
            kw.update(scale=_randn((n, c), dtype, seed + 9, 0.3), shift=_randn((n, c), dtype, seed + 10, 0.3))
    return _randn((n, length, c), dtype, 2 * seed, 2.0) + 0.5, kw


def _run(x, kw, norm, post, eps=1e-6, label="", **outs):
    kw = dict(kw)
    plan = isa.BlockNorm(x.shape[2], norm, post, eps, kw.pop("residual_scale", 1.0))
    dev = {k: v.cuda() for k, v in kw.items()}
    return plan.apply(x.cuda(), **dev, **outs)


def _compare(x, kw, norm, post, eps=1e-6, label=""):
    got_x, got = _run(x, kw, norm, post, eps)
    want_x, bx, want, b = bo.block_norm(x, norm=norm, post=post, eps=eps, **kw)
    if kw.get("y") is not None:
        _check(got_x, want_x, bx, label + " x_out")
    if norm:
        _check(got, want, b, label + " out")
    else:
        assert got is None


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("c", [1, 7, 8, 9, 64, 127, 129, 256, 321, 512, 513, 1001, 1024, 1030, 2048, 2056, 4095, 4104, 8192,
                               8200, 16384])
def test_channels(c, dtype):
    say("norm", c, dtype)
    n, length = (2, 5) if c < 2000 else (2, 2)
    x, kw = _case(n, length, c, dtype, "layer", "rms", seed=c)
    _compare(x, kw, "layer", "rms", label="c %d" % c)


@pytest.mark.parametrize("norm,post,modulated", list(itertools.product(["rms", "layer", None], ["rms", "layer", None],
                                                                       [True, False])))
def test_kinds(norm, post, modulated):
    say("norm kinds", norm, post, modulated)
    for dtype, c in ((F16, 320), (F32, 1001)):
        x, kw = _case(3, 7, c, dtype, norm, post, modulated, seed=3)
        _compare(x, kw, norm, post, label="%s %s" % (norm, post))


@pytest.mark.parametrize("n,length", [(1, 1), (16, 1), (1, 5000), (7, 1111), (3, 4099)])
def test_rows(n, length):
    """From one row to more than the groups of threads that walk them."""
    say("norm rows", n, length)
    for dtype, c in ((BF16, 40), (F16, 512)):
        x, kw = _case(n, length, c, dtype, "rms", None, True, seed=length)
        _compare(x, kw, "rms", None, label="%d x %d" % (n, length))


def test_norm_alone_and_sum_alone():
    x, kw = _case(2, 9, 96, F16)
    say("norm alone")
    for keep in (("weight",), ("bias",), ("scale",), ("shift",), ()):
        _compare(x, {k: kw[k] for k in keep}, "rms", None, label=str(keep))
    for keep in (("y",), ("y", "gate"), ("y", "residual_scale")):
        _compare(x, {k: kw[k] for k in keep}, None, None, label=str(keep))
    got_x, _ = isa.BlockNorm(96).apply(x.cuda())
    assert torch.equal(got_x.cpu(), x)


def test_rows_at_any_element_and_in_place():
    say("norm strides")
    for dtype, c in itertools.product((F32, F16), (33, 64, 1000)):
        x, kw = _case(2, 6, c, dtype, "layer", "layer", seed=c)
        wide_x, wide_y = torch.zeros(2, 6, 2 * c + 3, dtype=dtype), torch.zeros(6, 2, c + 1, dtype=dtype)
        wide_x[:, :, :c], wide_y[:, :, :c] = x, kw["y"].transpose(0, 1)
        wx, wy = wide_x.cuda(), wide_y.cuda()
        packed = torch.cat([kw["gate"], kw["scale"], kw["shift"]], 1).cuda()
        dev = {k: kw[k].cuda() for k in ("post_weight", "weight", "bias")}
        dev.update(gate=packed[:, :c], scale=packed[:, c:2 * c], shift=packed[:, 2 * c:])
        plan = isa.BlockNorm(c, "layer", "layer", 1e-6, 0.5)
        want = plan.apply(x.cuda(), kw["y"].cuda(), **{**dev, "gate": kw["gate"].cuda(), "scale": kw["scale"].cuda(),
                                                       "shift": kw["shift"].cuda()})
        out = torch.full((2, 6, c + 5), 7.0, dtype=dtype, device="cuda")
        gx, gz = plan.apply(wx[:, :, :c], wy.transpose(0, 1)[:, :, :c], out=out[:, :, :c], x_out=wx[:, :, :c], **dev)
        assert gx.data_ptr() == wx.data_ptr()
        assert torch.equal(gx, want[0]) and torch.equal(gz, want[1])
        assert (out[:, :, c:] == 7).all() and (wx[:, :, c:] == 0).all()
        y2 = kw["y"].cuda()
        gx, gz = plan.apply(x.cuda(), y2, out=y2, **dev)     # the output over the block's output
        assert torch.equal(gx, want[0]) and torch.equal(y2, want[1])
        x2 = x.cuda()
        assert torch.equal(plan.apply(x2, kw["y"].cuda(), x_out=x2, **dev)[0], want[0])


def test_one_row_of_vectors_for_all_entries():
    x, kw = _case(3, 4, 72, F16, seed=4)
    say("norm shared vectors")
    one = {k: kw[k][:1].cuda() for k in ("gate", "scale", "shift")}
    every = {k: v.expand(3, -1).contiguous() for k, v in one.items()}
    rest = {k: kw[k].cuda() for k in ("y", "weight", "bias")}
    plan = isa.BlockNorm(72)
    for a, b in zip(plan.apply(x.cuda(), **one, **rest), plan.apply(x.cuda(), **every, **rest)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_rows_of_zeros_and_small_rows(dtype):
    say("norm zeros", dtype)
    for c in (64, 1001):
        x = torch.zeros(1, 3, c, dtype=dtype)
        x[0, 1] = torch.finfo(dtype).tiny * 4
        x[0, 2, 0] = 1.0
        for norm in ("rms", "layer"):
            _, z = _run(x, {}, norm, None)
            want, b = bo.block_norm(x, norm=norm)[2:]
            _check(z, want, b, norm)
            assert (z[0, 0] == 0).all()
    x = torch.full((1, 1, 64), 2.0 ** -64, dtype=BF16)     # mean square under fp32's normal numbers, eps 0
    _, z = _run(x, {}, "rms", None, eps=0.0)
    assert (z - 1).abs().max() <= 2.0 ** -7


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_number_that_is_none_spoils_its_row_alone(bad):
    say("norm", bad)
    for c in (40, 1001, 5000):
        x, kw = _case(2, 8, c, F16, "rms", None, True, seed=1)
        clean = _run(x, kw, "rms", None)
        x[1, 3, c // 2] = bad
        got = _run(x, kw, "rms", None)
        rows = torch.ones(2, 8, dtype=torch.bool)
        rows[1, 3] = False
        for a, b in zip(got, clean):
            assert torch.equal(a.cpu()[rows], b.cpu()[rows])
        assert torch.isnan(got[1][1, 3].cpu()).any()


def test_in_a_graph_and_on_streams():
    say("norm graph")
    x, kw = _case(4, 50, 512, BF16, "rms", "rms", seed=9)
    dev = {k: v.cuda() for k, v in kw.items() if k != "residual_scale"}
    plan, buf = isa.BlockNorm(512, "rms", "rms", residual_scale=0.5), x.cuda()
    outs = torch.empty_like(buf), torch.empty_like(buf)
    plan.apply(buf, x_out=outs[0], out=outs[1], **dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.apply(buf, x_out=outs[0], out=outs[1], **dev)
    for seed in range(3):
        buf.copy_(_randn(x.shape, BF16, 50 + seed))
        want = plan.apply(buf, **dev)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs[0].zero_(), outs[1].zero_()
    torch.cuda.synchronize()
    plan.apply(buf, x_out=outs[0], out=outs[1], stream=side.cuda_stream, **dev)
    side.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_as_many_rows_as_an_int_counts():
    """The last step of a walk over the rows of an entry passes 2^31."""
    rows = 2 ** 31 - 1
    x = torch.full((1, 1, 1), 2.0, dtype=torch.bfloat16, device="cuda").expand(1, rows, 1)
    _, out = isa.BlockNorm(1, eps=12.0).apply(x)      # 2 / sqrt(4 + 12)
    assert out.shape == x.shape
    assert all(bool((part == 0.5).all()) for part in out.view(-1).split(1 << 28))
