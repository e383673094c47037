"""Attention to held states on the GPU where the states are loaded into the workspace
first (many rows), against the 64-bit form on what get() returns; each plan is checked to
be of this kind. Never-stored blocks also for the plans that read the bytes directly."""
import math

import pytest
import torch

import blocks_oracle as bo
import image_stencil_amd as isa
import test_gpu_blocks_together as together
from gpu_util import say
from test_gpu_cross_attention import _compare, _qkv, _randn
from test_gpu_lds_poison import _poison_lib

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
LOADED, DIRECT = "is_k14_held_load, is_k11_attention", "is_k15_held_attention"
# n, queries, keys, query heads, key heads, elements: just over 1024 row tiles (over 128 elements: 512)
SHAPES = [(3, 1500, 77, 8, 4, 40), (2, 4200, 333, 4, 4, 64), (1, 4100, 130, 8, 8, 128), (4, 2100, 100, 2, 2, 256),
          (2, 3100, 45, 6, 3, 200), (3, 5500, 1, 2, 2, 8), (2, 4150, 65, 4, 4, 96)]


def _held(k, v, **kw):
    h = isa.HeldStates(k.shape[0], k.shape[1], k.shape[2], k.shape[3], dtype=k.dtype)
    return h.put(k.cuda(), v.cuda(), **kw)


def _plan(q, h, kernel=LOADED, **kw):
    plan = isa.HeldAttention(q, h, **kw)
    say("held loaded", tuple(q.shape), (h.length, h.heads), plan.info()["kernel"], plan.info()["grid"])
    assert plan.info()["kernel"] == kernel
    return plan


def _see(n, lk, mask, lengths):
    if mask is None and lengths is None:
        return None
    see = torch.ones(n, lk, dtype=torch.bool)
    if mask is not None:
        see &= mask
    if lengths is not None:
        see &= torch.arange(lk)[None] < lengths[:, None]
    return see


def _run(shape, dtype, mask=None, lengths=None, scale=None, seed=0):
    n, lq, lk, hq, hkv, d = shape
    q, k, v = _qkv(*shape, dtype, seed)
    see = _see(n, lk, mask, lengths)
    if see is not None:      # what is held in masked places has no effect
        k[~see], v[~see] = float("inf"), float("nan")
    h = _held(k, v)
    plan = _plan(q, h, scale=scale)
    lse = torch.empty(n, hq, lq, device="cuda")
    kw = {"key_mask": None if mask is None else mask.cuda(), "key_lengths": None if lengths is None else lengths.cuda()}
    guard = torch.full((plan.workspace_bytes + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    out = plan.forward(q.cuda(), h, lse=lse, workspace=guard[:plan.workspace_bytes], **kw)
    assert (guard[plan.workspace_bytes:] == 0x5A).all()
    hk, hv = (t.cpu() for t in h.get())
    _compare(out, lse, q, hk, hv, see, scale, str(shape))
    assert torch.equal(out, plan.forward(q.cuda(), h, **kw))
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype):
    _run(shape, dtype)


@pytest.mark.parametrize("shape", SHAPES[:5])
def test_lengths_and_masks(shape):
    """All keys, some, one and none; holes; masked keys that hold no numbers."""
    n, lk = shape[0], shape[2]
    lengths = torch.tensor([lk, 0, 1, lk // 2][:n], dtype=torch.int32)
    mask = torch.rand(n, lk, generator=torch.Generator().manual_seed(1)) < 0.4
    _run(shape, F16, None, lengths)
    _run(shape, BF16, mask, None)
    _run(shape, F16, mask, torch.tensor([lk + 9, lk - 1, -3, 33][:n], dtype=torch.int32))
    _run(shape, F16, torch.zeros(n, lk, dtype=torch.bool), None)


@pytest.mark.parametrize("scale", [4.0, -1.0, 1e-3])
def test_scales(scale):
    _run(SHAPES[1], F16, scale=scale)


def test_blocks_of_very_different_sizes():
    q, k, v = _qkv(*SHAPES[1], F16)
    v[:, :32] *= 2.0 ** -12
    v[:, 32:64] *= 2.0 ** -20
    k[:, 64:96] *= 2.0 ** -14
    v[:, 96:128] *= 2.0 ** 13
    h = _held(k, v)
    out = _plan(q, h).forward(q.cuda(), h)
    hk, hv = (t.cpu() for t in h.get())
    _compare(out, None, q, hk, hv, None, None, "sizes")


def test_no_visible_key():
    say("held loaded, no key")
    n, lq, lk, hq, hkv, d = SHAPES[1]
    q, k, v = _qkv(*SHAPES[1], F16)
    q[0, 0, 0, 0] = float("inf")
    k[:], v[:] = float("nan"), float("inf")
    h, lse = _held(k, v), torch.ones(n, hq, lq, device="cuda")
    lengths = torch.tensor([0, -5], dtype=torch.int32).cuda()
    out = _plan(q, h).forward(q.cuda(), h, key_lengths=lengths, lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all()
    empty = isa.HeldStates(n, 0, hkv, d)
    lse.fill_(1)
    out = _plan(q, empty).forward(q.cuda(), empty, lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_every_visible_key_counts_once():
    lq, lk = 33000, 777
    q = torch.zeros(1, lq, 1, 32, dtype=F16)
    k, v = torch.zeros(1, lk, 1, 32, dtype=F16), torch.zeros(1, lk, 1, 32, dtype=F16)
    for e in range(10):
        v[0, :, 0, e] = ((torch.arange(lk) >> e) & 1).half()
    h, lse = _held(k, v), torch.empty(1, 1, lq, device="cuda")
    out = _plan(q, h).forward(q.cuda(), h, lse=lse)
    assert (lse.cpu() - math.log(lk)).abs().max() < 1e-5
    counts, want = out.cpu().double()[0, :, 0] * lk, bo.held(v)[0, :, 0].sum(0)
    assert ((counts - want).abs() <= want * 2.0 ** -10 + 1e-9).all()


def test_strides():
    for shape in (SHAPES[0], SHAPES[3]):
        n, lq, lk, hq, hkv, d = shape
        q, k, v = _qkv(*shape, F16)
        h = _held(k, v)
        want = _plan(q, h).forward(q.cuda(), h)
        wide = torch.full((n, lq, hq + 3, d + 8), float("nan"), dtype=F16, device="cuda")
        wide[:, :, 2:2 + hq, :d] = q.cuda()
        big = torch.full((n, lq + 1, hq, d + 16), 3.0, dtype=F16, device="cuda")
        qs, out = wide[:, :, 2:2 + hq, :d], big[:, :lq, :, :d]
        assert torch.equal(_plan(qs, h, out=out).forward(qs, h, out), want)
        assert (big[..., d:] == 3).all() and (big[:, lq:] == 3).all()


@pytest.mark.parametrize("shape,kernel", [(SHAPES[1], LOADED), (SHAPES[3], LOADED), ((2, 40, 333, 4, 4, 64), DIRECT),
                                          ((4, 1, 2000, 2, 2, 256), DIRECT)])
def test_blocks_that_were_never_stored(shape, kernel):
    """A store whose memory held anything: only the visible tokens were put."""
    n, lq, lk, hq, hkv, d = shape
    q, k, v = _qkv(*shape, BF16)
    lengths = torch.tensor([40, 64, 33, 1][:n], dtype=torch.int32)
    for fill in (0xFF, 0x7E):      # scales that are no numbers; numbers that their scales make infinite
        h = isa.HeldStates(n, lk, hkv, d, dtype=BF16)
        h.data.fill_(fill)
        h.put(k[:, :64].cuda(), v[:, :64].cuda(), key_lengths=lengths.cuda())
        plan = _plan(q, h, kernel)
        hk, hv = (t.cpu() for t in h.get())
        lse = torch.empty(n, hq, lq, device="cuda")
        out = plan.forward(q.cuda(), h, key_lengths=lengths.cuda(), lse=lse)
        _compare(out, lse, q, hk, hv, _see(n, lk, None, lengths), None, "lengths")
        mask = _see(n, lk, None, lengths) & (torch.arange(lk) % 3 > 0)[None]
        out = plan.forward(q.cuda(), h, key_mask=mask.cuda(), lse=lse)
        _compare(out, lse, q, hk, hv, mask, None, "mask")


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[3]])
def test_in_a_graph_and_on_streams(shape):
    n, lq, lk, hq, hkv, d = shape
    q, k, v = (t.cuda() for t in _qkv(*shape, BF16))
    h = isa.HeldStates(n, lk, hkv, d, dtype=BF16)
    plan, out = _plan(q, h), torch.empty_like(q)
    ws = plan.new_workspace()

    def step(**kw):
        h.put(k, v, **kw)
        plan.forward(q, h, out, workspace=ws, **kw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        for t in (q, k, v):
            t.copy_(_randn(t.shape, BF16, 10 * seed + t.shape[1]))
        other = isa.HeldStates(n, lk, hkv, d, dtype=BF16).put(k, v)
        want = plan.forward(q, other)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(h.data, other.data)
    side = torch.cuda.Stream()
    out.zero_(), h.data.zero_()
    torch.cuda.synchronize()
    step(stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("shape", SHAPES)
def test_lds_poison(shape):
    """LDS that is read before it was written would put NaN into the results."""
    n, lk = shape[0], shape[2]
    q, k, v = (t.cuda() for t in _qkv(*shape, F16))
    lengths = torch.tensor([lk, 0, 1, lk // 2][:n], dtype=torch.int32).cuda()
    mask = (_randn((n, lk), torch.float32, 5) < 0.3).cuda()
    h = isa.HeldStates(n, lk, shape[4], shape[5]).put(k, v)
    plan, other = _plan(q, h), _plan(q, h)
    other._lib = _poison_lib()
    for kw in ({}, {"key_mask": mask}, {"key_lengths": lengths}):
        assert torch.equal(plan.forward(q, h, **kw), other.forward(q, h, **kw)), kw


def test_a_block_of_many_rows_step_by_step():
    """The operators around attention together, with states that are loaded first."""
    n, lq, lk, hq, hkv, d = 2, 4200, 100, 4, 4, 64
    _plan(torch.empty(n, lq, hq, d, dtype=F16), isa.HeldStates(n, lk, hkv, d, device="cpu"))
    together.test_a_block_step_by_step(n, lq, lk, hq, hkv, d, F16, 512)
