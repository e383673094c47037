"""Cross attention on the GPU against the 64-bit form of attention_oracle.py:
lengths from 0 and 1 to thousands, every padded head size, shared key heads,
masks that leave rows empty, infinities and NaN in masked places, strided
layouts, HIP graphs and streams."""
import math

import pytest
import torch

import attention_oracle as ao
import image_stencil_amd as isa
from gpu_util import say

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _qkv(n, lq, lk, hq, hkv, d, dtype, seed=0, qscale=1.5):
    return (_randn((n, lq, hq, d), dtype, 3 * seed + 1, qscale), _randn((n, lk, hkv, d), dtype, 3 * seed + 2),
            _randn((n, lk, hkv, d), dtype, 3 * seed + 3))


def _check(got, want, bound, label):
    got = got.detach().cpu().double()
    same = (got == want) | ((got - want).abs() <= bound)   # equal infinities too
    assert same.all(), "%s: %d of %d off, worst %.3g over its bound" % (
        label, int((~same).sum()), same.numel(), float(((got - want).abs() / bound.clamp_min(1e-300)).nan_to_num(1e9).max()))


def _compare(out, lse, q, k, v, see=None, scale=None, label=""):
    d, lk = q.shape[3], k.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    if see is not None:   # the oracle skips masked keys whatever they hold
        k, v = k.clone(), v.clone()
    o, l, *rest = ao.attention(q.double(), k.double(), v.double(), scale, see)
    bo, bl = ao.attention_bounds(o, l, *rest, lk, d, q.dtype)
    _check(out, o, bo, label + " out")
    if lse is not None:
        _check(lse, l, bl, label + " lse")


def _run(q, k, v, mask=None, lengths=None, scale=None, label=""):
    out, lse = isa.cross_attention(q.cuda(), k.cuda(), v.cuda(), None if mask is None else mask.cuda(),
                                   None if lengths is None else lengths.cuda(), scale, return_lse=True)
    see = None
    if mask is not None or lengths is not None:
        see = torch.ones(q.shape[0], k.shape[1], dtype=torch.bool)
        if mask is not None:
            see &= mask.bool()
        if lengths is not None:
            see &= torch.arange(k.shape[1])[None] < lengths[:, None]
    _compare(out, lse, q, k, v, see, scale, label)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 64, 72, 80, 96, 104, 128, 136, 160, 192, 200, 256])
def test_head_sizes(dtype, d):
    say("head", dtype, d)
    _run(*_qkv(2, 70, 150, 2, 1, d, dtype), label="many queries")
    _run(*_qkv(2, 1, 150, 2, 1, d, dtype), label="one query")


@pytest.mark.parametrize("lq", [1, 2, 31, 33, 64, 65, 127, 129, 300])
@pytest.mark.parametrize("lk", [1, 2, 31, 32, 63, 64, 65, 129, 257, 1000])
def test_lengths(lq, lk):
    say("lengths", lq, lk)
    _run(*_qkv(1, lq, lk, 3, 3, 64, F16, lq + lk))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (6, 3), (8, 8), (40, 2), (7, 1), (64, 1)])
@pytest.mark.parametrize("lq", [1, 5, 90])
def test_shared_key_heads(hq, hkv, lq):
    say("heads", hq, hkv, lq)
    _run(*_qkv(2, lq, 203, hq, hkv, 64, BF16, hq))


@pytest.mark.parametrize("n,lq,lk,hq,hkv,d", [(1, 1, 40000, 8, 1, 128), (3, 2, 9001, 4, 4, 64), (1, 3, 20011, 2, 2, 256),
                                              (1, 130, 9001, 1, 1, 40), (1, 40, 16384, 1, 1, 128)])
def test_few_queries_many_keys(n, lq, lk, hq, hkv, d):
    """The keys of a row are split over workgroups; masked too, a part of them
    left empty as a whole."""
    say("long", n, lq, lk)
    q, k, v = _qkv(n, lq, lk, hq, hkv, d, BF16)
    _run(q, k, v)
    mask = torch.rand(n, lk, generator=torch.Generator().manual_seed(4)) < 0.5
    mask[:, lk // 3:] = False
    mask[:, -1] = True
    _run(q, k, v, mask)
    _run(q, k, v, lengths=torch.tensor([lk // 2, 1, 0][:n], dtype=torch.int32))


@pytest.mark.parametrize("lq", [1, 33, 200])
def test_masks_and_lengths(lq):
    """Lengths of 0, 1, all, below 0 and beyond lk; masks with holes, whole tiles
    masked, only the last key left, nothing left."""
    n, lk = 6, 333
    q, k, v = _qkv(n, lq, lk, 4, 2, 64, F16, lq)
    lengths = torch.tensor([0, 1, lk, 64, -5, 100000], dtype=torch.int32)
    _run(q, k, v, lengths=lengths, label="lengths")
    mask = torch.rand(n, lk, generator=torch.Generator().manual_seed(3)) < 0.5
    mask[0] = False
    mask[1, :-1] = False
    mask[2, :200] = False
    mask[3, 64:320] = False
    mask[4] = True
    _run(q, k, v, mask, label="mask")
    _run(q, k, v, mask.to(torch.uint8) * 255, label="mask bytes")
    _run(q, k, v, mask, lengths, label="both")


@pytest.mark.parametrize("lq", [1, 50])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_what_masked_keys_hold_has_no_effect(lq, bad):
    n, lk = 2, 200
    q, k, v = _qkv(n, lq, lk, 2, 2, 64, F16)
    mask = torch.rand(n, lk, generator=torch.Generator().manual_seed(5)) < 0.5
    kb, vb = k.clone(), v.clone()
    kb[~mask] = bad
    vb[~mask] = bad
    want = isa.cross_attention(q.cuda(), k.cuda(), v.cuda(), mask.cuda())
    got = isa.cross_attention(q.cuda(), kb.cuda(), vb.cuda(), mask.cuda())
    assert torch.equal(got, want)
    lengths = torch.tensor([70, 0], dtype=torch.int32)
    kb, vb = k.clone(), v.clone()
    for b in range(n):
        kb[b, lengths[b]:] = bad
        vb[b, lengths[b]:] = bad
    want = isa.cross_attention(q.cuda(), k.cuda(), v.cuda(), key_lengths=lengths.cuda())
    got = isa.cross_attention(q.cuda(), kb.cuda(), vb.cuda(), key_lengths=lengths.cuda())
    assert torch.equal(got, want) and (got[1] == 0).all()


def test_no_keys_and_no_queries():
    q, k, v = _qkv(2, 3, 0, 2, 2, 64, F16)
    out, lse = isa.cross_attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    q, k, v = _qkv(2, 0, 5, 2, 2, 64, F16)
    assert isa.cross_attention(q.cuda(), k.cuda(), v.cuda()).shape == (2, 0, 2, 64)


@pytest.mark.parametrize("lq", [1, 150])
def test_large_scores_and_scales(lq):
    """Scores in the hundreds (a softmax without its maximum would overflow),
    rising along the keys so that the running maximum moves at every tile;
    negative and large factors."""
    q, k, v = _qkv(1, lq, 700, 2, 2, 64, BF16, 9)
    q = (q.abs() + 0.5).to(BF16)
    k = (k.abs() * torch.linspace(0.1, 8.0, 700)[None, :, None, None]).to(BF16)
    _run(q, k, v, label="rising")
    _run(q, k.flip(1), v, label="falling")
    _run(q, k, v, scale=-0.3, label="negative")
    _run(q, k, v, scale=3.0, label="peaked")
    one = torch.zeros_like(q)
    _run(one, k, v, label="uniform")


@pytest.mark.parametrize("lq", [2, 100])
def test_strided_layouts(lq):
    """k and v of one packed projection, heads before tokens, one prompt for the
    whole batch, an output that is a slice."""
    n, lk, hq, hkv, d = 3, 90, 4, 2, 64
    q, k, v = _qkv(n, lq, lk, hq, hkv, d, F16, lq)
    want = isa.cross_attention(q.cuda(), k.cuda(), v.cuda())
    kv = torch.stack([k, v], 2).cuda()
    assert torch.equal(isa.cross_attention(q.cuda(), kv[:, :, 0], kv[:, :, 1]), want)
    qt, kt, vt = (t.cuda().permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (q, k, v))
    assert torch.equal(isa.cross_attention(qt, kt, vt), want)
    big = torch.full((n, lq, 3 * hq, d), 7.0, dtype=F16, device="cuda")
    plan = isa.CrossAttention(qt, kt, vt, big[:, :, hq:2 * hq])
    plan.forward(qt, kt, vt, big[:, :, hq:2 * hq])
    assert torch.equal(big[:, :, hq:2 * hq], want)
    assert (big[:, :, :hq] == 7).all() and (big[:, :, 2 * hq:] == 7).all()
    shared = isa.cross_attention(q.cuda(), k[:1].cuda().expand(n, -1, -1, -1), v[:1].cuda().expand(n, -1, -1, -1))
    each = isa.cross_attention(q.cuda(), k[:1].repeat(n, 1, 1, 1).cuda(), v[:1].repeat(n, 1, 1, 1).cuda())
    assert torch.equal(shared, each)


def test_joining_two_sets_of_keys_by_lse():
    q, k, v = _qkv(2, 60, 300, 2, 2, 64, F16)
    parts = [isa.cross_attention(q.cuda(), t[0].cuda(), t[1].cuda(), return_lse=True)
             for t in ((k[:, :110], v[:, :110]), (k[:, 110:], v[:, 110:]))]
    lse = torch.stack([l for _, l in parts]).cpu().double()
    w = torch.softmax(lse, 0).permute(0, 1, 3, 2)[..., None]
    joined = sum(w[i] * parts[i][0].cpu().double() for i in range(2))
    o, l, *rest = ao.attention(q.double(), k.double(), v.double(), 0.125)
    bo, bl = ao.attention_bounds(o, l, *rest, 300, 64, F16)
    # each part is within its bound, and a weighted mean of two bounds is at most both together
    _check(joined, o, 3 * bo, "joined")
    _check(torch.logsumexp(lse, 0), l, 3 * bl, "joined lse")


def test_keys_beyond_32_bit_offsets():
    """A cache whose entries and tokens lie far apart: token strides of 2^22
    elements over 600 keys reach 5 GiB into one tensor."""
    lk, stride = 600, 1 << 22
    cache = torch.empty((lk * stride,), dtype=F16, device="cuda")
    k, v = (cache.as_strided((1, lk, 1, 64), (0, stride, 64, 1), 64 * i) for i in range(2))
    q, kc, vc = _qkv(1, 40, lk, 1, 1, 64, F16)
    k.copy_(kc)
    v.copy_(vc)
    say("far keys")
    for rows in (1, 40):
        out = isa.cross_attention(q[:, :rows].contiguous().cuda(), k, v)
        assert torch.equal(out, isa.cross_attention(q[:, :rows].contiguous().cuda(), kc.cuda(), vc.cuda()))
    _compare(out, None, q, kc, vc)


@pytest.mark.parametrize("lq,lk", [(1, 20000), (1, 100), (200, 500)])
def test_graph_replays_and_streams(lq, lk):
    """A captured forward replays to the eager bits, with eager work between; the
    workspace may hold anything before a call."""
    q, k, v = (t.cuda() for t in _qkv(2, lq, lk, 4, 2, 64, F16))
    lengths = torch.tensor([lk, lk // 3], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    plan = isa.CrossAttention(q, k, v, out)
    ws = plan.new_workspace()
    plan.forward(q, k, v, out, key_lengths=lengths, workspace=ws)
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.forward(q, k, v, out, key_lengths=lengths, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(q, k, v, out, key_lengths=lengths, workspace=ws)
    for _ in range(3):
        out.fill_(float("nan"))
        if ws is not None:
            ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_the_same_bits_every_time():
    q, k, v = (t.cuda() for t in _qkv(1, 3, 30000, 4, 2, 128, BF16))
    want = isa.cross_attention(q, k, v)
    for _ in range(3):
        assert torch.equal(isa.cross_attention(q, k, v), want)
