"""States held in 8 bits on the GPU: what is held against the table of e4m3 numbers,
bit for bit, and the attention to it against the 64-bit form on the loaded states."""
import math

import pytest
import torch

import blocks_oracle as bo
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _compare, _qkv, _randn

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def _equal(got, want, label=""):
    got = got.detach().cpu().double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert same.all(), "%s: %d of %d differ" % (label, int((~same).sum()), same.numel())


def _held(k, v, **kw):
    h = isa.HeldStates(k.shape[0], k.shape[1], k.shape[2], k.shape[3], dtype=k.dtype)
    return h.put(k.cuda(), v.cuda(), **kw)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 64, 72, 96, 128, 136, 160, 192, 200, 224, 248, 256])
def test_what_is_held(d, dtype):
    say("held", d, dtype)
    n, length, heads = 2, 70, 2
    k, v = _randn((n, length, heads, d), dtype, d), _randn((n, length, heads, d), dtype, d + 1, 3.0)
    gk, gv = _held(k, v).get()
    _equal(gk, bo.held(k), "k")
    _equal(gv, bo.held(v), "v")


@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 63, 64, 65, 1000])
def test_lengths(length):
    say("held lengths", length)
    k, v = _randn((2, length, 3, 40), F16, length), _randn((2, length, 3, 40), F16, length + 1)
    gk, gv = _held(k, v).get()
    _equal(gk, bo.held(k))
    _equal(gv, bo.held(v))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_size_of_number(dtype):
    """Blocks whose largest magnitude lies at, beside and between the borders of the
    scale, from the smallest numbers of the type to the largest; ties."""
    say("held sizes", dtype)
    f = torch.finfo(dtype)
    tops = [f.max, f.max / 1.5, f.tiny, f.smallest_normal / 64, 0.0]
    for e in (-30, -9, -1, 0, 7, 13) if dtype == F16 else (-140, -126, -121, -120, -119, -112, -60, 0, 100, 118):
        for s in (1.0, 1.75, 1.75 * (1 + f.eps), 1.75 * (1 - f.eps / 2), 1.0 - f.eps, 1.9375, 2.0 - f.eps):
            tops.append(s * 2.0 ** e)
    tops = torch.tensor(tops, dtype=torch.float64).to(dtype)
    k = torch.zeros(1, 32 * len(tops), 1, 32, dtype=dtype)
    between = (bo.E4M3[:-1] + bo.E4M3[1:]) / 2
    g = torch.Generator().manual_seed(1)
    for i, t in enumerate(tops.tolist()):
        fill = (torch.rand(32, 32, generator=g, dtype=torch.float64) * 2 - 1) * t
        fill[:16] *= 2.0 ** -torch.randint(0, 14, (16, 32), generator=g).double()
        fill[16:20] = between.repeat(2)[:128].reshape(4, 32) * (t / 448.0)
        fill[5, 7] = t
        k[0, 32 * i:32 * i + 32, 0] = fill.to(dtype)
    gk, gv = _held(k, -k).get()
    _equal(gk, bo.held(k))
    _equal(gv, bo.held(-k))


def test_infinities_and_nan_are_held_as_nan():
    say("held inf")
    k = _randn((1, 64, 2, 40), F16, 3)
    k[0, 5, 0, 3], k[0, 40, 1, 0], k[0, 41, 1, 39] = float("inf"), float("-inf"), float("nan")
    gk, gv = _held(k, k).get()
    _equal(gk, bo.held(k))
    _equal(gv, bo.held(k))
    assert torch.isnan(gk).sum() == 3


def test_masked_tokens_are_held_as_zeros():
    """Lengths from none to all, holes; infinities and huge numbers in masked places
    change nothing."""
    say("held masks")
    n, length = 4, 100
    k, v = _randn((n, length, 2, 72), BF16, 1), _randn((n, length, 2, 72), BF16, 2)
    lengths = torch.tensor([0, 1, 57, 300], dtype=torch.int32)
    mask = torch.rand(n, length, generator=torch.Generator().manual_seed(0)) < 0.5
    for m, ln in ((None, lengths), (mask, None), (mask, lengths)):
        see = torch.ones(n, length, dtype=torch.bool)
        if m is not None:
            see &= m
        if ln is not None:
            see &= torch.arange(length)[None] < ln[:, None]
        kk, vv = k.clone(), v.clone()
        kk[~see], vv[~see] = float("inf"), float("nan")
        kk[~see, 0, :7] = 3e38
        h = _held(kk, vv, key_mask=None if m is None else m.cuda(), key_lengths=None if ln is None else ln.cuda())
        gk, gv = h.get()
        _equal(gk, bo.held(k, see))
        _equal(gv, bo.held(v, see))
        h2 = _held(k, v, key_mask=None if m is None else m.to(torch.uint8).cuda() * 200,
                   key_lengths=None if ln is None else ln.cuda())
        assert torch.equal(h.data, h2.data)


def test_parts():
    """Tokens are put at blocks' starts; other blocks keep what they hold, and the rest of
    a block that is only begun becomes zeros."""
    say("held parts")
    n, length, heads, d = 2, 150, 2, 40
    a, b = _randn((n, length, heads, d), F16, 1), _randn((n, 40, heads, d), F16, 2, 2.0)
    h = _held(a, -a)
    h.put(b.cuda(), 3 * b.cuda(), at=64)
    want = bo.held(a)
    part = torch.zeros(n, 64, heads, d, dtype=torch.float64)
    part[:, :40] = bo.held(b)
    want[:, 64:128] = part
    gk, gv = h.get()
    _equal(gk, want)
    part[:, :40] = bo.held(3 * b)
    want = bo.held(-a)
    want[:, 64:128] = part
    _equal(gv, want)
    for at, count in ((0, 1), (31, 2), (5, 100), (149, 1), (150, 0), (33, None)):
        k, v = h.get(at, count)
        end = length if count is None else at + count
        assert torch.equal(k, gk[:, at:end]) and torch.equal(v, gv[:, at:end])
    tail = h.put(b[:, :22].cuda(), b[:, :22].cuda(), at=128).get(128)[0]
    _equal(tail, bo.held(b[:, :22]))
    assert (isa.HeldStates(1, 40, 1, 8).get()[0] == 0).all()


def test_layouts():
    say("held layouts")
    n, length, heads, d = 2, 77, 3, 40
    k, v = _randn((n, length, heads, d), F16, 1), _randn((n, length, heads, d), F16, 2)
    want = _held(k, v).data
    packed = torch.zeros(n, length, 2, heads, d + 1, dtype=F16, device="cuda")     # heads at any element
    packed[:, :, 0, :, :d], packed[:, :, 1, :, :d] = k.cuda(), v.cuda()
    kk = packed[:, :, 0, :, :d]
    vv = torch.zeros(heads, n, length, d, dtype=F16, device="cuda")
    vv.copy_(v.permute(2, 0, 1, 3))
    h = isa.HeldStates(n, length, heads, d).put(kk, vv.permute(1, 2, 0, 3))
    assert torch.equal(h.data, want)
    one = k[:1].expand(n, -1, -1, -1)
    assert torch.equal(isa.HeldStates(n, length, heads, d).put(one.cuda()[:1].expand(n, -1, -1, -1), v.cuda()).data,
                       _held(one.contiguous(), v).data)
    ref_k, ref_v = h.get()
    out = torch.full((n, length + 2, 2, heads, d + 3), 9.0, dtype=F16, device="cuda")
    gk, gv = h.get(k_out=out[:, :length, 0, :, :d], v_out=vv.permute(1, 2, 0, 3))
    assert torch.equal(gk, ref_k) and torch.equal(gv, ref_v)
    assert (out[:, :, 1] == 9).all() and (out[:, length:] == 9).all() and (out[..., d:] == 9).all()


# ------------------------------------------------------------------- the attention
def _attend(n, lq, lk, hq, hkv, d, dtype, mask=None, lengths=None, scale=None, seed=0, spoil=True):
    q, k, v = _qkv(n, lq, lk, hq, hkv, d, dtype, seed)
    see = None
    if mask is not None or lengths is not None:
        see = torch.ones(n, lk, dtype=torch.bool)
        if mask is not None:
            see &= mask
        if lengths is not None:
            see &= torch.arange(lk)[None] < lengths[:, None]
        if spoil:      # what is held in masked places has no effect
            k[~see], v[~see] = float("inf"), float("nan")
    h = _held(k, v)
    out, lse = isa.held_attention(q.cuda(), h, None if mask is None else mask.cuda(),
                                  None if lengths is None else lengths.cuda(), scale, return_lse=True)
    hk, hv = (t.cpu() for t in h.get())
    _compare(out, lse, q, hk, hv, see, scale, "%d x %d over %d, %d/%d x %d" % (n, lq, lk, hq, hkv, d))
    return q, h, out, lse


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [8, 16, 32, 40, 64, 96, 104, 128, 160, 192, 200, 224, 256])
def test_heads(d, dtype):
    say("held attention heads", d, dtype)
    for lq, lk, hq, hkv in ((1, 333, 4, 2), (9, 100, 2, 1), (70, 150, 3, 3)):
        _attend(2, lq, lk, hq, hkv, d, dtype, seed=d)


@pytest.mark.parametrize("lk", [1, 2, 31, 32, 33, 64, 65, 127, 129, 511, 513, 1000, 5000])
def test_key_lengths(lk):
    say("held attention keys", lk)
    for lq in (1, 40):
        _attend(2, lq, lk, 4, 2, 64, F16, seed=lk)
        lengths = torch.tensor([lk // 2, lk], dtype=torch.int32)
        _attend(2, lq, lk, 4, 2, 64, F16, lengths=lengths, seed=lk)


@pytest.mark.parametrize("lq", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 100, 300])
def test_queries(lq):
    say("held attention queries", lq)
    for hq, hkv in ((1, 1), (4, 1), (6, 2)):
        _attend(2, lq, 200, hq, hkv, 64, BF16, seed=lq)


@pytest.mark.parametrize("lq", [1, 12, 150])
@pytest.mark.parametrize("share", [0.0, 0.02, 0.5, 0.97])
def test_masks(lq, share):
    say("held attention masks", lq, share)
    n, lk = 3, 700
    mask = torch.rand(n, lk, generator=torch.Generator().manual_seed(lq)) < share
    _attend(n, lq, lk, 4, 2, 96, F16, mask=mask)
    _attend(n, lq, lk, 4, 2, 96, F16, mask=mask, lengths=torch.tensor([lk, 333, 0], dtype=torch.int32))


@pytest.mark.parametrize("lq", [1, 200])
def test_no_visible_key(lq):
    """Zeros and -infinity, whatever the queries and the states hold."""
    say("held attention none", lq)
    q, k, v = _qkv(3, lq, 300, 2, 2, 64, F16)
    q[0, 0, 0, 0] = float("inf")
    k[1:], v[1:] = float("nan"), float("nan")
    h = _held(k, v)
    lengths = torch.tensor([0, 0, -5], dtype=torch.int32).cuda()
    out, lse = isa.held_attention(q.cuda(), h, key_lengths=lengths, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    empty = isa.HeldStates(3, 0, 2, 64)
    out, lse = isa.held_attention(q.cuda(), empty, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert isa.held_attention(q.cuda()[:, :0], h).shape == (3, 0, 2, 64)


@pytest.mark.parametrize("lq", [1, 33, 200])
def test_large_scores_and_scales(lq):
    say("held attention scales", lq)
    for scale in (0.0, 4.0, -1.0, 1e-3):
        _attend(1, lq, 400, 2, 1, 64, F16, scale=scale or None)
    q, k, v = _qkv(1, lq, 300, 2, 2, 64, F16)
    v[:, :32] *= 2.0 ** -12     # blocks of very different sizes, down to fp16's smallest numbers
    v[:, 32:64] *= 2.0 ** -20
    k[:, 64:96] *= 2.0 ** -14
    v[:, 96:128] *= 2.0 ** 13
    h = _held(k, v)
    out, lse = isa.held_attention(q.cuda(), h, return_lse=True)
    hk, hv = (t.cpu() for t in h.get())
    _compare(out, lse, q, hk, hv, None, None, "sizes")


def test_long_keys_and_splits():
    say("held attention long")
    for n, lq, lk, hq, hkv, d, dtype in ((1, 1, 40000, 8, 1, 128, BF16), (2, 3, 9000, 4, 2, 64, F16), (1, 1, 20001, 2, 2, 256, F16)):
        q, h, out, lse = _attend(n, lq, lk, hq, hkv, d, dtype)
        plan = isa.HeldAttention(q.cuda(), h)
        assert plan.info()["grid"][1] > 1 and plan.workspace_bytes > 0
        guard = torch.full((plan.workspace_bytes + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        got = plan.forward(q.cuda(), h, workspace=guard[:plan.workspace_bytes])
        assert torch.equal(got, out) and (guard[plan.workspace_bytes:] == 0x5A).all()


def test_every_visible_key_counts_once():
    """Queries of zeros weigh every key alike: the sum of marked values shows a key
    that was lost or taken twice."""
    say("held attention counts")
    for lq, lk in ((1, 4097), (20, 1000), (300, 777)):
        q = torch.zeros(1, lq, 1, 32, dtype=F16)
        k = torch.zeros(1, lk, 1, 32, dtype=F16)
        v = torch.zeros(1, lk, 1, 32, dtype=F16)
        for e in range(13):
            v[0, :, 0, e] = ((torch.arange(lk) >> e) & 1).half()
        h = _held(k, v)
        out, lse = isa.held_attention(q.cuda(), h, return_lse=True)
        assert (lse.cpu() - math.log(lk)).abs().max() < 1e-5
        counts = out.cpu().double()[0, :, 0] * lk
        want = bo.held(v)[0, :, 0].sum(0)
        assert ((counts - want).abs() <= want * 2.0 ** -10 + 1e-9).all()


def test_strides_of_queries():
    say("held attention strides")
    for lq in (3, 200):
        q, k, v = _qkv(2, lq, 150, 4, 2, 40, F16)
        h = _held(k, v)
        want = isa.held_attention(q.cuda(), h)
        wide = torch.zeros(2, lq, 8, 48, dtype=F16, device="cuda")
        wide[:, :, 2:6, :40] = q.cuda()
        big = torch.full((2, lq, 4, 56), 3.0, dtype=F16, device="cuda")
        plan = isa.HeldAttention(wide[:, :, 2:6, :40], h, big[..., :40])
        assert torch.equal(plan.forward(wide[:, :, 2:6, :40], h, big[..., :40]), want)
        assert (big[..., 40:] == 3).all()


@pytest.mark.parametrize("lq,lk", [(1, 9000), (1, 100), (200, 500)])
def test_in_a_graph_and_on_streams(lq, lk):
    say("held graph", lq, lk)
    q, k, v = (t.cuda() for t in _qkv(2, lq, lk, 4, 2, 64, BF16))
    h = isa.HeldStates(2, lk, 2, 64, dtype=BF16)
    plan, out = isa.HeldAttention(q, h), torch.empty_like(q)
    ws = plan.new_workspace()
    kg, vg = torch.empty_like(k), torch.empty_like(v)

    def step():
        h.put(k, v)
        plan.forward(q, h, out, workspace=ws)
        h.get(k_out=kg, v_out=vg)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        for t in (q, k, v):
            t.copy_(_randn(t.shape, BF16, 10 * seed + t.shape[1]))
        other = isa.HeldStates(2, lk, 2, 64, dtype=BF16).put(k, v)
        want = plan.forward(q, other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(h.data, other.data) and torch.equal(kg, other.get()[0])
    side = torch.cuda.Stream()
    out.zero_(), h.data.zero_(), kg.zero_()
    torch.cuda.synchronize()
    s = side.cuda_stream
    h.put(k, v, stream=s)
    plan.forward(q, h, out, workspace=ws, stream=s)
    h.get(k_out=kg, v_out=vg, stream=s)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(kg, other.get()[0])
