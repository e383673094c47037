"""Attention operators on the GPU where inputs are unusual: single keys with any
stride, entries without a key under infinite queries, infinities and NaN that are
seen, streams and threads, guarded workspaces."""
import math

import pytest
import torch

import attention_oracle as ao
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _compare, _qkv

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("stride", [0, 8, 2 ** 31 - 1, 2 ** 32 // 126 + 1, 2 ** 33 // 126, 2 ** 40 + 4])
@pytest.mark.parametrize("lq", [1, 40, 200])
def test_the_token_stride_of_a_single_key_does_not_matter(lq, stride):
    say("one key", lq, stride)
    q, k, v = _qkv(2, lq, 1, 2, 2, 64, F16, lq)
    ks, vs = (t.cuda().as_strided((2, 1, 2, 64), (128, stride, 64, 1)) for t in (k, v))
    mask = torch.tensor([[True], [False]])
    assert torch.equal(isa.cross_attention(q.cuda(), ks, vs), v.cuda().expand(2, lq, 2, 64))
    out, lse = isa.cross_attention(q.cuda(), ks, vs, mask.cuda(), return_lse=True)
    _compare(out, lse, q, k, v, mask, label="one key")


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("n,lq,lk,hq,hkv,d", [(3, 1, 70, 4, 2, 64), (3, 1, 20000, 4, 2, 64), (3, 40, 300, 2, 2, 40),
                                              (3, 200, 333, 2, 2, 64), (3, 200, 333, 2, 1, 128), (2, 3, 700, 1, 1, 256),
                                              (4, 4000, 77, 8, 8, 40), (1, 300, 12000, 2, 2, 64)])
def test_no_visible_key_gives_zeros_whatever_q_holds(bad, n, lq, lk, hq, hkv, d):
    """An entry that is padding as a whole: its queries may be anything, and its
    rows are still zeros with lse = -infinity. The other entries keep their bits."""
    say("empty", bad, n, lq, lk, d)
    q, k, v = (t.cuda() for t in _qkv(n, lq, lk, hq, hkv, d, F16, lk))
    mask = torch.rand(n, lk, generator=torch.Generator().manual_seed(d)) < 0.5
    mask[0] = False
    mask = mask.cuda()
    want, want_lse = isa.cross_attention(q, k, v, mask, return_lse=True)
    q[0, :, :, ::3] = bad
    out, lse = isa.cross_attention(q, k, v, mask, return_lse=True)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    lengths = torch.full((n,), lk, dtype=torch.int32, device="cuda")
    lengths[0] = 0
    out = isa.cross_attention(q, k, v, key_lengths=lengths)
    assert (out[0] == 0).all()


FORMS = [(1, 70, 64), (1, 20000, 64), (40, 300, 40), (200, 333, 64), (200, 333, 128), (3, 700, 256)]   # lq, lk, d


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("lq,lk,d", FORMS)
def test_a_query_that_is_no_number_spoils_its_row_alone(bad, lq, lk, d):
    """The other rows stay within their bounds (not to the bit: when one row's
    running maximum moves, those of its wave move with it)."""
    q, k, v = _qkv(2, lq, lk, 4, 2, d, F16, lk)
    mask = torch.rand(2, lk, generator=torch.Generator().manual_seed(d)) < 0.5
    for see in (None, mask):
        p = q.clone()
        p[1, lq // 2, 3, 5] = math.nan if math.isnan(bad) else bad
        p[1, lq // 2, 3, 6] = -p[1, lq // 2, 3, 5]
        args = (k.cuda(), v.cuda(), None if see is None else see.cuda())
        out, lse = isa.cross_attention(p.cuda(), *args, return_lse=True)
        assert torch.isnan(out[1, lq // 2, 3]).all() and torch.isnan(lse[1, 3, lq // 2])
        want, want_lse = isa.cross_attention(q.cuda(), *args, return_lse=True)
        out[1, lq // 2, 3], lse[1, 3, lq // 2] = want[1, lq // 2, 3], want_lse[1, 3, lq // 2]
        _compare(out, lse, q, k, v, see, label="other rows")


@pytest.mark.parametrize("lq,lk,d", FORMS)
def test_a_visible_key_that_is_no_number_spoils_its_entry_and_head(lq, lk, d):
    q, k, v = (t.cuda() for t in _qkv(2, lq, lk, 4, 2, d, F16, lk))
    want = isa.cross_attention(q, k, v)
    for at in (0, lk // 2, lk - 1):
        p = k.clone()
        p[0, at, 1, d - 1] = math.nan
        out = isa.cross_attention(q, p, v)
        assert torch.isnan(out[0, :, 2:]).all()
        assert torch.equal(out[0, :, :2], want[0, :, :2]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("lq,lk,d", FORMS)
def test_a_visible_value_that_is_no_number_reaches_its_element_alone(bad, lq, lk, d):
    q, k, v = (t.cuda() for t in _qkv(2, lq, lk, 4, 2, d, F16, lk, qscale=0.2))
    want = isa.cross_attention(q, k, v)
    p = v.clone()
    p[1, lk // 3, 0, 7] = bad
    out = isa.cross_attention(q, k, p)
    assert (torch.isnan(out[1, :, :2, 7]) if math.isnan(bad) else out[1, :, :2, 7] == bad).all()
    out[1, :, :2, 7] = want[1, :, :2, 7]
    assert torch.equal(out, want)


@pytest.mark.parametrize("lq,lk,d", FORMS)
def test_scores_of_minus_infinity_drop_their_keys(lq, lk, d):
    """A bias folded into the keys: positive queries and an element of -infinity
    leave a key out as a mask does, whole tiles at the start and the end too."""
    q, k, v = _qkv(2, lq, lk, 4, 2, d, F16, lk)
    q = q.abs() + 2.0 ** -10
    see = torch.rand(2, lk, generator=torch.Generator().manual_seed(d)) < 0.5
    see[0, :2 * lk // 3] = False
    see[0, -1] = True
    see[1, lk // 3:] = False
    see[1, 0] = True
    p = k.clone()
    p[..., d - 1][~see] = -math.inf
    out, lse = isa.cross_attention(q.cuda(), p.cuda(), v.cuda(), return_lse=True)
    _compare(out, lse, q, k, v, see, label="-inf scores")


@pytest.mark.parametrize("lq,lk", [(1, 20000), (40, 9001), (130, 9001)])
def test_nothing_is_written_past_the_workspace(lq, lk):
    """A plan that splits its keys, in a workspace of just its size amid other
    memory; the part of it that the join reads was written by this call."""
    q, k, v = (t.cuda() for t in _qkv(1, lq, lk, 2, 1, 64, F16, lq))
    plan = isa.CrossAttention(q, k, v)
    need, pad = plan.workspace_bytes, 1 << 20
    assert need > 0 and need % 4 == 0
    want = plan.forward(q, k, v)
    for fill in (0, 255, 0x7f):
        room = torch.full((need + 2 * pad,), fill, dtype=torch.uint8, device="cuda")
        out = plan.forward(q, k, v, workspace=room[pad:pad + need])
        assert torch.equal(out, want)
        assert (room[:pad] == fill).all() and (room[pad + need:] == fill).all()


def test_calls_on_streams_given_as_numbers():
    """stream= of every call, with work of its own queued before and after on it."""
    q, k, v = (t.cuda() for t in _qkv(2, 300, 500, 4, 2, 64, F16))
    pos, pos_k = (torch.arange(n, dtype=torch.int32, device="cuda")[None, :, None] for n in (300, 500))
    rot = isa.Rotary(64)
    want_r = rot.apply(q, pos)
    want_q, want_k = rot.apply_qk_norm(q, k, pos, pos_k)
    plan = isa.CrossAttention(q, k, v)
    want = plan.forward(want_q, want_k, v)
    side = torch.cuda.Stream()
    r, yq, yk, out = (torch.empty_like(t) for t in (q, q, k, q))
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for t in (r, yq, yk, out):
                t.fill_(7)
        assert rot.apply(q, pos, out=r, stream=side.cuda_stream) is r
        rot.apply_qk_norm(q, k, pos, pos_k, q_out=yq, k_out=yk, stream=side.cuda_stream)
        plan.forward(yq, yk, v, out, workspace=plan.new_workspace(), stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(r, want_r) and torch.equal(yq, want_q) and torch.equal(yk, want_k)
        assert torch.equal(out, want)


def test_threads_and_streams_share_plans():
    """Two threads, each with a stream and a workspace, on one plan of each kind."""
    import threading
    q, k, v = (t.cuda() for t in _qkv(2, 3, 9000, 4, 2, 64, F16))
    pos = torch.arange(3, dtype=torch.int32, device="cuda")[None, :, None]
    plan, rot = isa.CrossAttention(q, k, v), isa.Rotary(64)
    want, want_r = plan.forward(q, k, v), rot.apply(q, pos)
    torch.cuda.synchronize()
    results, failures = [], []

    def work(seed):
        try:
            stream, ws = torch.cuda.Stream(), plan.new_workspace()
            stream.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(stream):
                for _ in range(20):
                    results.append((plan.forward(q, k, v, workspace=ws), rot.apply(q, pos)))
            stream.synchronize()
        except Exception as e:      # shown by the test's thread
            failures.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    assert len(results) == 40
    for out, r in results:
        assert torch.equal(out, want) and torch.equal(r, want_r)


@pytest.mark.parametrize("dtype", [torch.float32, F16, BF16])
@pytest.mark.parametrize("d,rot", [(64, 64), (40, 24), (20, 20), (7, 4)])
def test_rotary_bases_at_every_16_bytes(dtype, d, rot):
    """Bases 16, 32 and 48 bytes into memory, in and out apart and in place, give
    the bits of an aligned tensor; what lies around stays."""
    n, length, heads = 2, 33, 3
    size = torch.finfo(dtype).bits // 8
    x = torch.randn(n, length, heads, d, generator=torch.Generator().manual_seed(d)).to(dtype).cuda()
    pos = torch.arange(length, dtype=torch.int32, device="cuda")[None, :, None]
    plan = isa.Rotary(d, rot)
    want = plan.apply(x, pos)
    for off in (16 // size, 32 // size, 48 // size):
        mem = torch.full((x.numel() + 2 * off + 64,), 7.0, dtype=dtype, device="cuda")
        y = mem[off:off + x.numel()].view(x.shape)
        y.copy_(x)
        assert torch.equal(plan.apply(y, pos), want)
        assert torch.equal(plan.apply(y, pos, out=y), want)
        out = mem.clone()[off:off + x.numel()].view(x.shape)
        assert torch.equal(plan.apply(x, pos, out=out), want)
        assert (mem[:off] == 7).all() and (mem[off + x.numel():] == 7).all()
    shifted = torch.zeros(x.numel() + 64, dtype=dtype, device="cuda")[1:1 + x.numel()].view(x.shape)
    with pytest.raises(isa.ImgStencilError):
        plan.apply(shifted, pos)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("size", [1e-15, 1e-19, 1e-20, 1e-21])
def test_norms_of_small_heads_without_eps(dtype, kind, size):
    """eps 0 and heads whose mean square is below fp32's normal numbers: what 32 bits
    hold of it (steps of 2^-149: squares, their sum and mean are off by half a step
    each) still gives a norm. A head of zeros has none."""
    d = 64
    x = (size * torch.randn(1, 5, 3, d, generator=torch.Generator().manual_seed(7))).to(dtype)
    pos = torch.zeros(1, 5, 1, dtype=torch.int32, device="cuda")
    y, _ = isa.Rotary(d, 0).apply_qk_norm(x.cuda(), x[:, :, :1].cuda(), pos, eps=0.0, norm=kind)
    want, scale = ao.norm(x.double(), torch.ones(d).double(), 0.0, kind)
    centred = x.double() - (x.double().mean(-1, keepdim=True) if kind == "layer" else 0.0)
    mean = (centred * centred).mean(-1, keepdim=True)
    steps = 0.5 * 3 * 2.0 ** -150 / mean
    bound = ao.rounding(want, dtype) + (1 + ao.half(dtype)) * (ao.norm_error(d, kind) + steps) * scale
    assert ((y.cpu().double() - want).abs() <= bound).all()
    z, _ = isa.Rotary(d, 0).apply_qk_norm(torch.zeros_like(x).cuda(), x[:, :, :1].cuda(), pos, eps=0.0, norm=kind)
    assert torch.isnan(z).all()
