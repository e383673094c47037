"""The attention kernels' forms at the sizes where they change: keys kept for
several row tiles, rings of two and four buffers with masks over one to many
tiles, own and shared key tiles, splits; rotary heads whose parts end in a chunk
that reaches back, in place, next to infinities; and the example that runs the
operators together."""
import math
import os
import sys

import pytest
import torch

import attention_oracle as ao
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _compare, _qkv, _run
from test_gpu_rotary import _positions, _randn

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("d,lk", [(24, 200), (40, 77), (64, 256), (96, 128), (128, 65), (128, 1)])
def test_keys_kept_for_several_row_tiles(d, lk):
    n, lq, hq, hkv = 4, 4000, 8, 8
    say("kept", d, lk)
    q, k, v = _qkv(n, lq, lk, hq, hkv, d, F16, d)
    info = isa.CrossAttention(q, k, v).info()
    assert info["grid"][0] < n * hkv * ((lq + 127) // 128), info    # fewer workgroups than row tiles
    _run(q, k, v, label="whole")
    _run(q, k, v, lengths=torch.tensor([lk, lk // 2, 1, 0], dtype=torch.int32), label="lengths")
    mask = torch.rand(n, lk, generator=torch.Generator().manual_seed(d)) < 0.6
    mask[1] = False
    _run(q, k, v, mask, label="mask")


@pytest.mark.parametrize("d", [32, 64, 96, 160])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6, 7, 9])
def test_masks_over_every_number_of_tiles(d, tiles):
    """Shared tiles of 64 keys and own tiles of 32, ends before, at and after a
    tile's; mask rows that start at every byte of a word (odd lengths)."""
    for lk in (64 * tiles - 1, 64 * tiles, 64 * tiles + 1):
        say("tiles", d, lk)
        g = torch.Generator().manual_seed(lk + d)
        for lq in (3, 300):
            q, k, v = _qkv(3, lq, lk, 2, 1, d, BF16, lk)
            _run(q, k, v, torch.rand(3, lk, generator=g) < 0.5, label="mask")
    _run(q, k, v, lengths=torch.tensor([lk, 32, 64], dtype=torch.int32), label="lengths")


def test_masked_splits_hold_nothing_of_masked_keys():
    """Splits and own tiles whose keys are all masked, infinities among them."""
    n, lk, d = 1, 12000, 64
    for lq in (1, 20, 300):
        q, k, v = _qkv(n, lq, lk, 2, 2, d, F16, lq)
        mask = torch.zeros(n, lk, dtype=torch.bool)
        mask[:, 5000:5003] = True
        kb, vb = k.clone(), v.clone()
        kb[:, ~mask[0]], vb[:, ~mask[0]] = math.nan, math.inf
        assert isa.CrossAttention(q, k, v).info()["grid"][1] > 1
        out = isa.cross_attention(q.cuda(), kb.cuda(), vb.cuda(), mask.cuda())
        _compare(out, None, q, k, v, mask, label="splits %d" % lq)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("d,rot", [(20, 20), (44, 44), (100, 50), (250, 246), (60, 36), (36, 18)])
def test_half_layout_in_place_where_chunks_overlap(dtype, d, rot):
    """The halves and the rest end in chunks that reach back over their
    neighbour's elements: in place gives the bits of a new tensor."""
    say("overlap", dtype, d, rot)
    x = _randn((2, 33, 5, d), dtype, d).cuda()
    pos = _positions(2, 33, 1, d).cuda()
    plan = isa.Rotary(d, rot)
    want = plan.apply(x, pos)
    w = (1 + 0.1 * _randn((d,), F32, 3)).cuda()
    wq, wk = plan.apply_qk_norm(x, x[:, :, :2], pos, q_weight=w, k_weight=w)
    y = x.clone()
    assert plan.apply(y, pos, out=y) is y and torch.equal(y, want)
    y = x.clone()
    k = x[:, :, :2].clone()
    plan.apply_qk_norm(y, k, pos, q_weight=w, k_weight=w, q_out=y, k_out=k)
    assert torch.equal(y, wq) and torch.equal(k, wk)
    assert torch.equal(wq[:, :, :2], wk)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_what_passes_through_ignores_its_neighbours(layout, bad):
    """Infinities and NaN in elements that do not turn stay where they are."""
    x = _randn((1, 9, 3, 64), F16, 5)
    plan, pos = isa.Rotary(64, 24, layout=layout), _positions(1, 9, 1, 6).cuda()
    want = plan.apply(x.cuda(), pos).cpu()
    y = x.clone()
    y[..., 30::7] = bad
    got = plan.apply(y.cuda(), pos).cpu()
    hit = torch.zeros(64, dtype=torch.bool)
    hit[30::7] = True
    assert torch.equal(got[..., ~hit], want[..., ~hit])
    assert torch.equal(torch.nan_to_num(got[..., hit], 7.0), torch.nan_to_num(y[..., hit], 7.0))


def test_example_attends_like_the_formulas():
    """examples/attend_reference.py: its attention step against the 64-bit forms
    on the features and projections that the block computed."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import attend_reference as ex
    sizes = (20, 24, 13, 17)
    block = ex.AttendReference(ex.weights(), *sizes)
    g = torch.Generator().manual_seed(3)
    frame, ref = (torch.rand((2, h, w), generator=g).half().cuda() for h, w in (sizes[:2], sizes[2:]))
    f, r = block.features(frame), block.features(ref)
    d = ex.CHANNELS // ex.HEADS
    q = (f.reshape(2, -1, ex.CHANNELS) @ block.w["q"]).view(2, -1, ex.HEADS, d)
    kv = (r.reshape(2, -1, ex.CHANNELS) @ block.w["kv"]).view(2, -1, 2, ex.HEADS, d)
    freqs, turned, bounds = ao.frequencies(d, 2), [], []
    for x, at in ((q, block.at), (kv[:, :, 0], block.at_ref)):
        z, size = ao.norm(x.cpu().double(), torch.ones(d).double(), 1e-6, "rms")
        want, _ = ao.rotate(z, at.cpu().expand(2, -1, -1), d, 2, "half", freqs)
        _, m = ao.rotate(size, at.cpu().expand(2, -1, -1), d, 2, "half", freqs)
        bounds.append(ao.rotary_bound(want, m, F16) + ao.norm_error(d, "rms") * (1 + ao.half(F16)) * m)
        turned.append(want)
    yq, yk = block.rotary.apply_qk_norm(q, kv[:, :, 0], block.at, block.at_ref, block.w["q_norm"], block.w["k_norm"])
    for got, want, bound in zip((yq, yk), turned, bounds):
        assert ((got.cpu().double() - want).abs() <= bound).all()
    out = isa.cross_attention(yq, yk, kv[:, :, 1])
    _compare(out, None, yq.cpu(), yk.cpu(), kv[:, :, 1].cpu(), label="example")
    assert torch.equal(block.attend(f, r), f + out.view_as(f))
    y = block(frame, ref)
    assert y.shape == (2, *sizes[:2], ex.CHANNELS) and torch.isfinite(y.float()).all()
