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
