"""Cross attention in the LDS-poison debug build: LDS that is read before it was
written (a missing wait or barrier, rows that no load covers) would put NaN into
the results; they must be the release build's bits."""
import pytest
import torch

import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _qkv
from test_gpu_lds_poison import _poison_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,lq,lk,hq,hkv,d", [(2, 300, 333, 2, 2, 64), (2, 300, 333, 2, 1, 128), (1, 150, 1000, 1, 1, 40),
                                              (1, 1, 700, 4, 1, 96), (1, 5, 9000, 2, 2, 256), (4, 4000, 77, 8, 8, 40),
                                              (1, 200, 200, 1, 1, 160), (3, 2, 33, 2, 2, 32)])
def test_attention_in_the_poison_build(n, lq, lk, hq, hkv, d):
    say("attention poison", n, lq, lk, d)
    q, k, v = (t.cuda() for t in _qkv(n, lq, lk, hq, hkv, d, torch.float16, lk))
    mask = (torch.rand(n, lk, generator=torch.Generator().manual_seed(lk)) < 0.5).cuda()
    lengths = torch.tensor([lk, lk // 2, 1, 0][:n], dtype=torch.int32, device="cuda")
    plan, poisoned = isa.CrossAttention(q, k, v), isa.CrossAttention(q, k, v)
    poisoned._lib = _poison_lib()
    for kw in ({}, {"key_mask": mask}, {"key_lengths": lengths}):
        want, got = plan.forward(q, k, v, **kw), poisoned.forward(q, k, v, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got, want), kw
