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
