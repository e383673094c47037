"""The operators around attention in the LDS-poison debug build: LDS that is read before
it was written would put NaN into the results; they must be the release build's bits."""
import pytest
import torch

import image_stencil_amd as isa
from gpu_util import say
from test_gpu_block_norm import _case as norm_case
from test_gpu_cross_attention import _qkv, _randn
from test_gpu_dense import _case as dense_case
from test_gpu_lds_poison import _poison_lib

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("c", [100, 1000, 2000, 4000, 8000, 16000])
def test_norm(c):
    say("norm poison", c)
    x, kw = norm_case(2, 5, c, BF16, "layer", "layer", seed=c)
    kw.pop("residual_scale")
    dev = {k: v.cuda() for k, v in kw.items()}
    plan, poisoned = isa.BlockNorm(c, "layer", "layer"), isa.BlockNorm(c, "layer", "layer")
    poisoned._lib = _poison_lib()
    for a, b in zip(plan.apply(x.cuda(), **dev), poisoned.apply(x.cuda(), **dev)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,k,m", [(1, 200, 300), (20, 1000, 77), (40, 8192, 64), (300, 344, 130), (1000, 1024, 1000),
                                      (2000, 264, 2048), (5000, 520, 1300), (8000, 128, 2050)])
def test_dense(rows, k, m):
    x, w, b, r = (t.cuda() for t in dense_case(1, rows, k, m, F16))
    plan, poisoned = (isa.Dense(x, w, residual=r, activation="gelu") for _ in range(2))
    say("dense poison", rows, k, m, plan.info()["kernel"], plan.info()["tile"], plan.info()["grid"])
    poisoned._lib = _poison_lib()
    assert torch.equal(plan.forward(x, w, b, r), poisoned.forward(x, w, b, r))


@pytest.mark.parametrize("n,lq,lk,hq,hkv,d", [(2, 1, 700, 4, 2, 64), (1, 40, 333, 2, 1, 128), (1, 3, 5000, 2, 2, 256),
                                              (3, 2, 33, 2, 2, 32), (1, 9000, 100, 8, 8, 40)])
def test_held(n, lq, lk, hq, hkv, d):
    say("held poison", lq, lk, d)
    q, k, v = (t.cuda() for t in _qkv(n, lq, lk, hq, hkv, d, F16))
    lengths = torch.tensor([lk, lk // 2, 0][:n], dtype=torch.int32, device="cuda")
    mask = (_randn((n, lk), torch.float32, 5) < 0.3).cuda()
    held, poisoned = isa.HeldStates(n, lk, hkv, d), isa.HeldStates(n, lk, hkv, d)
    poisoned._lib = _poison_lib()
    held.put(k, v, key_lengths=lengths), poisoned.put(k, v, key_lengths=lengths)
    assert torch.equal(held.data, poisoned.data)
    for a, b in zip(held.get(), poisoned.get()):
        assert torch.equal(a, b)
    plan, other = isa.HeldAttention(q, held), isa.HeldAttention(q, held)
    other._lib = _poison_lib()
    for kw in ({}, {"key_mask": mask}, {"key_lengths": lengths}):
        assert torch.equal(plan.forward(q, held, **kw), other.forward(q, held, **kw)), kw
