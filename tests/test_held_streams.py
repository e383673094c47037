"""Held states and streams other than the one they were made on."""
import types

import pytest
import torch

import image_stencil_amd as isa
from gpu_util import say
from test_attention_binding import fake, gpu  # noqa: F401
from test_gpu_cross_attention import _randn

F16 = torch.float16


@pytest.mark.parametrize("capturing", [False, True])
def test_a_new_store_is_cleared_before_the_constructor_returns(fake, monkeypatch, capturing):  # noqa: F811
    """Zeros still on their way could land after what a put on another stream writes. (A
    capture cannot wait: there they are the graph's.)"""
    steps, zeros = [], torch.zeros
    stream = types.SimpleNamespace(synchronize=lambda: steps.append(("wait", fake["current"])))

    def cleared(*size, device=None, **kw):
        steps.append("zeros")
        return gpu(zeros(*size, **kw), 1)
    monkeypatch.setattr(torch, "zeros", cleared)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *index: stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    isa.HeldStates(2, 40, 1, 8, device="cuda:1")
    assert steps == ["zeros"] if capturing else steps == ["zeros", ("wait", 1)]


@pytest.mark.gpu
def test_a_put_on_another_stream_stays():
    """The store is made behind long work of its stream, and put to on another at once."""
    say("held, another stream")
    k, v = _randn((2, 300, 2, 64), F16, 1).cuda(), _randn((2, 300, 2, 64), F16, 2).cuda()
    want = isa.HeldStates(2, 300, 2, 64).put(k, v).data
    big = torch.zeros(8192, 8192, dtype=F16, device="cuda")
    torch.cuda.synchronize()
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(first):
        for _ in range(10):
            big = big @ big
        states = isa.HeldStates(2, 300, 2, 64)
        states.put(k, v, stream=second.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(states.data, want)
