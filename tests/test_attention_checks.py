"""Argument checks of the attention entry points of the C ABI, on the CPU: calls
that a kernel could not answer are refused before any launch, so made-up
addresses are safe."""
import ctypes

import pytest

import image_stencil_amd as isa
from image_stencil_amd import _abi
from test_attention_host import INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE, _create, _desc, _tokens

A, B, POS = 0x100000, 0x900000, 0xF00000   # made-up addresses, far apart


@pytest.mark.parametrize("scale,status", [(2.5e38, INVALID), (-2.5e38, INVALID), (2.3e38, 0), (-2.3e38, 0),
                                          (1e-44, 0)])
def test_scale_times_log2e_is_finite(scale, status):
    """Scores are multiplied by scale * log2(e) in fp32: an infinite factor would
    turn scores of 0 into NaN."""
    st, plan = _create(_desc(scale=scale))
    assert st == status
    _abi.load().cross_attention_destroy(plan)


def _grid(**kw):
    st, plan = _create(_desc(**kw))
    if st != 0:
        return st
    info = _abi.conv2d_plan_info()
    assert _abi.load().cross_attention_get_plan_info(plan, ctypes.byref(info)) == 0
    _abi.load().cross_attention_destroy(plan)
    return info.grid_x * info.grid_y * info.block


@pytest.mark.parametrize("kw,fits", [
    (dict(n=2 ** 21, lq=1, lk=4, hq=8, hkv=8, d=64), False),           # own tiles, 256 threads: 2^32
    (dict(n=2 ** 21 - 1, lq=1, lk=4, hq=8, hkv=8, d=64), True),
    (dict(n=2 ** 21, lq=1, lk=4, hq=16, hkv=16, d=8), False),          # windows with one query each
    (dict(n=2 ** 21, lq=1, lk=4, hq=8, hkv=8, d=160), True),           # 128 threads
    (dict(n=2 ** 22, lq=1, lk=4, hq=8, hkv=8, d=160), False),
    (dict(n=2 ** 21, lq=128, lk=1000, hq=8, hkv=8, d=64), False),      # shared tiles
    (dict(n=8, lq=2 ** 26, lk=10000, hq=8, hkv=8, d=64), False),
    (dict(n=8, lq=2 ** 26, lk=64, hq=8, hkv=8, d=64), True)])          # the same rows with the keys kept
def test_plans_fit_a_launch(kw, fits):
    """A launch counts its threads in 32 bits: a plan that needs more is refused
    when it is made, not when it runs."""
    threads = _grid(**kw)
    if fits:
        assert 256 < threads < 2 ** 32
    else:
        assert threads == UNSUPPORTED


def test_rotary_calls_fit_a_launch():
    lib, plan = _abi.load(), isa.Rotary(64)
    far = 1 << 45
    for length, heads in ((2 ** 30, 1), (2 ** 31 - 1, 1), (2 ** 30, 4)):
        t = _tokens(n=1, length=length, heads=heads)
        assert lib.rotary_forward(plan.handle, _abi.IS_F16, t, A, far, 0, t, far * 2, None) == UNSUPPORTED
        d = _abi.qk_norm_desc(_abi.IS_F16, _abi.IS_NORM_RMS, 1e-6, _tokens(), t, _tokens(), t, 0, 0)
        assert lib.qk_norm_rotary_forward(plan.handle, ctypes.byref(d), A, far, None, None, POS, 3 * far, B, 2 * far,
                                          None) == UNSUPPORTED
