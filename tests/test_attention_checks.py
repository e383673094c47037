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
