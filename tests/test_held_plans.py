"""Which form an attention to held states takes (host only), and what a plan that loads
the states first refuses."""
import ctypes

import pytest

from image_stencil_amd import _abi
from test_attention_host import INVALID, MISALIGNED, WORKSPACE
from test_blocks_host import _attend, _size

LOADED, DIRECT = b"is_k14_held_load, is_k11_attention", b"is_k15_held_attention"


def _kernel(plan):
    info = _abi.conv2d_plan_info()
    assert _abi.load().held_attention_get_plan_info(plan, ctypes.byref(info)) == 0
    return info.kernel


@pytest.mark.parametrize("d,lq,kernel", [(40, 4096, DIRECT), (40, 4097, LOADED), (128, 4096, DIRECT), (128, 4097, LOADED),
                                         (136, 2048, DIRECT), (136, 2049, LOADED)])
def test_row_tiles_choose_the_form(d, lq, kernel):
    """2 entries x 2 key heads, two query heads each: 1024 row tiles of 32, or 512, are the
    most that read the held bytes directly."""
    st, plan = _attend(d=d, lq=lq)
    assert st == 0 and _kernel(plan) == kernel
    _abi.load().held_attention_destroy(plan)


def test_forward_refusals_where_the_states_are_loaded_first():
    lib = _abi.load()
    _, plan = _attend(lq=5000, length=4000, mb=4000)
    assert _kernel(plan) == LOADED
    size, need = _size(length=4000, heads=2)[1], ctypes.c_size_t()
    assert lib.held_attention_workspace_size(plan, ctypes.byref(need)) == 0
    assert need.value >= 2 * 2 * 4000 * 2 * 40 * 2
    far = 1 << 40

    def st(q=far, held=2 * far, bytes_=size, mask=None, lengths=None, out=3 * far, lse=None, ws=4 * far, wb=need.value):
        return lib.held_attention_forward(plan, q, held, bytes_, mask, lengths, out, lse, ws, wb, None)

    assert st(q=None) == INVALID and st(held=None) == INVALID and st(out=None) == INVALID
    assert st(bytes_=size - 1) == WORKSPACE and st(ws=None) == WORKSPACE and st(wb=need.value - 1) == WORKSPACE
    assert st(q=far + 8) == MISALIGNED and st(held=far + 8) == MISALIGNED and st(ws=far + 8) == MISALIGNED
    assert st(lse=far + 2) == MISALIGNED and st(lengths=far + 2) == MISALIGNED
    assert st(out=far) == INVALID and st(out=2 * far + 64) == INVALID and st(ws=2 * far) == INVALID
    assert st(lse=3 * far) == INVALID and st(ws=far) == INVALID and st(mask=3 * far) == INVALID
    lib.held_attention_destroy(plan)
