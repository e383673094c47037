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


def test_qk_norm_refuses_outputs_over_the_other_tensor():
    """Queries and keys run in one launch, in no order: what one of them writes must
    not be what the other still reads (its elements, weights or positions) or
    writes."""
    lib, plan = _abi.load(), isa.Rotary(64)
    Q, K, QO, KO = 0x100000, 0x400000, 0x900000, 0xC00000
    WQ, WK, PQ, PK = 0x1000, 0x2000, 0xE00000, 0xF00000

    def st(q=Q, k=K, wq=WQ, wk=WK, qo=QO, ko=KO, qp=PQ, kp=PK, tokens=None):
        tq, tk, tqo, tko = tokens or (_tokens(), _tokens(heads=2), _tokens(), _tokens(heads=2))
        d = _abi.qk_norm_desc(_abi.IS_BF16, _abi.IS_NORM_RMS, 1e-6, tq, tk, tqo, tko, 0, 0)
        return lib.qk_norm_rotary_forward(plan.handle, ctypes.byref(d), q, k, wq, wk, qp, kp, qo, ko, None)

    assert st(qo=K) == INVALID and st(ko=Q) == INVALID and st(qo=K, ko=Q) == INVALID
    assert st(qo=K + 64) == INVALID and st(ko=Q + 64) == INVALID      # dense tensors over each other
    assert st(qo=K - 64) == INVALID and st(ko=QO + 128) == INVALID
    assert st(qo=WK - 32) == INVALID and st(ko=WQ - 32) == INVALID    # weights
    assert st(qo=PK - 16) == INVALID and st(ko=PQ - 16) == INVALID    # positions
    # a wide q_out whose row holds the start of a dense k
    wide = _tokens(token_stride=4 * 64 * 3, batch_stride=3 * 4 * 64 * 3)
    assert st(qo=K, tokens=(_tokens(), _tokens(heads=2), wide, _tokens(heads=2))) == INVALID
    # Slices of one packed projection, in place or into another one, lie between
    # each other: such a call gets past these checks, to the one for its size.
    far, n4 = 1 << 44, 4 * 64
    for token, batch, k_at in ((8 * 64, 0, n4 * 2),                          # heads of a token together
                               (64, 8 * 64 * 2 ** 30, n4 * 2 ** 30 * 2),     # tokens of a head together
                               (16 * 64, 0, 64 * 2)):                        # heads of q and k in turn
        head = {64: 64 * 2 ** 30}.get(token, 64 if token == 8 * 64 else 128)
        t4, t2 = (_tokens(n=1, length=2 ** 30, heads=h, token_stride=token, head_stride=head, batch_stride=batch)
                  for h in (4, 2))
        huge = (t4, t2, t4, t2)
        at = 1 << 40
        assert st(q=at, k=at + k_at, qo=at, ko=at + k_at, tokens=huge) == UNSUPPORTED, token
        assert st(q=at, k=at + k_at, qo=far, ko=far + k_at, tokens=huge) == UNSUPPORTED, token
        assert st(q=at, k=at + k_at, qo=at + k_at, ko=far, tokens=huge) == INVALID, token
    # a tensor without elements overlaps nothing
    none = _tokens(length=0)
    t = _tokens(n=1, length=2 ** 30)
    assert st(q=1 << 40, qo=1 << 40, k=1 << 40, ko=1 << 40, tokens=(t, none, t, none)) == UNSUPPORTED


def test_strides_of_single_steps_do_not_matter_in_place():
    """The stride of a dimension of one element says nothing: x and y at one base
    that differ only there are the same tensor (the call gets to the check of its
    size)."""
    lib, plan = _abi.load(), isa.Rotary(64)
    x = _tokens(n=1, length=2 ** 30, heads=1)
    for kw in ({"batch_stride": 5}, {"head_stride": 1 << 40}, {"batch_stride": 0, "head_stride": 0}):
        y = _tokens(n=1, length=2 ** 30, heads=1, **kw)
        assert lib.rotary_forward(plan.handle, _abi.IS_F16, x, 1 << 40, POS, 0, y, 1 << 40, None) == UNSUPPORTED, kw
    y = _tokens(n=1, length=2 ** 30, heads=1, token_stride=128)
    assert lib.rotary_forward(plan.handle, _abi.IS_F16, x, 1 << 40, POS, 0, y, 1 << 40, None) == INVALID


# --------------------------------------------------- plans that split their keys
SPLIT = dict(n=1, lq=1, lk=40000, hq=8, hkv=1, d=128)


def _need(plan):
    need = ctypes.c_size_t()
    assert _abi.load().cross_attention_workspace_size(plan, ctypes.byref(need)) == 0
    return need.value


@pytest.mark.parametrize("kw", [SPLIT, dict(n=3, lq=2, lk=9001, hq=4, hkv=4, d=64), dict(n=1, lq=3, lk=20011, hq=2, hkv=2, d=256),
                                dict(n=1, lq=130, lk=9001, hq=1, hkv=1, d=40)])
def test_split_plans_cover_the_keys_and_their_workspace_the_parts(kw):
    """Every key lies in one split, no split is empty, and the workspace holds a
    row of d values and a log-sum for every row of every row tile and split."""
    st, plan = _create(_desc(**kw))
    assert st == 0
    info = _abi.conv2d_plan_info()
    assert _abi.load().cross_attention_get_plan_info(plan, ctypes.byref(info)) == 0
    splits, keys, rows = info.grid_y, info.tile_w, info.tile_h
    own = b"own" in info.kernel
    assert splits > 1 and keys % (32 if own else 64) == 0 and rows == (32 if own else 128)
    assert (splits - 1) * keys < kw["lk"] <= splits * keys
    tiles = -(-kw["lq"] * (kw["hq"] // kw["hkv"]) // rows)
    assert info.grid_x == kw["n"] * kw["hkv"] * tiles
    assert _need(plan) == info.grid_x * splits * rows * (kw["d"] + 1) * 4
    _abi.load().cross_attention_destroy(plan)


def test_plans_without_splits_need_no_workspace():
    for kw in ({}, dict(lq=16384, lk=16384, hq=16, hkv=4, d=128, n=1), dict(n=8, lq=4096, lk=120, hq=8, hkv=8, d=40)):
        st, plan = _create(_desc(**kw))
        assert st == 0 and _need(plan) == 0
        _abi.load().cross_attention_destroy(plan)


def test_workspaces_that_do_not_serve_are_refused():
    lib = _abi.load()
    st, plan = _create(_desc(**SPLIT))
    assert st == 0
    need = _need(plan)
    Q, K, V, OUT, LSE, MASK, LEN, WS = (i << 28 for i in range(1, 9))
    assert need < 1 << 28

    def forward(ws=WS, ws_bytes=need, lse=None, mask=None, lengths=None):
        return lib.cross_attention_forward(plan, Q, K, V, mask, lengths, OUT, lse, ws, ws_bytes, None)

    assert forward(ws=None) == WORKSPACE and forward(ws=None, ws_bytes=0) == WORKSPACE
    assert forward(ws_bytes=need - 1) == WORKSPACE and forward(ws_bytes=0) == WORKSPACE
    assert forward(ws=WS + 8) == MISALIGNED and forward(ws=WS + 1) == MISALIGNED
    for other in (Q, K, V, OUT):
        assert forward(ws=other) == INVALID and forward(ws=other - need + 16) == INVALID
    assert forward(ws=OUT + 8 * 128 * 2 - 16) == INVALID               # the output's last bytes
    assert forward(lse=LSE, ws=LSE + 16) == INVALID and forward(lse=WS + need - 16) == INVALID
    assert forward(mask=MASK, ws=MASK + 39984) == INVALID and forward(lengths=LEN, ws=LEN) == INVALID
    assert forward(mask=WS + need - 1) == INVALID and forward(lengths=WS + need - 4) == INVALID
    lib.cross_attention_destroy(plan)
