"""The operators around attention on the CPU: the 64-bit forms against torch's own,
plans, and what the C ABI and the binding refuse. Refusals come before any launch, so
made-up addresses are safe."""
import ctypes
import math

import pytest
import torch

import blocks_oracle as bo
import image_stencil_amd as isa
from image_stencil_amd import _abi
from test_attention_host import INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE

A, B, C, D = 0x1000000, 0x9000000, 0x11000000, 0x19000000   # made-up addresses, far apart


# -------------------------------------------------------------------- the oracle
def test_oracle_norms_match_torch():
    g = torch.Generator().manual_seed(0)
    x, y = torch.randn(2, 5, 24, generator=g), torch.randn(2, 5, 24, generator=g)
    w, b = torch.randn(24, generator=g), torch.randn(24, generator=g)
    want = torch.nn.functional.layer_norm(x.double() + 0.5 * y.double(), (24,), w.double(), b.double(), 1e-5)
    got = bo.block_norm(x, y, "layer", eps=1e-5, residual_scale=0.5, weight=w, bias=b)[2]
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)
    want = torch.nn.functional.rms_norm(x.double(), (24,), w.double(), 1e-5)
    assert torch.allclose(bo.block_norm(x, norm="rms", eps=1e-5, weight=w)[2], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("act,f", [("gelu", torch.nn.functional.gelu), ("silu", torch.nn.functional.silu),
                                   ("gelu_tanh", lambda z: torch.nn.functional.gelu(z, approximate="tanh"))])
def test_oracle_activations_match_torch(act, f):
    z = torch.linspace(-6, 6, 1001, dtype=torch.float64)
    assert torch.allclose(bo.activate(z, act), f(z), rtol=1e-10, atol=1e-14)


def test_oracle_e4m3_matches_torch():
    x = torch.cat([torch.linspace(-448, 448, 100001), bo.E4M3.float(), (bo.E4M3[:-1] + bo.E4M3[1:]).float() / 2])
    assert torch.equal(bo.nearest_e4m3(x.double()), x.to(torch.float8_e4m3fn).double())


# --------------------------------------------------------------- block_norm, C ABI
def _rows(n=2, length=3, c=64, batch=None, row=None):
    row = c if row is None else row
    return _abi.is_rows(n, length, length * row if batch is None else batch, row)


@pytest.mark.parametrize("kw,status", [
    (dict(c=0), INVALID), (dict(c=16385), UNSUPPORTED), (dict(norm=3), INVALID), (dict(post=5), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(residual_scale=math.inf), INVALID), (dict(residual_scale=math.nan), INVALID), (dict(dtype=7), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(norm=0), INVALID),
    (dict(y=None), INVALID), (dict(y=None, x_out=None, post=1), INVALID), (dict(y=None, x_out=None, gate=A + 64), INVALID),
    (dict(x=A + 8), MISALIGNED), (dict(y=B + 2), MISALIGNED), (dict(out=D + 8), MISALIGNED),
    (dict(gate=0x21000001), MISALIGNED), (dict(w=0x21000002), MISALIGNED),
    (dict(gate_stride=-1), INVALID), (dict(x_out_=_rows(row=-64)), INVALID),
    (dict(y_=_rows(n=3)), INVALID), (dict(out_=_rows(row=32)), INVALID), (dict(x_out_=_rows(batch=0)), INVALID),
    (dict(out=A + 64), INVALID), (dict(out=B + 64), INVALID), (dict(out=C), INVALID), (dict(x_out=A + 128), INVALID),
    (dict(w=D + 64), INVALID), (dict(shift=C + 64), INVALID), (dict(x_=_rows(row=128), x_out=A), INVALID)])
def test_block_norm_refusals(kw, status):
    """Names with a trailing _ are the descriptor's rows, other names of it its fields,
    the rest pointers."""
    names = ("c", "norm", "post", "eps", "residual_scale", "dtype", "gate_stride")
    fields = {k.rstrip("_"): v for k, v in kw.items() if k in names or isinstance(v, _abi.is_rows)}
    ptrs = {k: v for k, v in kw.items() if k not in names and not isinstance(v, _abi.is_rows)}
    d = _abi.block_norm_desc(_abi.IS_F16, 64, _abi.IS_NORM_RMS, 0, 1e-6, 1.0, _rows(), _rows(), _rows(), _rows(), 0, 0, 0)
    for k, v in fields.items():
        setattr(d, k, v)
    p = dict(x=A, y=B, gate=None, pw=None, w=None, b=None, scale=None, shift=None, x_out=C, out=D)
    p.update(ptrs)
    assert _abi.load().block_norm_forward(ctypes.byref(d), *p.values(), None) == status


def test_block_norm_empty_and_null():
    lib = _abi.load()
    assert lib.block_norm_forward(None, *[None] * 11) == INVALID
    for n, length in ((0, 3), (2, 0)):
        r = _rows(n=n, length=length)
        d = _abi.block_norm_desc(_abi.IS_F32, 64, 1, 0, 0.0, 1.0, r, r, r, r, 0, 0, 0)
        assert lib.block_norm_forward(ctypes.byref(d), *[None] * 11) == 0


def test_block_norm_calls_fit_a_launch():
    n = 2 ** 23
    r = _rows(n=n, length=1, c=16384)
    far = 1 << 42
    d = _abi.block_norm_desc(_abi.IS_F16, 16384, 1, 0, 1e-6, 1.0, r, r, r, r, 0, 0, 0)
    st = _abi.load().block_norm_forward(ctypes.byref(d), far, 2 * far, None, None, None, None, None, None, 3 * far, 4 * far,
                                        None)
    assert st == UNSUPPORTED
    # more rows than 32 bits count, in few channels
    r = _abi.is_rows(2 ** 30, 2 ** 12, 2 ** 12, 1)
    d = _abi.block_norm_desc(_abi.IS_F16, 1, 1, 0, 1e-6, 1.0, r, r, r, r, 0, 0, 0)
    st = _abi.load().block_norm_forward(ctypes.byref(d), 1 << 44, None, None, None, None, None, None, None, None, 1 << 45,
                                        None)
    assert st == UNSUPPORTED


# ------------------------------------------------------------------- dense, C ABI
def _dense_desc(n=2, length=40, k=64, m=96, dtype=_abi.IS_F16, act=0, xs=None, rs=None, os=None, ws=None):
    S = ctypes.c_int64 * 2
    return _abi.dense_desc(n, length, k, m, dtype, act, S(*(xs or (length * k, k))), S(*(rs or (length * m, m))),
                           S(*(os or (length * m, m))), k if ws is None else ws)


def _dense(**kw):
    plan = ctypes.c_void_p()
    d = _dense_desc(**kw)
    return _abi.load().dense_create(ctypes.byref(d), ctypes.byref(plan)), plan


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(length=-1), INVALID), (dict(k=0), INVALID), (dict(m=0), INVALID), (dict(act=5), INVALID),
    (dict(act=-1), INVALID), (dict(ws=-64), INVALID), (dict(dtype=_abi.IS_F32), UNSUPPORTED), (dict(k=60), UNSUPPORTED),
    (dict(xs=(2560, 68)), MISALIGNED), (dict(xs=(2564, 64)), MISALIGNED), (dict(ws=68), MISALIGNED),
    (dict(xs=(2 ** 30, 2 ** 21 + 8)), UNSUPPORTED), (dict(ws=2 ** 21 + 8), UNSUPPORTED),
    (dict(length=1, xs=(2 ** 21 + 8, 64)), UNSUPPORTED), (dict(os=(0, 96)), INVALID), (dict(os=(40 * 96, 48)), INVALID),
    (dict(xs=(-8, 64)), INVALID), (dict(n=2 ** 20, length=2 ** 20, m=2 ** 20), UNSUPPORTED),
    (dict(n=2 ** 10, length=2 ** 10, m=2 ** 28), UNSUPPORTED),
    (dict(), 0), (dict(n=0), 0), (dict(length=0), 0), (dict(m=1), 0), (dict(m=7, os=(40 * 7, 7)), 0), (dict(ws=2 ** 21), 0),
    (dict(xs=(0, 64)), 0), (dict(xs=(2560, 0)), 0)])
def test_dense_create_refusals(kw, status):
    st, plan = _dense(**kw)
    assert st == status
    assert bool(plan.value) == (status == 0)
    _abi.load().dense_destroy(plan)


@pytest.mark.parametrize("kw", [dict(n=1, length=2 ** 31 - 1, k=8, m=8), dict(n=1, length=1, k=2 ** 31 - 8, m=1),
                                dict(n=1, length=1, k=8, m=2 ** 31 - 1), dict(n=2, length=2 ** 31 - 64, k=8, m=8)])
def test_dense_sizes_that_whole_tiles_take_past_an_int(kw):
    """Rows, inputs or features rounded up to tiles would be negative."""
    st, plan = _dense(xs=(0, 0), os=(2 ** 31 * 8, 8), rs=(0, 0), **kw)
    assert st == UNSUPPORTED and not plan.value


def test_dense_null_arguments():
    lib, n, info = _abi.load(), ctypes.c_size_t(), _abi.conv2d_plan_info()
    d = _dense_desc()
    assert lib.dense_create(None, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.dense_create(ctypes.byref(d), None) == INVALID
    assert lib.dense_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.dense_get_plan_info(None, ctypes.byref(info)) == INVALID
    assert lib.dense_forward(None, A, B, None, None, C, None, 0, None) == INVALID
    lib.dense_destroy(None)


def test_dense_forward_refusals():
    lib = _abi.load()
    _, plan = _dense()

    def st(x=A, w=B, bias=None, res=None, out=C, ws=None, size=0):
        return lib.dense_forward(plan, x, w, bias, res, out, ws, size, None)

    assert st(x=None) == INVALID and st(w=None) == INVALID and st(out=None) == INVALID
    assert st(x=A + 8) == MISALIGNED and st(w=B + 2) == MISALIGNED and st(out=C + 8) == MISALIGNED
    assert st(res=D + 8) == MISALIGNED and st(bias=D + 2) == MISALIGNED
    for over in (A, A + 64, B, B + 16):
        assert st(out=over) == INVALID
    assert st(bias=C + 16) == INVALID and st(res=C + 16) == INVALID
    lib.dense_destroy(plan)
    # residual at out, but with other strides
    S = (40 * 96 * 2, 96 * 2)
    _, plan = _dense(rs=S)
    assert lib.dense_forward(plan, A, B, None, C, C, None, 0, None) == INVALID
    lib.dense_destroy(plan)
    _, plan = _dense(n=0)
    assert lib.dense_forward(plan, None, None, None, None, None, None, 0, None) == 0
    lib.dense_destroy(plan)


@pytest.mark.parametrize("n,length,k,m", [(1, 1, 8, 1), (1, 1, 16384, 8192), (1, 40, 8192, 64), (16, 1, 1024, 4096),
                                          (3, 1021, 344, 777), (1, 2 ** 20, 64, 64), (2 ** 20, 1, 64, 64), (1, 256, 64, 8192),
                                          (1, 257, 8, 9), (5, 100, 4096, 1024)])
@pytest.mark.parametrize("gap", [0, 8])
def test_dense_plans_cover_their_rows_and_features(n, length, k, m, gap):
    """Tiles times their number hold all rows and features, and a split sum's workspace
    every part; entries with gaps between them are not joined."""
    batch = length * k + gap
    st, plan = _dense(n=n, length=length, k=k, m=m, xs=(batch, k))
    assert st == 0
    info, ws = _abi.conv2d_plan_info(), ctypes.c_size_t()
    lib = _abi.load()
    assert lib.dense_get_plan_info(plan, ctypes.byref(info)) == 0
    assert lib.dense_workspace_size(plan, ctypes.byref(ws)) == 0
    one = gap == 0 or n == 1 or length == 1
    entries, rows = (1, n * length) if one else (n, length)
    tiles = entries * -(-rows // info.tile_h) * -(-m // info.tile_w)
    assert info.grid_x == tiles and info.flops == 2.0 * n * length * k * m
    assert ws.value == (0 if info.grid_y == 1 else info.grid_y * n * length * -(-m // 8) * 8 * 4)
    assert 1 <= info.grid_y <= max(1, -(-k // 64))
    lib.dense_destroy(plan)


@pytest.mark.parametrize("lq,length,hq,heads,d", [(1, 1, 1, 1, 8), (1, 40000, 8, 1, 128), (5, 100, 4, 2, 40), (1000, 333, 4, 4, 64),
                                                  (9000, 300, 8, 8, 64), (40, 0, 2, 1, 256), (300, 9000, 16, 4, 256)])
def test_held_attention_plans_cover_their_keys_and_rows(lq, length, hq, heads, d):
    n = 2
    st, plan = _attend(n=n, length=length, heads=heads, d=d, lq=lq, hq=hq, mb=length)
    assert st == 0
    info, ws = _abi.conv2d_plan_info(), ctypes.c_size_t()
    lib = _abi.load()
    assert lib.held_attention_get_plan_info(plan, ctypes.byref(info)) == 0
    assert lib.held_attention_workspace_size(plan, ctypes.byref(ws)) == 0
    rows = lq * (hq // heads)
    assert info.grid_y * info.tile_w >= length
    if info.kernel == b"is_k15_held_attention":
        assert info.tile_w % 32 == 0 and (info.grid_y - 1) * info.tile_w < max(length, 1)
        assert info.grid_x == n * heads * -(-rows // 32)
        assert ws.value == (0 if info.grid_y == 1 else info.grid_x * info.grid_y * 32 * (d + 1) * 4)
    else:
        assert rows > 32 and ws.value >= 2 * n * length * heads * d * 2
    lib.held_attention_destroy(plan)


def test_dense_split_plans_need_their_workspace():
    st, plan = _dense(n=1, length=64, k=8192, m=64)
    assert st == 0
    n = ctypes.c_size_t()
    lib = _abi.load()
    assert lib.dense_workspace_size(plan, ctypes.byref(n)) == 0
    info = _abi.conv2d_plan_info()
    assert lib.dense_get_plan_info(plan, ctypes.byref(info)) == 0
    if info.grid_y > 1:
        assert n.value >= info.grid_y * 64 * 64 * 4
        assert lib.dense_forward(plan, A, B, None, None, C, None, 0, None) == WORKSPACE
        assert lib.dense_forward(plan, A, B, None, None, C, D, n.value - 1, None) == WORKSPACE
        assert lib.dense_forward(plan, A, B, None, None, C, D + 8, n.value, None) == MISALIGNED
        for over in (A, B, C):
            assert lib.dense_forward(plan, A, B, None, None, C, over, n.value, None) == INVALID
        assert lib.dense_forward(plan, A, B, None, D, C, D, n.value, None) == INVALID
    lib.dense_destroy(plan)


# -------------------------------------------------------------- held states, C ABI
def _states(n=2, length=100, heads=3, d=40, dtype=_abi.IS_F16):
    return _abi.held_states_desc(n, length, heads, d, dtype)


def _size(**kw):
    n, d = ctypes.c_size_t(), _states(**kw)
    return _abi.load().held_states_size(ctypes.byref(d), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(length=-1), INVALID), (dict(heads=0), INVALID), (dict(d=0), INVALID),
    (dict(d=36), UNSUPPORTED), (dict(d=264), UNSUPPORTED), (dict(dtype=_abi.IS_F32), UNSUPPORTED),
    (dict(n=2 ** 20, length=2 ** 20), UNSUPPORTED), (dict(), 0), (dict(n=0), 0), (dict(length=0), 0), (dict(d=256), 0)])
def test_held_states_size(kw, status):
    st, size = _size(**kw)
    assert st == status
    if st == 0:
        s = dict(n=2, length=100, heads=3, d=40)
        s.update(kw)
        blocks = s["n"] * s["heads"] * -(-s["length"] // 32)
        assert size == blocks * (64 * (-(-s["d"] // 32) * 32) + 8)
    d = _states()
    assert _abi.load().held_states_size(ctypes.byref(d), None) == INVALID
    assert _abi.load().held_states_size(None, ctypes.byref(ctypes.c_size_t())) == INVALID


def _tok(n=2, length=100, heads=3, d=40, **kw):
    t = _abi.is_tokens(n, length, heads, length * heads * d, heads * d, d)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def test_held_store_refusals():
    lib, size = _abi.load(), _size()[1]

    def st(kt=None, k=A, vt=None, v=B, mask=None, ms=0, lengths=None, at=0, held=C, bytes_=size, d=None):
        d = d or _states()
        return lib.held_store(ctypes.byref(d), kt or _tok(), k, vt or _tok(), v, mask, ms, lengths, at, held, bytes_, None)

    assert st(k=None) == INVALID and st(v=None) == INVALID and st(held=None) == INVALID
    assert st(at=32) == INVALID and st(at=-32) == INVALID and st(kt=_tok(length=50), vt=_tok(length=50), at=16) == INVALID
    assert st(kt=_tok(length=50)) == INVALID and st(kt=_tok(n=1)) == INVALID and st(vt=_tok(heads=2)) == INVALID
    assert st(kt=_tok(length=101), vt=_tok(length=101)) == INVALID
    assert st(k=A + 8) == MISALIGNED and st(v=B + 2) == MISALIGNED and st(held=C + 8) == MISALIGNED
    assert st(lengths=D + 2) == MISALIGNED and st(ms=-1) == INVALID
    assert st(bytes_=size - 1) == WORKSPACE
    assert st(held=A) == INVALID and st(held=B + 16) == INVALID and st(mask=C + 64) == INVALID
    assert st(lengths=C + 64) == INVALID and st(kt=_tok(token_stride=-8)) == INVALID
    assert st(d=_states(d=44)) == UNSUPPORTED
    assert st(kt=_tok(length=0), vt=_tok(length=0), k=None, v=None, held=None, bytes_=0, at=32) == 0   # nothing to store


def test_held_load_refusals():
    lib, size = _abi.load(), _size()[1]

    def st(kt=None, k=A, vt=None, v=B, at=0, held=C, bytes_=size):
        d = _states()
        return lib.held_load(ctypes.byref(d), held, bytes_, at, kt or _tok(), k, vt or _tok(), v, None)

    assert st(k=None) == INVALID and st(held=None) == INVALID and st(at=1) == INVALID and st(at=-1) == INVALID
    assert st(kt=_tok(length=50)) == INVALID and st(vt=_tok(heads=1)) == INVALID
    assert st(k=A + 2) == MISALIGNED and st(held=C + 4) == MISALIGNED and st(bytes_=size - 1) == WORKSPACE
    assert st(k=C) == INVALID and st(v=C + 16) == INVALID and st(v=A) == INVALID and st(v=A + 16) == INVALID
    assert st(kt=_tok(token_stride=0)) == INVALID and st(vt=_tok(batch_stride=8)) == INVALID


def _attend(n=2, length=100, heads=2, d=40, dtype=_abi.IS_F16, lq=5, hq=4, scale=0.0, qs=None, os=None, mb=100):
    S, plan = ctypes.c_int64 * 3, ctypes.c_void_p()
    dense = (lq * hq * d, hq * d, d)
    desc = _abi.held_attention_desc(_states(n, length, heads, d, dtype), lq, hq, scale, S(*(qs or dense)),
                                    S(*(os or dense)), mb)
    return _abi.load().held_attention_create(ctypes.byref(desc), ctypes.byref(plan)), plan


@pytest.mark.parametrize("kw,status", [
    (dict(lq=-1), INVALID), (dict(hq=0), INVALID), (dict(hq=3), INVALID), (dict(heads=0), INVALID),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=2.5e38), INVALID), (dict(mb=-1), INVALID),
    (dict(d=44), UNSUPPORTED), (dict(dtype=_abi.IS_F32), UNSUPPORTED), (dict(qs=(800, 164, 40)), MISALIGNED),
    (dict(os=(800, 160, 44)), MISALIGNED), (dict(os=(800, 160, 0)), INVALID), (dict(qs=(800, -160, 40)), INVALID),
    (dict(lq=2 ** 30), UNSUPPORTED), (dict(), 0), (dict(qs=(0, 160, 40)), 0), (dict(lq=0), 0), (dict(n=0), 0),
    (dict(length=0), 0), (dict(lq=3000), 0)])
def test_held_attention_create_refusals(kw, status):
    st, plan = _attend(**kw)
    assert st == status
    _abi.load().held_attention_destroy(plan)


@pytest.mark.parametrize("lq", [5, 1000])
def test_held_attention_forward_refusals(lq):
    """lq = 1000: the states are loaded into the workspace first."""
    lib = _abi.load()
    _, plan = _attend(lq=lq, length=40000)
    size, need = _size(length=40000, heads=2)[1], ctypes.c_size_t()
    assert lib.held_attention_workspace_size(plan, ctypes.byref(need)) == 0
    assert need.value > 0
    far = 1 << 40

    def st(q=far, held=2 * far, bytes_=size, mask=None, lengths=None, out=3 * far, lse=None, ws=4 * far, wb=need.value):
        return lib.held_attention_forward(plan, q, held, bytes_, mask, lengths, out, lse, ws, wb, None)

    assert st(q=None) == INVALID and st(held=None) == INVALID and st(out=None) == INVALID
    assert st(bytes_=size - 1) == WORKSPACE and st(ws=None) == WORKSPACE and st(wb=need.value - 1) == WORKSPACE
    assert st(q=far + 8) == MISALIGNED and st(held=far + 8) == MISALIGNED and st(ws=far + 8) == MISALIGNED
    assert st(lse=far + 2) == MISALIGNED and st(lengths=far + 2) == MISALIGNED
    assert st(out=far) == INVALID and st(out=2 * far + 64) == INVALID and st(ws=2 * far) == INVALID
    assert st(lse=3 * far) == INVALID and st(ws=far) == INVALID and st(mask=3 * far) == INVALID
    assert lib.held_attention_forward(None, far, far, 0, None, None, far, None, None, 0, None) == INVALID
    lib.held_attention_destroy(plan)


# --------------------------------------------------------------------- the binding
H, F = torch.float16, torch.float32


def test_block_norm_binding_refusals():
    x = torch.zeros(2, 3, 64, dtype=H)
    with pytest.raises(ValueError):
        isa.BlockNorm(64, norm="batch")
    with pytest.raises(ValueError):
        isa.BlockNorm(64, post="batch")
    for c in (0, 16385):
        with pytest.raises(ValueError):
            isa.BlockNorm(c)
    for eps in (-1.0, math.inf, math.nan, 1e-50):
        with pytest.raises(ValueError):
            isa.BlockNorm(64, eps=eps)
    plan, summed = isa.BlockNorm(64), isa.BlockNorm(64, norm=None)
    for kw, err in [(dict(x=x.double()), TypeError), (dict(x=x[0]), ValueError), (dict(x=x[..., :32]), ValueError),
                    (dict(x=[1]), TypeError), (dict(y=x.float()), TypeError), (dict(y=x[:1]), ValueError),
                    (dict(y=x.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                    (dict(gate=torch.zeros(2, 64, dtype=H)), ValueError), (dict(x_out=x), ValueError),
                    (dict(y=x, gate=torch.zeros(3, 64, dtype=H)), ValueError),
                    (dict(y=x, gate=torch.zeros(2, 64)), TypeError), (dict(y=x, gate=torch.zeros(64, dtype=H)), ValueError),
                    (dict(post_weight=torch.zeros(64)), ValueError), (dict(y=x, post_weight=torch.zeros(64)), ValueError),
                    (dict(weight=torch.zeros(64, dtype=H)), TypeError), (dict(weight=torch.zeros(32)), ValueError),
                    (dict(weight=torch.zeros(128)[::2]), ValueError), (dict(out=x.float()), TypeError),
                    (dict(out=x[:, :2]), ValueError), (dict(y=x, x_out=x[:1]), ValueError), (dict(), TypeError)]:
        with pytest.raises(err):
            plan.apply(**dict(dict(x=x), **kw))
    with pytest.raises(ValueError):
        summed.apply(x)
    for name in ("weight", "bias"):
        with pytest.raises(ValueError):
            summed.apply(x, x, **{name: torch.zeros(64)})
    with pytest.raises(ValueError):
        plan.apply(x, stream=5)


def test_dense_binding_refusals():
    x, w, r = torch.zeros(2, 3, 64, dtype=H), torch.zeros(10, 64, dtype=H), torch.zeros(2, 3, 10, dtype=H)
    for args, kw, err in [((x, w), dict(activation="tanh"), ValueError), ((x.float(), w.float()), {}, TypeError),
                          ((x, w.float()), {}, TypeError), ((x, w[:, :32]), {}, ValueError), ((x, w[0]), {}, ValueError),
                          ((x[0], w), {}, ValueError), ((x, w.T.contiguous().T), {}, ValueError),
                          ((x, w), dict(out=x), ValueError), ((x, w), dict(residual=r.float()), TypeError),
                          (([1], w), {}, TypeError)]:
        with pytest.raises(err):
            isa.Dense(*args, **kw)
    with pytest.raises(isa.ImgStencilError):
        isa.Dense(torch.zeros(2, 3, 60, dtype=H), torch.zeros(10, 60, dtype=H))
    plan = isa.Dense(x, w)
    for kw, err in [(dict(x=x[:1]), ValueError), (dict(w=w[:5]), ValueError), (dict(x=x.bfloat16()), TypeError),
                    (dict(bias=torch.zeros(9)), ValueError), (dict(bias=torch.zeros(10, dtype=H)), TypeError),
                    (dict(residual=r[:1]), ValueError), (dict(out=torch.zeros(2, 3, 20, dtype=H)[..., :10]), ValueError),
                    (dict(workspace=5), TypeError), (dict(stream=5), ValueError), (dict(), TypeError), (dict(x=3), TypeError)]:
        with pytest.raises(err):
            plan.forward(**dict(dict(x=x, w=w), **kw))


def test_held_binding_refusals():
    for kw, err in [(dict(dtype=F), TypeError), (dict(d=36), isa.ImgStencilError), (dict(d=264), isa.ImgStencilError),
                    (dict(length=2 ** 31), ValueError), (dict(n=-1), isa.ImgStencilError)]:
        with pytest.raises(err):
            isa.HeldStates(**dict(dict(n=2, length=100, heads=2, d=40, device="cpu"), **kw))
    held = isa.HeldStates(2, 100, 2, 40, device="cpu")
    k = torch.zeros(2, 64, 2, 40, dtype=H)
    for kw, err in [(dict(k=k[:1]), ValueError), (dict(v=k[:, :5]), ValueError), (dict(k=k.float()), TypeError),
                    (dict(at=64), ValueError), (dict(at=16), ValueError), (dict(at=-32), ValueError), (dict(k=1), TypeError),
                    (dict(key_mask=torch.ones(2, 60, dtype=torch.bool)), ValueError),
                    (dict(key_mask=torch.ones(2, 64)), TypeError), (dict(key_lengths=torch.ones(2)), TypeError),
                    (dict(key_lengths=torch.ones(3, dtype=torch.int32)), ValueError), (dict(), TypeError)]:
        with pytest.raises(err):
            held.put(**dict(dict(k=k, v=k), **kw))
    for kw, err in [(dict(at=101), ValueError), (dict(at=-1), ValueError), (dict(length=101), ValueError),
                    (dict(k_out=k), ValueError), (dict(length=64, v_out=k.float()), TypeError), (dict(stream=3), ValueError),
                    (dict(), TypeError)]:
        with pytest.raises(err):
            held.get(**kw)
    q = torch.zeros(2, 5, 4, 40, dtype=H)
    for args, kw, err in [((q, k), {}, TypeError), ((q.float(), held), {}, TypeError), ((q.bfloat16(), held), {}, TypeError),
                          ((q[:1], held), {}, ValueError), ((q[:, :, :3], held), {}, ValueError),
                          ((q, held), dict(scale=0.0), ValueError), ((q, held), dict(scale=1e-50), ValueError),
                          ((q, held), dict(out=q[:1]), ValueError)]:
        with pytest.raises(err):
            isa.HeldAttention(*args, **kw)
    plan, other = isa.HeldAttention(q, held), isa.HeldStates(2, 101, 2, 40, device="cpu")
    for kw, err in [(dict(held=other), ValueError), (dict(held=k), TypeError), (dict(q=q[:, :4]), ValueError),
                    (dict(key_mask=torch.ones(2, 99, dtype=torch.bool)), ValueError),
                    (dict(lse=torch.zeros(2, 4, 5, dtype=H)), TypeError), (dict(lse=torch.zeros(2, 5, 4)), ValueError),
                    (dict(stream=4), ValueError), (dict(), TypeError)]:
        with pytest.raises(err):
            plan.forward(**dict(dict(q=q, held=held), **kw))
