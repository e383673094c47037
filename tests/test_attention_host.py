"""Host checks of the attention operators (no GPU needed): the oracle against
torch's own float64 attention and complex rotations, plan frequencies against the
formulas, plan facts, and every refusal of the C ABI and of the binding. A
refused call returns before any launch, so made-up addresses are safe."""
import ctypes
import math

import pytest
import torch

import attention_oracle as ao
import image_stencil_amd as isa
from image_stencil_amd import _abi

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = (_abi.IS_ERR_INVALID_ARG, _abi.IS_ERR_UNSUPPORTED,
                                               _abi.IS_ERR_MISALIGNED, _abi.IS_ERR_WORKSPACE)


# ------------------------------------------------------------------- the oracle
def test_oracle_attention_matches_torch():
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 5, 4, 16, dtype=torch.float64, generator=g)
    k, v = (torch.randn(2, 9, 2, 16, dtype=torch.float64, generator=g) for _ in range(2))
    see = torch.rand(2, 9, generator=g) < 0.6
    see[:, 0] = True
    out, lse, *_ = ao.attention(q, k, v, 0.25, see)
    kk, vv = (t.repeat_interleave(2, 2).permute(0, 2, 1, 3) for t in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(q.permute(0, 2, 1, 3), kk, vv,
                                                            attn_mask=see[:, None, None, :], scale=0.25)
    assert torch.allclose(out, want.permute(0, 2, 1, 3), rtol=1e-13, atol=1e-13)
    assert torch.isfinite(lse).all()
    see[1] = False
    out, lse, *_ = ao.attention(q, k, v, 0.25, see)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_oracle_rotation_keeps_dot_products_of_relative_positions(layout):
    """q at i and k at j meet as q at i + 7 and k at j + 7 do; pairs keep their length."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, 2, 1, 24, dtype=torch.float64, generator=g)
    f = ao.frequencies(16, 1)
    dots = []
    for shift in (0, 7):
        pos = torch.tensor([[[3 + shift], [11 + shift]]], dtype=torch.int32)
        y, _ = ao.rotate(x, pos, 16, 1, layout, f)
        dots.append((y[0, 0, 0] * y[0, 1, 0]).sum())
        assert torch.equal(y[..., 16:], x[..., 16:])
        assert abs(y.square().sum() - x.square().sum()) < 1e-12
    assert abs(dots[0] - dots[1]) < 1e-12


# -------------------------------------------------------------- rotary: the plan
@pytest.mark.parametrize("rot,axes,scaling", [(64, 1, "none"), (64, 2, "linear"), (96, 3, "ramp"), (128, 1, "ntk"),
                                              (2, 1, "none"), (0, 2, "none"), (256, 1, "ramp")])
def test_plan_frequencies(rot, axes, scaling):
    kw = dict(base=5000.0, scaling=scaling, factor=8.0, original_len=1024, ramp=(1.0, 32.0))
    got = isa.Rotary(256, rot, axes=axes, **kw).frequencies()
    want = ao.frequencies(rot, axes, **kw)
    assert len(got) == rot // 2 // axes
    for a, b in zip(got, want):
        assert abs(a - b) <= 1e-14 * b
    if scaling == "ntk":   # the fastest pair stays, the slowest is slowed by the factor
        plain = ao.frequencies(rot, axes, base=5000.0)
        assert got[0] == plain[0] and abs(got[-1] * 8.0 / plain[-1] - 1) < 1e-12


def _rotary_status(**kw):
    d = dict(d=64, rot=64, axes=1, layout=0, scaling=0, original_len=0, base=1e4, factor=1.0, ramp_low=1.0,
             ramp_high=32.0, magnitude=1.0)
    d.update(kw)
    desc = _abi.rotary_desc(**d)
    plan = ctypes.c_void_p()
    st = _abi.load().rotary_create(ctypes.byref(desc), ctypes.byref(plan))
    assert (st == 0) == bool(plan.value)
    if st == 0:
        _abi.load().rotary_destroy(plan)
    return st


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"d": 0}, INVALID), ({"rot": 63}, INVALID), ({"rot": 66}, INVALID), ({"rot": -2}, INVALID),
    ({"d": 257}, UNSUPPORTED), ({"axes": 0}, INVALID), ({"axes": 4}, UNSUPPORTED), ({"axes": 3}, INVALID),
    ({"layout": 2}, INVALID), ({"scaling": 4}, INVALID), ({"scaling": -1}, INVALID), ({"base": 0.0}, INVALID),
    ({"base": math.inf}, INVALID), ({"base": math.nan}, INVALID), ({"magnitude": 0.0}, INVALID),
    ({"magnitude": math.nan}, INVALID), ({"scaling": 1, "factor": 0.5}, INVALID),
    ({"scaling": 1, "factor": math.nan}, INVALID), ({"scaling": 0, "factor": 0.0}, 0),
    ({"scaling": 2, "factor": 2.0, "rot": 2}, UNSUPPORTED), ({"scaling": 3, "original_len": 0}, INVALID),
    ({"scaling": 3, "original_len": 10, "ramp_low": 4.0, "ramp_high": 4.0}, INVALID),
    ({"scaling": 3, "original_len": 10, "ramp_low": -1.0}, INVALID), ({"rot": 0}, 0), ({"d": 7, "rot": 6, "axes": 3}, 0)])
def test_rotary_create_refusals(kw, status):
    assert _rotary_status(**kw) == status


def _tokens(n=2, length=3, heads=4, d=64, **kw):
    t = _abi.is_tokens(n, length, heads, length * heads * d, heads * d, d)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


A, B, POS = 0x100000, 0x900000, 0xF00000   # made-up addresses, far apart


def test_rotary_forward_refusals():
    lib, plan = _abi.load(), isa.Rotary(64)

    def st(dtype=_abi.IS_F16, xt=None, x=A, pos=POS, pb=3, yt=None, y=B, handle=plan.handle):
        return lib.rotary_forward(handle, dtype, xt or _tokens(), x, pos, pb, yt or _tokens(), y, None)

    assert st(handle=None) == INVALID
    assert lib.rotary_forward(plan.handle, 1, None, A, POS, 3, _tokens(), B, None) == INVALID
    assert st(dtype=3) == UNSUPPORTED
    assert st(x=None) == INVALID and st(y=None) == INVALID and st(pos=None) == INVALID
    assert st(x=A + 8) == MISALIGNED and st(y=B + 2) == MISALIGNED and st(pos=POS + 2) == MISALIGNED
    assert st(y=A + 64) == INVALID                                        # ranges meet
    assert st(y=A, yt=_tokens(token_stride=512, batch_stride=4096)) == INVALID   # same base, other strides
    assert st(y=POS - 16) == INVALID                                      # positions inside the output
    assert st(yt=_tokens(length=4)) == INVALID and st(yt=_tokens(heads=2)) == INVALID
    assert st(xt=_tokens(n=-1), yt=_tokens(n=-1)) == INVALID
    assert st(xt=_tokens(head_stride=-64)) == INVALID
    assert st(yt=_tokens(head_stride=0)) == INVALID                       # two heads at one address
    assert st(yt=_tokens(token_stride=128)) == INVALID                    # tokens over each other
    assert st(pb=-1) == INVALID
    assert st(xt=_tokens(batch_stride=1 << 50)) == UNSUPPORTED
    # nothing to do: no launch, no pointer needed
    for empty in ({"n": 0}, {"length": 0}, {"heads": 0}):
        assert st(xt=_tokens(**empty), yt=_tokens(**empty), x=None, y=None, pos=None) == 0


def test_qk_norm_refusals():
    lib, plan = _abi.load(), isa.Rotary(64)

    def st(q=A, k=0x400000, wq=0x1000, wk=0x2000, qo=B, ko=0xC00000, qp=POS, kp=POS, **kw):
        d = dict(dtype=_abi.IS_BF16, norm=_abi.IS_NORM_RMS, eps=1e-6, q=_tokens(), k=_tokens(heads=2),
                 q_out=_tokens(), k_out=_tokens(heads=2), q_pos_batch_stride=0, k_pos_batch_stride=0)
        d.update(kw)
        return lib.qk_norm_rotary_forward(plan.handle, ctypes.byref(_abi.qk_norm_desc(**d)), q, k, wq, wk, qp, kp, qo,
                                          ko, None)

    assert lib.qk_norm_rotary_forward(plan.handle, None, A, A, None, None, POS, POS, B, B, None) == INVALID
    assert st(dtype=9) == UNSUPPORTED
    assert st(norm=0) == INVALID and st(norm=3) == INVALID
    assert st(eps=-1.0) == INVALID and st(eps=math.nan) == INVALID and st(eps=math.inf) == INVALID
    assert st(q=None) == INVALID and st(k=None) == INVALID and st(ko=None) == INVALID and st(kp=None) == INVALID
    assert st(wq=0x1004) == MISALIGNED and st(k=0x400002) == MISALIGNED
    assert st(qo=0x1000 - 32) == INVALID                                  # weights inside the output
    assert st(ko=B) == INVALID                                            # both outputs at one base
    assert st(k_out=_tokens(heads=3)) == INVALID
    empty = _tokens(length=0)
    assert st(q_out=empty, k_out=empty, **{}) == INVALID                  # only one side empty


# ---------------------------------------------------------------- cross attention
def _desc(n=2, lq=5, lk=7, hq=4, hkv=2, d=64, dtype=_abi.IS_F16, scale=0.0, **kw):
    S = ctypes.c_int64 * 3
    out = _abi.cross_attention_desc(n, lq, lk, hq, hkv, d, dtype, scale, S(lq * hq * d, hq * d, d),
                                    S(lk * hkv * d, hkv * d, d), S(lk * hkv * d, hkv * d, d),
                                    S(lq * hq * d, hq * d, d), lk)
    for k, v in kw.items():
        setattr(out, k, S(*v) if isinstance(v, tuple) else v)
    return out


def _create(desc):
    plan = ctypes.c_void_p()
    st = _abi.load().cross_attention_create(ctypes.byref(desc), ctypes.byref(plan))
    assert (st == 0) == bool(plan.value)
    return st, plan


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"n": 0}, 0), ({"lq": 0}, 0), ({"lk": 0}, 0), ({"n": -1}, INVALID), ({"lq": -1}, INVALID),
    ({"lk": -1}, INVALID), ({"hq": 0}, INVALID), ({"hkv": 0}, INVALID), ({"hq": 3}, INVALID), ({"d": 0}, INVALID),
    ({"d": 20}, UNSUPPORTED), ({"d": 264}, UNSUPPORTED), ({"d": 8}, 0), ({"d": 256}, 0),
    ({"dtype": _abi.IS_F32}, UNSUPPORTED), ({"dtype": 3}, UNSUPPORTED), ({"dtype": _abi.IS_BF16}, 0),
    ({"scale": math.inf}, INVALID), ({"scale": math.nan}, INVALID), ({"scale": -0.5}, 0),
    ({"mask_batch_stride": -1}, INVALID), ({"q_stride": (1280, 256, 60)}, MISALIGNED),
    ({"k_stride": (900, 128, 64)}, MISALIGNED), ({"v_stride": (896, 124, 64)}, MISALIGNED),
    ({"out_stride": (1284, 256, 64)}, MISALIGNED), ({"out_stride": (0, 256, 64)}, INVALID),
    ({"out_stride": (1280, 64, 64)}, INVALID), ({"k_stride": (0, 128, 64)}, 0), ({"k_stride": (0, 0, 0)}, 0),
    ({"k_stride": (-896, 128, 64)}, INVALID), ({"k_stride": (1 << 40, (1 << 23) + 8, 64)}, UNSUPPORTED),
    ({"v_stride": (1 << 50, 128, 64)}, UNSUPPORTED), ({"lq": 1 << 30, "lk": 1}, UNSUPPORTED)])
def test_cross_attention_create_refusals(kw, status):
    st, plan = _create(_desc(**kw))
    assert st == status
    _abi.load().cross_attention_destroy(plan)


def test_cross_attention_null_arguments():
    lib = _abi.load()
    assert lib.cross_attention_create(None, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.cross_attention_create(ctypes.byref(_desc()), None) == INVALID
    assert lib.cross_attention_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib.cross_attention_forward(None, A, A, A, None, None, B, None, None, 0, None) == INVALID
    assert lib.rotary_create(None, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.rotary_get_frequencies(None, None, 0, ctypes.byref(ctypes.c_int())) == INVALID
    lib.cross_attention_destroy(None)
    lib.rotary_destroy(None)


def test_cross_attention_forward_refusals():
    lib = _abi.load()
    _, plan = _create(_desc())
    K, V, LSE = 0x400000, 0x500000, 0xC00000

    def st(q=A, k=K, v=V, mask=None, lengths=None, out=B, lse=None, ws=None, ws_bytes=0, handle=plan):
        return lib.cross_attention_forward(handle, q, k, v, mask, lengths, out, lse, ws, ws_bytes, None)

    assert st(q=None) == INVALID and st(k=None) == INVALID and st(v=None) == INVALID and st(out=None) == INVALID
    assert st(q=A + 8) == MISALIGNED and st(k=K + 2) == MISALIGNED and st(v=V + 8) == MISALIGNED
    assert st(out=B + 8) == MISALIGNED and st(lse=LSE + 2) == MISALIGNED and st(lengths=LSE + 1) == MISALIGNED
    assert st(out=A) == INVALID and st(out=K) == INVALID and st(out=V - 16) == INVALID
    assert st(lse=B + 16) == INVALID and st(lse=A) == INVALID
    assert st(mask=B + 3) == INVALID and st(lengths=B + 4) == INVALID
    lib.cross_attention_destroy(plan)
    for kw in ({"n": 0}, {"lq": 0}):                     # nothing to write
        _, plan = _create(_desc(**kw))
        assert st(q=None, k=None, v=None, out=None, handle=plan) == 0
        lib.cross_attention_destroy(plan)


# ------------------------------------------------------------------- the binding
def _t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals():
    r = isa.Rotary(64, axes=2)
    pos = torch.zeros(2, 3, 2, dtype=torch.int32)
    x = _t(2, 3, 4, 64)
    with pytest.raises(TypeError, match="on a GPU"):
        r.apply(x, pos)
    with pytest.raises(TypeError, match="int32"):
        r.apply(x, pos.long())
    with pytest.raises(ValueError, match="positions must be"):
        r.apply(x, pos[:, :2])
    with pytest.raises(ValueError, match="positions must be"):
        r.apply(x, pos[:, :, 0])
    with pytest.raises(ValueError, match="contiguous rows"):
        r.apply(x, torch.zeros(2, 2, 3, dtype=torch.int32).transpose(1, 2))
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        r.apply(x.double(), pos)
    with pytest.raises(ValueError, match="64"):
        r.apply(_t(2, 3, 4, 32), pos)
    with pytest.raises(ValueError, match="contiguous last"):
        r.apply(_t(2, 3, 64, 4).transpose(2, 3), pos)
    with pytest.raises(ValueError, match="out has shape"):
        r.apply(x, pos, out=_t(2, 3, 2, 64))
    with pytest.raises(ValueError, match="norm must be"):
        r.apply_qk_norm(x, x, pos, norm="l2")
    with pytest.raises(TypeError, match="q_weight"):
        r.apply_qk_norm(x, x, pos, q_weight=_t(64))
    with pytest.raises(ValueError, match="k_weight"):
        r.apply_qk_norm(x, x, pos, k_weight=_t(32, dtype=torch.float32))
    with pytest.raises(TypeError, match="k must be"):
        r.apply_qk_norm(x, x.float(), pos)
    with pytest.raises(ValueError, match="k_positions"):
        r.apply_qk_norm(x, _t(2, 5, 1, 64), pos)
    with pytest.raises(ValueError, match="layout"):
        isa.Rotary(64, layout="quarter")
    with pytest.raises(ValueError, match="scaling"):
        isa.Rotary(64, scaling="cubic")
    with pytest.raises(isa.ImgStencilError):
        isa.Rotary(64, 65)

    q, k = _t(2, 5, 4, 64), _t(2, 7, 2, 64)
    with pytest.raises(TypeError, match="on a GPU"):
        isa.cross_attention(q, k, k)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        isa.cross_attention(q.float(), k, k)
    with pytest.raises(TypeError, match="v must be"):
        isa.cross_attention(q, k, k.bfloat16())
    with pytest.raises(ValueError, match="batch"):
        isa.cross_attention(q, k[:1], k[:1])
    with pytest.raises(ValueError, match="share"):
        isa.cross_attention(q, _t(2, 7, 3, 64), _t(2, 7, 3, 64))
    with pytest.raises(ValueError, match="v "):
        isa.cross_attention(q, k, _t(2, 6, 2, 64))
    with pytest.raises(ValueError, match="expected 64"):
        isa.cross_attention(q, _t(2, 7, 2, 32), _t(2, 7, 2, 32))
    with pytest.raises(ValueError, match="scale"):
        isa.cross_attention(q, k, k, scale=0.0)
    p = isa.CrossAttention(q, k, k)
    with pytest.raises(ValueError, match="the plan is for"):
        p.forward(q[:, :4], k, k)
    with pytest.raises(ValueError, match="the plan is for"):
        p.forward(q, k, k.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(TypeError, match="bfloat16|float16"):
        p.forward(q.bfloat16(), k, k)
    with pytest.raises(TypeError, match="key_mask"):
        p.forward(q, k, k, key_mask=torch.zeros(2, 7))
    with pytest.raises(ValueError, match="key_mask"):
        p.forward(q, k, k, key_mask=torch.zeros(2, 5, dtype=torch.bool))
    with pytest.raises(TypeError, match="key_lengths"):
        p.forward(q, k, k, key_lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="key_lengths"):
        p.forward(q, k, k, key_lengths=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="lse"):
        p.forward(q, k, k, lse=torch.zeros(2, 4, 5, dtype=torch.float16))
    with pytest.raises(ValueError, match="lse"):
        p.forward(q, k, k, lse=torch.zeros(2, 5, 4))
    with pytest.raises(ValueError, match="stream"):
        p.forward(q, k, k, stream=1)


def test_bf16_stays_out_of_the_convolutions():
    d = isa.make_desc(1, 4, 8, 8, 4, 3, 3, dtype="f16")
    d.in_dtype = d.out_dtype = _abi.IS_BF16
    with pytest.raises(isa.ImgStencilError) as e:
        isa.conv2d_create(d)
    assert e.value.status == UNSUPPORTED
