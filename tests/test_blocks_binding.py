"""What the binding of the operators around attention hands to the library, on the
CPU: tensors that pass for device tensors and a library that records its calls in
place of launching."""
import pytest
import torch

import image_stencil_amd as isa
from image_stencil_amd import blocks, held as held_module
from test_attention_binding import Recorder, _span, _t, fake, gpu  # noqa: F401


@pytest.fixture
def lone(fake, monkeypatch):  # noqa: F811
    """Every given tensor passes for one of the same device, allocated ones too."""
    for module in (blocks, held_module):
        monkeypatch.setattr(module, "_one_device", lambda tensors: True)
    return fake


def _held(n=2, length=70, heads=2, d=64, index=0, lib=None):
    states = isa.HeldStates(n, length, heads, d, device="cpu")
    states.data = gpu(states.data, index)
    states._lib = lib or Recorder()
    return states


def _calls(lib, index=0):
    """Every operator once, with tensors of GPU `index`."""
    x, w, q, k = (_t(2, 5, 64, index=index), _t(32, 64, index=index), _t(2, 5, 4, 64, index=index),
                  _t(2, 70, 2, 64, index=index))
    norm, dense, states = isa.BlockNorm(64), isa.Dense(x, w), _held(index=index, lib=lib)
    attend = isa.HeldAttention(q, states)
    norm._lib = dense._lib = attend._lib = lib
    return [("block_norm_forward", lambda **kw: norm.apply(x, **kw), {"out": x}),
            ("dense_forward", lambda **kw: dense.forward(x, w, **kw), {"out": _t(2, 5, 32, index=index)}),
            ("held_store", lambda **kw: states.put(k, k, **kw), {}),
            ("held_load", lambda **kw: states.get(**kw), {"k_out": k, "v_out": _t(2, 70, 2, 64, index=index)}),
            ("held_attention_forward", lambda **kw: attend.forward(q, states, **kw), {"out": q})]


def test_calls_make_the_device_of_their_tensors_current(lone):
    """A launch goes to the current device, and torch's default stream is handle 0 on
    every one: without the switch the kernel would run on another GPU."""
    at = []
    lib = Recorder(lambda name, args: at.append((name, lone["current"], args[-1])))
    for index in (1, 0):
        for name, call, outputs in _calls(lib, index):
            for kw in (outputs, outputs, dict(outputs, stream=7)):
                at.clear()
                call(**kw)
                assert at == [(name, index, kw.get("stream", 1000 + index))]
                assert lone["current"] == 0

    def fails(name, args):
        raise RuntimeError(name)
    for _, call, outputs in _calls(Recorder(fails), 1):
        with pytest.raises(RuntimeError):
            call(**outputs)
        assert lone["current"] == 0


def test_a_stream_of_its_own_needs_outputs(lone):
    """Memory allocated in the call belongs to torch's current stream: a kernel on
    another stream could write it while freed work of the current one still uses it."""
    lib = Recorder()
    for _, call, outputs in _calls(lib):
        if outputs:
            with pytest.raises(ValueError, match="stream"):
                call(stream=5)
    assert not lib.calls
    norm = isa.BlockNorm(64)
    norm._lib = lib
    x = _t(2, 5, 64)
    for kw in ({}, {"out": x}, {"x_out": x}):
        with pytest.raises(ValueError, match="stream"):
            norm.apply(x, x, stream=5, **kw)
    assert not lib.calls


def test_a_workspace_with_gaps_or_repeats_is_refused(lone):
    """The kernels take consecutive bytes from the workspace's base, whatever the
    tensor's strides say: one byte repeated counts as enough, and is not."""
    x, w = _t(1, 300, 4096), _t(1024, 4096)
    dense, states = isa.Dense(x, w), _held(1, 40000, 1, 128)
    q = _t(1, 1, 8, 128)
    attend = isa.HeldAttention(q, states)
    for plan, call in ((dense, lambda ws: dense.forward(x, w, workspace=ws)),
                       (attend, lambda ws: attend.forward(q, states, workspace=ws))):
        plan._lib = Recorder()
        need = plan.workspace_bytes
        assert need > 0
        call(torch.zeros(need, dtype=torch.uint8))
        call(torch.zeros((need + 3) // 4, dtype=torch.float32))
        for bad in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)
        with pytest.raises(TypeError, match="workspace"):
            call(need)
        assert len(plan._lib.calls) == 2


def test_a_missing_output_has_room_for_what_the_plan_writes(lone):
    """Plans made for slices of wider tensors, called without them."""
    x, w = _t(2, 5, 64), _t(32, 64)
    wide = torch.zeros(2, 5, 96, dtype=torch.float16)[:, :, 32:64]
    plan = isa.Dense(x, w, wide)
    plan._lib = Recorder()
    got = plan.forward(x, w)
    room = got.untyped_storage().nbytes() // 2 - got.storage_offset()
    assert tuple(plan._desc.out_stride) == got.stride()[:2]
    assert _span(got.shape, got.stride()) <= room
    q, states = _t(2, 5, 4, 64), _held()
    wide = torch.zeros(2, 5, 12, 64, dtype=torch.float16)[:, :, 4:8]
    plan = isa.HeldAttention(q, states, wide)
    plan._lib = Recorder()
    got = plan.forward(q, states)
    room = got.untyped_storage().nbytes() // 2 - got.storage_offset()
    assert tuple(plan._desc.out_stride) == got.stride()[:3]
    assert _span(got.shape, got.stride()) <= room
    # the norm's outputs are dense, whatever x is
    norm = isa.BlockNorm(32)
    norm._lib = Recorder()
    x = gpu(torch.zeros(2, 5, 96, dtype=torch.float16)[:, :, 32:64])
    x_out, out = norm.apply(x, x)
    for t, rows in ((x_out, norm._lib.calls[0][1][0].x_out), (out, norm._lib.calls[0][1][0].out)):
        assert t.is_contiguous() and (rows.batch_stride, rows.row_stride) == t.stride()[:2]


def test_layouts_seen_before_do_not_pass_for_others(lone):
    """A call's layout is checked once; another in any of its parts is checked again."""
    k, lengths, mask = _t(2, 70, 2, 64), _t(2, dtype=torch.int32), _t(2, 70, dtype=torch.bool)
    states = _held()
    states.put(k, k, 0, mask, lengths)
    for bad in (dict(at=32), dict(key_mask=_t(2, 71, dtype=torch.bool)), dict(key_lengths=_t(3, dtype=torch.int32)),
                dict(key_lengths=_t(2, dtype=torch.int64)), dict(key_mask=_t(70, 2, dtype=torch.bool).t())):
        with pytest.raises((ValueError, TypeError)):
            states.put(k, k, **dict({"key_mask": mask, "key_lengths": lengths}, **bad))
    assert len(states._lib.calls) == 1
    states.get(32, 38, k_out=_t(2, 38, 2, 64), v_out=_t(2, 38, 2, 64))
    for at, length in ((33, 38), (-1, 38), (32, 39), (32, -38)):
        with pytest.raises(ValueError):
            states.get(at, length, k_out=_t(2, 38, 2, 64), v_out=_t(2, 38, 2, 64))
    assert len(states._lib.calls) == 2


def test_a_plan_serves_tensors_that_differ_in_strides_of_single_steps(lone):
    """The stride of a dimension of one element says nothing."""
    x, w = _t(1, 5, 64), _t(32, 64)
    plan = isa.Dense(x, w)
    plan._lib = Recorder()
    plan.forward(gpu(torch.zeros(1, 5, 64, dtype=torch.float16).as_strided((1, 5, 64), (8, 64, 1))), w)
    assert len(plan._lib.calls) == 1
    with pytest.raises(ValueError, match="the plan is for"):
        plan.forward(_t(1, 5, 128)[:, :, :64], w)


def test_sizes_beyond_the_descriptors_are_refused():
    """The C descriptors hold sizes as int: larger ones would be cut to their low 32
    bits and a part of the tensor would be left out, without an error."""
    def meta(*shape, dtype=torch.float16):
        return torch.empty(shape, dtype=dtype, device="meta")
    big = 2 ** 32 + 8
    for shape in ((big, 2, 8), (2, big, 8), (2 ** 31, 1, 8)):
        with pytest.raises(ValueError, match="2147483647"):
            isa.BlockNorm(8).apply(meta(*shape))
        with pytest.raises(ValueError, match="2147483647"):
            isa.Dense(meta(*shape), meta(16, 8))
    with pytest.raises(ValueError, match="2147483647"):
        isa.Dense(meta(1, 2, 8), meta(big, 8))
    with pytest.raises(ValueError, match="2147483647"):
        isa.Dense(meta(1, 2, big), meta(16, big))
    for sizes in ((big, 1, 1), (1, big, 1), (1, 1, big)):
        with pytest.raises(ValueError, match="2147483647"):
            isa.HeldStates(*sizes, 8, device="meta")
    states = isa.HeldStates(1, 70, 1, 8, device="meta")
    with pytest.raises(ValueError, match="2147483647"):
        isa.HeldAttention(meta(1, big, 1, 8), states)


def test_an_eps_that_fp32_rounds_to_0_is_refused():
    """eps is held in fp32: a positive one that becomes 0 turns rows of zeros into NaN."""
    with pytest.raises(ValueError, match="eps"):
        isa.BlockNorm(8, eps=1e-50)
    isa.BlockNorm(8, eps=1e-44)


@pytest.mark.parametrize("scale", [1e-46, 1e39, float("nan"), float("inf")])
def test_factors_outside_the_range_of_fp32_are_refused(lone, scale):
    with pytest.raises((ValueError, isa.ImgStencilError)):
        isa.HeldAttention(_t(2, 5, 4, 64), _held(), scale=scale)
    if scale != 1e-46:      # a residual scale that becomes 0 is one that adds nothing
        with pytest.raises((ValueError, isa.ImgStencilError)):
            isa.BlockNorm(64, residual_scale=scale).apply(_t(2, 5, 64), _t(2, 5, 64), out=_t(2, 5, 64), x_out=_t(2, 5, 64))
