"""What the attention binding hands to the library, on the CPU: tensors that pass
for device tensors and a library that records its calls in place of launching."""
import pytest
import torch

import image_stencil_amd as isa
from image_stencil_amd import attention


class OnGpu(torch.Tensor):
    """A host tensor that says it lies on GPU `index`."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index

    __torch_function__ = torch._C._disabled_torch_function_impl


def gpu(t, index=0):
    t = torch.Tensor._make_subclass(OnGpu, t)
    t.index = index
    return t


class Recorder:
    """Stands in for the library: every function records its arguments."""

    def __init__(self, on_call=None):
        self.calls, self.on_call = [], on_call

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            if self.on_call:
                self.on_call(name, args)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    """One machine with GPUs 0 (current) and 1; current streams 1000 and 1001."""
    state = {"current": 0}

    class Device:
        def __init__(self, index):
            self.index = index.index if isinstance(index, torch.device) else index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *exc):
            state["current"] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", Device)
    # Every given tensor passes for one of the same device, allocated ones too.
    monkeypatch.setattr(attention, "_one_device", lambda tensors: True)
    return state


def _t(*shape, dtype=torch.float16, index=0):
    return gpu(torch.zeros(shape, dtype=dtype), index)


def _span(shape, stride):
    """Elements from the first to the end of the last."""
    return 1 + sum((n - 1) * s for n, s in zip(shape, stride))


def test_a_missing_output_has_room_for_what_the_plan_writes(fake):
    """A plan made for a slice of a wider tensor, called without that tensor: the
    memory that is allocated holds every element the plan's strides reach."""
    n, lq, heads, d = 2, 5, 4, 64
    q, k = _t(n, lq, heads, d), _t(n, 7, heads, d)
    wide = torch.zeros(n, lq, 3 * heads, d, dtype=torch.float16)[:, :, heads:2 * heads]
    for out in (wide, wide.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), None):
        plan = isa.CrossAttention(q, k, k, out)
        plan._lib = Recorder()
        got = plan.forward(q, k, k)
        assert got.shape == q.shape
        strides = tuple(plan._desc.out_stride) + (1,)
        room = got.untyped_storage().nbytes() // 2 - got.storage_offset()
        assert _span(got.shape, strides) <= room, "writes %d elements into %d" % (_span(got.shape, strides), room)
        assert got.stride() == strides     # and it is read as it was written
        assert plan._lib.calls[-1][1][6] == got.data_ptr()


def test_a_workspace_with_gaps_or_repeats_is_refused(fake):
    """The kernel takes consecutive bytes from the workspace's base, whatever the
    tensor's strides say: one byte repeated counts as enough, and is not."""
    q, k = _t(1, 1, 8, 128), _t(1, 40000, 1, 128)
    plan = isa.CrossAttention(q, k, k)
    plan._lib = Recorder()
    need = plan.workspace_bytes
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8)
    plan.forward(q, k, k, workspace=ws)
    plan.forward(q, k, k, workspace=torch.zeros((need + 3) // 4, dtype=torch.float32))
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            plan.forward(q, k, k, workspace=bad)
    with pytest.raises(TypeError, match="workspace"):
        plan.forward(q, k, k, workspace=need)
    assert len(plan._lib.calls) == 2


def test_rotary_on_a_stream_of_its_own_needs_outputs(fake):
    """Memory allocated in the call belongs to torch's current stream: a kernel on
    another stream could write it while freed work of the current one still uses it."""
    plan, x, pos = isa.Rotary(64), _t(2, 3, 4, 64), _t(2, 3, 1, dtype=torch.int32)
    plan._lib = Recorder()
    with pytest.raises(ValueError, match="stream"):
        plan.apply(x, pos, stream=5)
    for outs in ({}, {"q_out": x}, {"k_out": x}):
        with pytest.raises(ValueError, match="stream"):
            plan.apply_qk_norm(x, _t(2, 3, 4, 64), pos, stream=5, **outs)
    assert not plan._lib.calls
    plan.apply(x, pos, out=x, stream=5)
    y = _t(2, 3, 4, 64)
    plan.apply_qk_norm(x, y, pos, q_out=x, k_out=y, stream=5)
    assert [args[-1] for _, args in plan._lib.calls] == [5, 5]
    plan.apply(x, pos)
    plan.apply_qk_norm(x, y, pos)
    assert [args[-1] for _, args in plan._lib.calls[2:]] == [1000, 1000]


def test_calls_make_the_device_of_their_tensors_current(fake):
    """A launch goes to the current device, and torch's default stream is handle 0
    on every one: without the switch the kernel would run on another GPU."""
    at = []
    lib = Recorder(lambda name, args: at.append((name, fake["current"], args[-1])))
    r, x, pos = isa.Rotary(64), _t(2, 3, 4, 64, index=1), _t(2, 3, 1, dtype=torch.int32, index=1)
    c = isa.CrossAttention(x, x, x)
    r._lib = c._lib = lib
    r.apply(x, pos)
    r.apply_qk_norm(x, x, pos)
    c.forward(x, x, x)
    names = ["rotary_forward", "qk_norm_rotary_forward", "cross_attention_forward"]
    assert at == [(n, 1, 1001) for n in names]
    assert fake["current"] == 0
    # a stream of the caller's belongs to the tensors' device as well
    at.clear()
    r.apply(x, pos, out=x, stream=7)
    assert at == [("rotary_forward", 1, 7)] and fake["current"] == 0
    # and the device stays where it is for tensors of the current one
    at.clear()
    x, pos = _t(2, 3, 4, 64), _t(2, 3, 1, dtype=torch.int32)
    r.apply(x, pos)
    r.apply_qk_norm(x, x, pos)
    c.forward(x, x, x)
    assert at == [(n, 0, 1000) for n in names]

    def fails(name, args):
        raise RuntimeError(name)
    r._lib = Recorder(fails)
    with pytest.raises(RuntimeError):
        r.apply(_t(2, 3, 4, 64, index=1), _t(2, 3, 1, dtype=torch.int32, index=1))
    assert fake["current"] == 0


@pytest.mark.parametrize("scale", [1e-46, -1e-60, 1e39, float("nan"), float("inf")])
def test_a_factor_outside_the_range_of_fp32_is_refused(scale):
    """The factor is held in fp32, where a smaller one would become 0, which stands
    for 1 / sqrt(d)."""
    q, k = torch.zeros(2, 5, 4, 64, dtype=torch.float16), torch.zeros(2, 7, 4, 64, dtype=torch.float16)
    with pytest.raises((ValueError, isa.ImgStencilError)):
        isa.CrossAttention(q, k, k, scale=scale)


@pytest.mark.parametrize("scale", [1e-44, -1e-30, 2.3e38, -0.125])
def test_a_factor_of_fp32_is_kept(scale):
    q, k = torch.zeros(2, 5, 4, 64, dtype=torch.float16), torch.zeros(2, 7, 4, 64, dtype=torch.float16)
    assert isa.CrossAttention(q, k, k, scale=scale)._desc.scale == torch.tensor(scale, dtype=torch.float32).item()


def test_a_plan_serves_tensors_that_differ_in_strides_of_single_steps(fake):
    """The stride of a dimension of one element says nothing: a batch of one sliced
    out of a wider tensor, or a single token of a cache, lies as the plan expects."""
    q, k = _t(1, 5, 4, 64), _t(1, 1, 4, 64)
    plan = isa.CrossAttention(q, k, k, q)
    plan._lib = Recorder()
    q2 = gpu(torch.zeros(3, 5, 4, 64, dtype=torch.float16)[:, :, :][1:2].as_strided((1, 5, 4, 64), (7, 256, 64, 1)))
    k2 = gpu(torch.zeros(1, 9, 4, 64, dtype=torch.float16)[:, 3:4].as_strided((1, 1, 4, 64), (11, 1 << 30, 64, 1)))
    plan.forward(q2, k2, k2, q2)
    assert len(plan._lib.calls) == 1
    for bad in (_t(1, 5, 8, 64)[:, :, :4], _t(1, 4, 5, 64).transpose(1, 2)):
        with pytest.raises(ValueError, match="the plan is for"):
            plan.forward(bad, k, k, q)
    empty = _t(1, 0, 4, 64)
    plan = isa.CrossAttention(q, empty, empty, q)
    plan._lib = Recorder()
    plan.forward(q, empty.as_strided((1, 0, 4, 64), (64, 256, 128, 1)), empty, q)
    assert len(plan._lib.calls) == 1


def test_sizes_beyond_the_descriptors_are_refused():
    """The C descriptors hold sizes as int: larger ones would be cut to their low
    32 bits and a part of the tensor would be left out, without an error."""
    def meta(*shape, dtype=torch.float16):
        return torch.empty(shape, dtype=dtype, device="meta")
    r = isa.Rotary(64)
    for n, length, heads in ((2 ** 32 + 2, 3, 4), (2, 2 ** 32 + 3, 4), (2, 3, 2 ** 32 + 4), (2 ** 31, 1, 1)):
        x, pos = meta(n, length, heads, 64), meta(n, length, 1, dtype=torch.int32)
        for call in (lambda: r.apply(x, pos), lambda: r.apply_qk_norm(x, meta(1, 1, 1, 64), pos, pos[:1, :1]),
                     lambda: r.apply_qk_norm(meta(1, 1, 1, 64), x, pos[:1, :1], pos)):
            with pytest.raises(ValueError, match="2147483647"):
                call()
    big = 2 ** 32 + 1
    for q, k in ((meta(big, 1, 1, 64), meta(big, 2, 1, 64)), (meta(1, big, 1, 64), meta(1, 2, 1, 64)),
                 (meta(1, 1, 1, 64), meta(1, big, 1, 64)), (meta(1, 1, big, 64), meta(1, 2, 1, 64))):
        with pytest.raises(ValueError, match="2147483647"):
            isa.CrossAttention(q, k, k)


def test_an_eps_that_fp32_rounds_to_0_is_refused():
    """eps is held in fp32: a positive one that becomes 0 turns heads of zeros into
    NaN."""
    r, x, pos = isa.Rotary(64), torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="eps"):
        r.apply_qk_norm(x, x, pos, eps=1e-50)
    for eps in (0.0, 1e-44, 1e-6):
        with pytest.raises(TypeError, match="on a GPU"):   # past the check
            r.apply_qk_norm(x, x, pos, eps=eps)


def test_a_magnitude_outside_the_range_of_fp32_is_refused():
    """The magnitude is used in fp32: one that becomes 0 or infinite there turns
    all that it multiplies into that, or NaN."""
    for magnitude in (1e-46, 1e39):
        with pytest.raises(isa.ImgStencilError):
            isa.Rotary(64, magnitude=magnitude)
    isa.Rotary(64, magnitude=1e-30)
    isa.Rotary(64, magnitude=1e38)
