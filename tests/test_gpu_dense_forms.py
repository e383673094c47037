"""Every form of a dense layer's kernels on the GPU against the 64-bit form, each at a
shape whose plan is checked to be that form: ragged rows, features and inputs, ends,
strides, gapped entries, far arguments of the activations, neighbours that are no numbers,
graphs. HELD: how many tiles run at a time; with more, workgroups walk several."""
import pytest
import torch

import blocks_oracle as bo
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _check, _randn
from test_gpu_lds_poison import _poison_lib

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
HELD = {256: 256, 128: 512, 64: 1024}

# name: (n, rows, inputs, features), gap between entries, (kernel, tile), split, several tiles a workgroup
FEW, TILES = "is_k13_dense_few", "is_k13_dense"
FORMS = {
    "few 16 x 16": ((1, 9, 264, 70), 0, (FEW, (16, 16)), False, False),
    "few 32 x 16": ((1, 12, 72, 5003), 0, (FEW, (32, 16)), False, False),
    "few 32 x 32": ((1, 40, 264, 5461), 0, (FEW, (32, 32)), False, False),
    "64": ((1, 400, 136, 130), 0, (TILES, (64, 64)), False, False),
    "64, several": ((1, 27001, 40, 131), 0, (TILES, (64, 64)), False, True),
    "64, split": ((1, 100, 8192, 130), 0, (TILES, (64, 64)), True, False),
    "128": ((1, 9533, 72, 405), 0, (TILES, (128, 128)), False, False),
    "128, several": ((1, 11487, 104, 1103), 0, (TILES, (128, 128)), False, True),
    "128, split": ((1, 200, 4104, 3001), 0, (TILES, (128, 128)), True, False),
    "256": ((1, 6000, 1000, 1500), 0, (TILES, (256, 256)), False, False),
    "256, odd": ((1, 5001, 520, 3001), 0, (TILES, (256, 256)), False, False),
    "256, several": ((1, 19855, 136, 1275), 0, (TILES, (256, 256)), False, True),
    "256, entries": ((2, 5001, 1000, 1501), 16, (TILES, (256, 256)), False, False),
    "256, entries, several": ((2, 9000, 264, 1501), 16, (TILES, (256, 256)), False, True),
}
# One shape of every kernel and end, for what does not depend on how many tiles there are.
KERNELS = ["few 16 x 16", "few 32 x 16", "few 32 x 32", "64", "64, split", "128", "128, split", "256, odd"]


def _is(plan, name):
    _, _, form, split, several = FORMS[name]
    info = plan.info()
    say("dense form", name, info["kernel"], info["tile"], info["grid"])
    assert (info["kernel"], info["tile"]) == form
    assert (info["grid"][1] > 1) == split
    if form[0] == TILES:
        assert (info["grid"][0] * info["grid"][1] > HELD[form[1][0]]) == several


def _case(name, dtype, seed=0):
    """x (entries with the form's gap between them), w, bias, residual on the CPU."""
    (n, rows, k, m), gap = FORMS[name][:2]
    x = torch.zeros(n, rows * k + gap, dtype=dtype).as_strided((n, rows, k), (rows * k + gap, k, 1))
    x.copy_(_randn((n, rows, k), dtype, 5 * seed))
    return (x, _randn((m, k), dtype, 5 * seed + 1, 1.5 / k ** 0.5), 0.5 * _randn((m,), F32, 5 * seed + 2),
            _randn((n, rows, m), dtype, 5 * seed + 3))


def _cuda(t):
    """On the GPU with the same strides and gaps."""
    size = 1 + sum((s - 1) * d for s, d in zip(t.shape, t.stride()))
    y = torch.zeros(size, dtype=t.dtype, device="cuda").as_strided(t.shape, t.stride())
    return y.copy_(t)


@pytest.mark.parametrize("dtype,act,bias,residual", [(BF16, "gelu_tanh", True, False), (F16, "silu", True, True),
                                                     (BF16, "none", False, True), (F16, "gelu", False, False)])
@pytest.mark.parametrize("name", FORMS)
def test_forms(name, dtype, act, bias, residual):
    x, w, b, r = _case(name, dtype)
    b, r = b if bias else None, r if residual else None
    xd, wd, bd, rd = (None if t is None else _cuda(t) for t in (x, w, b, r))
    plan = isa.Dense(xd, wd, residual=rd, activation=act)
    _is(plan, name)
    got = plan.forward(xd, wd, bd, rd)
    _check(got, *bo.dense(x, w, b, act, r), name)
    for _ in range(2):
        assert torch.equal(got, plan.forward(xd, wd, bd, rd))      # no order of sums that varies


def test_several_tiles_and_parts_a_workgroup():
    """One feature of many rows: 64 x 64 tiles, more parts than run at a time. Small whole
    numbers, so that every sum is exact."""
    rows, k = 18382, 10752
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = (torch.randint(-4, 5, s, generator=g, device="cuda", dtype=torch.int8).to(F16) for s in ((1, rows, k), (1, k)))
    plan = isa.Dense(x, w)
    info = plan.info()
    say("dense tiles and parts", info)
    assert info["tile"] == (64, 64) and info["grid"][1] > 1 and info["grid"][0] * info["grid"][1] > HELD[64]
    assert torch.equal(plan.forward(x, w)[0], (x[0].float() @ w.float().t().contiguous()).to(F16))


@pytest.mark.parametrize("act,residual", [("relu", False), ("relu", True), ("none", False), ("gelu", True),
                                          ("gelu_tanh", True), ("silu", False)])
@pytest.mark.parametrize("name", ["256, odd", "128"])
def test_remaining_ends_of_large_tiles(name, act, residual):
    x, w, b, r = _case(name, F16, 1)
    r = r if residual else None
    plan = isa.Dense(x, w, residual=r, activation=act)
    _is(plan, name)
    got = plan.forward(x.cuda(), w.cuda(), b.cuda(), None if r is None else r.cuda())
    _check(got, *bo.dense(x, w, b, act, r), name)


@pytest.mark.parametrize("name", KERNELS)
def test_strides(name):
    """Slices of wider tensors, an output inside a larger one, rows at odd addresses, the
    residual in place; what lies around stays."""
    (n, rows, k, m), dtype = FORMS[name][0], F16
    x, w, b, r = _case(name, dtype, 2)
    exact = bo.dense(x, w, b, "silu", r)
    wide = torch.full((n, rows, 2 * k + 8), float("nan"), dtype=dtype, device="cuda")
    wide[:, :, k:2 * k] = x.cuda()
    ww = torch.full((m, k + 16), float("nan"), dtype=dtype, device="cuda")
    ww[:, 8:8 + k] = w.cuda()
    big = torch.full((n, rows + 1, m + 3), 5.0, dtype=dtype, device="cuda")
    res = torch.full((n, rows, m + 1), float("nan"), dtype=dtype, device="cuda")
    res[:, :, :m] = r.cuda()
    xs, ws, out, rs = wide[:, :, k:2 * k], ww[:, 8:8 + k], big[:, :rows, :m], res[:, :, :m]
    plan = isa.Dense(xs, ws, out=out, residual=rs, activation="silu")
    _is(plan, name)
    first = plan.forward(xs, ws, b.cuda(), rs, out).clone()
    _check(first, *exact, name)
    assert (big[:, rows:] == 5).all() and (big[:, :, m:] == 5).all()
    out.copy_(rs)
    plan = isa.Dense(xs, ws, out=out, residual=out, activation="silu")
    _is(plan, name)
    assert torch.equal(plan.forward(xs, ws, b.cuda(), out, out), first)
    assert (big[:, rows:] == 5).all() and (big[:, :, m:] == 5).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("name", KERNELS)
def test_far_arguments(name, act):
    """Far out on both sides, infinities (the limits) and NaN, in every feature block and
    the same in every row."""
    z = torch.tensor([-6e4, -300.0, -50.0, -20.0, -14.5, -13.0, -9.0, -6.0, -4.0, -1.0, -1e-3, 0.0, 1e-3, 1.0, 4.0, 9.0, 20.0,
                      300.0, 6e4, float("inf"), float("-inf"), float("nan")])
    n, rows, k, m = FORMS[name][0]
    at = torch.arange(m) % len(z)
    for dtype in (F16, BF16):
        x, w = torch.zeros(n, rows, k, dtype=dtype, device="cuda"), torch.zeros(m, k, dtype=dtype, device="cuda")
        plan = isa.Dense(x, w, activation=act)
        _is(plan, name)
        got = plan.forward(x, w, z[at].cuda())
        nan = (at == len(z) - 1)
        assert torch.isnan(got[..., nan.cuda()]).all()
        rest = got[..., ~nan.cuda()]
        assert torch.equal(rest, rest[:1, :1].expand_as(rest))
        want, bound = bo.dense(torch.zeros(1, 1, 8, dtype=dtype), torch.zeros(len(z), 8, dtype=dtype), z, act)
        if act not in ("none", "relu"):
            want[..., -2], want[..., -3] = 0.0, float("inf")
        most = torch.finfo(dtype).max
        v, t, e = rest[0, 0].cpu().double(), want[0, 0, at[~nan]], bound[0, 0, at[~nan]]
        good = (v == t) | ((v - t).abs() <= e) | ((t.abs() > most) & (v.abs() >= most) & (v.sign() == t.sign()))
        assert good.all(), (act, dtype, z[at[~nan]][~good], v[~good], t[~good])


@pytest.mark.parametrize("name", KERNELS + ["256, several", "256, entries, several"])
def test_rows_are_independent(name):
    """Neither a row's nor a feature's bits depend on neighbours that are no numbers."""
    x, w, b, r = (_cuda(t) for t in _case(name, BF16, 3))
    plan = isa.Dense(x, w, residual=r, activation="gelu")
    _is(plan, name)
    a = plan.forward(x, w, b, r)
    row, feature = x.shape[1] - 2, w.shape[0] // 2
    x[-1, row, 3], w[feature, 5] = float("nan"), float("nan")
    c = plan.forward(x, w, b, r)
    assert torch.isnan(c[-1, row]).all() and torch.isnan(c[..., feature]).all()
    for t in (a, c):
        t[-1, row] = 0
        t[..., feature] = 0
    assert torch.equal(a, c)


@pytest.mark.parametrize("name", ["few 32 x 32", "128, split", "256, odd", "256, several"])
def test_in_a_graph(name):
    x, w, b, r = (t.cuda() for t in _case(name, F16, 4))
    plan, out = isa.Dense(x, w, residual=r, activation="gelu"), torch.empty_like(r)
    _is(plan, name)
    ws = plan.new_workspace()
    plan.forward(x, w, b, r, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(x, w, b, r, out, ws)
    for seed in range(3):
        x.copy_(_randn(x.shape, F16, 70 + seed))
        want = plan.forward(x, w, b, r)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("name", KERNELS + ["256, several", "128, several", "256, entries"])
def test_lds_poison(name):
    """LDS that is read before it was written would put NaN into the results."""
    x, w, b, r = (_cuda(t) for t in _case(name, F16, 5))
    plan, poisoned = (isa.Dense(x, w, residual=r, activation="gelu") for _ in range(2))
    _is(plan, name)
    poisoned._lib = _poison_lib()
    assert torch.equal(plan.forward(x, w, b, r), poisoned.forward(x, w, b, r))
