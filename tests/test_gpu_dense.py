"""Dense layers on the GPU against the 64-bit form: rows from one to thousands around
every tile's edge, odd features, short and ragged inner sizes, every activation,
residuals, strides, entries that cannot be joined, split sums, graphs and streams."""
import itertools

import pytest
import torch

import blocks_oracle as bo
import image_stencil_amd as isa
from gpu_util import say
from test_gpu_cross_attention import _check, _randn

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _case(n, length, k, m, dtype, seed=0):
    return (_randn((n, length, k), dtype, 5 * seed), _randn((m, k), dtype, 5 * seed + 1, 1.5 / k ** 0.5),
            0.5 * _randn((m,), F32, 5 * seed + 2), _randn((n, length, m), dtype, 5 * seed + 3))


def _compare(n, length, k, m, dtype, act="none", bias=True, residual=True, seed=0):
    x, w, b, r = _case(n, length, k, m, dtype, seed)
    b, r = b if bias else None, r if residual else None
    got = isa.dense(x.cuda(), w.cuda(), None if b is None else b.cuda(), act, None if r is None else r.cuda())
    want, bound = bo.dense(x, w, b, act, r)
    _check(got, want, bound, "%d x %d, %d -> %d %s" % (n, length, k, m, act))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300])
def test_rows(rows, dtype):
    say("dense rows", rows, dtype)
    for k, m in ((64, 64), (200, 77), (1024, 300)):
        _compare(1, rows, k, m, dtype, "gelu", seed=rows)


@pytest.mark.parametrize("m", [1, 2, 7, 8, 15, 16, 17, 33, 63, 65, 127, 130, 255, 259, 777])
def test_features(m):
    say("dense features", m)
    for rows in (1, 20, 70, 400):
        _compare(1, rows, 136, m, BF16, "silu", seed=m)


@pytest.mark.parametrize("k", [8, 16, 24, 32, 40, 56, 64, 72, 120, 128, 136, 192, 248, 256, 264, 1000, 4104])
def test_inner_sizes(k):
    """Every remainder of a step of 64 inputs and of a chunk of 32."""
    say("dense inner", k)
    for rows in (3, 40, 130, 600):
        _compare(1, rows, k, 130, F16, seed=k)


@pytest.mark.parametrize("act,bias,residual", list(itertools.product(ACTS, [True, False], [True, False])))
def test_ends(act, bias, residual):
    say("dense end", act, bias, residual)
    for rows in (5, 90, 300):
        _compare(2, rows, 96, 50, F16, act, bias, residual, seed=rows)


@pytest.mark.parametrize("rows,k,m", [(2600, 512, 5000), (4099, 264, 1030), (3000, 1024, 2048), (16384, 64, 256)])
def test_large_tiles(rows, k, m):
    """Shapes that the largest tiles take, with edges inside them."""
    say("dense large", rows, k, m)
    plan = isa.Dense(torch.zeros(1, rows, k, dtype=BF16), torch.zeros(m, k, dtype=BF16))
    say(plan.info())
    _compare(1, rows, k, m, BF16, "gelu_tanh", seed=rows)


@pytest.mark.parametrize("rows,k,m", [(40, 8192, 64), (64, 4104, 24), (100, 8192, 130), (33, 16384, 8), (1, 16384, 8),
                                      (20, 8192, 16)])
def test_long_sums(rows, k, m):
    """Few tiles and long sums, which are split."""
    say("dense long sums", rows, k, m)
    for act, residual in (("none", False), ("gelu", True)):
        _compare(1, rows, k, m, F16, act, True, residual, seed=rows)
    x, w, b, r = (t.cuda() for t in _case(1, rows, k, m, F16))
    plan = isa.Dense(x, w, residual=r)
    if plan.workspace_bytes:
        guard = torch.full((plan.workspace_bytes + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        got = plan.forward(x, w, b, r, workspace=guard[:plan.workspace_bytes])
        assert torch.equal(got, plan.forward(x, w, b, r))      # no order of sums that varies
        assert (guard[plan.workspace_bytes:] == 0x5A).all()


def test_large_arguments_of_activations():
    """Far out on both sides, infinities (the limits) and NaN."""
    say("dense far activations")
    z = torch.tensor([-6e4, -300.0, -50.0, -20.0, -14.5, -13.0, -9.0, -6.0, -4.0, -1.0, -1e-3, 0.0, 1e-3, 1.0, 4.0, 9.0, 20.0,
                      300.0, 6e4, float("inf"), float("-inf"), float("nan")])
    w = torch.zeros(len(z), 8)
    for act in ACTS:
        for dtype in (F16, BF16):
            for rows in (1, 70):
                x = torch.zeros(1, rows, 8, dtype=dtype)
                got = isa.dense(x.cuda(), w.to(dtype).cuda(), z.cuda(), act).cpu()
                assert torch.equal(got, got[:, :1].expand_as(got).clone()) or torch.isnan(got).any()
                want, bound = bo.dense(x, w.to(dtype), z, act)
                if act not in ("none", "relu"):
                    want[..., -2] = 0.0      # the limit at -infinity
                    want[..., -3] = float("inf")
                for i in range(len(z) - 1):
                    v, t = got[0, 0, i].double(), want[0, 0, i]
                    most = torch.finfo(dtype).max
                    assert v == t or abs(v - t) <= bound[0, 0, i] or (abs(t) > most and abs(v) >= most), (act, z[i], v, t)
                assert torch.isnan(got[..., -1]).all(), act


@pytest.mark.parametrize("rows", [4, 100, 700])
def test_strides(rows):
    """Slices of wider tensors, transposed entries and rows, a repeated row, weights
    in a wider matrix, an output inside a larger one, the residual in place."""
    say("dense strides", rows)
    n, k, m = 3, 72, 50
    x, w, b, r = (t.cuda() for t in _case(n, rows, k, m, F16, seed=rows))
    exact = bo.dense(x.cpu(), w.cpu(), b.cpu(), "silu", r.cpu())

    def check(got, want=None):     # (another layout may take another kernel, and so other bits)
        _check(got, *(want or exact), "strides")
    wide = torch.zeros(n, rows, 2 * k + 8, dtype=F16, device="cuda")
    wide[:, :, k:2 * k] = x
    ww = torch.zeros(m, k + 16, dtype=F16, device="cuda")
    ww[:, 8:8 + k] = w
    big = torch.full((n, rows + 1, m + 3), 5.0, dtype=F16, device="cuda")
    out = big[:, :rows, :m]
    res = torch.zeros(n, rows, m + 1, dtype=F16, device="cuda")
    res[:, :, :m] = r
    plan = isa.Dense(wide[:, :, k:2 * k], ww[:, 8:8 + k], out=out, residual=res[:, :, :m], activation="silu")
    check(plan.forward(wide[:, :, k:2 * k], ww[:, 8:8 + k], b, res[:, :, :m], out))
    assert (big[:, rows:] == 5).all() and (big[:, :, m:] == 5).all()
    swapped = torch.zeros(rows, n, k, dtype=F16, device="cuda")     # rows of the entries alternate
    swapped.copy_(x.transpose(0, 1))
    check(isa.dense(swapped.transpose(0, 1), w, b, "silu", r))
    one = x[:1].cpu().repeat(n, 1, 1)                                # entries repeated
    check(isa.dense(x[:1].expand(n, -1, -1), w, b, "silu", r), bo.dense(one, w.cpu(), b.cpu(), "silu", r.cpu()))
    same = x[:, :1].cpu().repeat(1, rows, 1)                         # rows repeated
    check(isa.dense(x[:, :1].expand(-1, rows, -1), w, b, "silu", r), bo.dense(same, w.cpu(), b.cpu(), "silu", r.cpu()))
    place = r.clone()
    plan = isa.Dense(x, w, out=place, residual=place, activation="silu")
    check(plan.forward(x, w, b, place, place))


def test_rows_are_independent_and_repeatable():
    """A row's bits do not depend on its neighbours' values, nor on the run."""
    say("dense rows independent")
    for rows, k, m in ((20, 512, 640), (300, 512, 640)):
        x, w, b, r = (t.cuda() for t in _case(1, rows, k, m, BF16))
        a = isa.dense(x, w, b, "gelu", r)
        y = x.clone()
        y[0, 7] = float("nan")
        c = isa.dense(y, w, b, "gelu", r)
        keep = torch.arange(rows, device="cuda") != 7
        assert torch.equal(a[0, keep], c[0, keep]) and torch.isnan(c[0, 7]).all()
        for _ in range(3):
            assert torch.equal(a, isa.dense(x, w, b, "gelu", r))


def test_empty():
    w = torch.zeros(16, 64, dtype=F16, device="cuda")
    for n, length in ((0, 5), (3, 0)):
        assert isa.dense(torch.zeros(n, length, 64, dtype=F16, device="cuda"), w).shape == (n, length, 16)


@pytest.mark.parametrize("rows,k,m", [(1, 1024, 512), (100, 8192, 64), (300, 256, 512)])
def test_in_a_graph_and_on_streams(rows, k, m):
    say("dense graph", rows)
    x, w, b, r = (t.cuda() for t in _case(1, rows, k, m, F16))
    plan, out = isa.Dense(x, w, residual=r, activation="gelu"), torch.empty_like(r)
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
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    plan.forward(x, w, b, r, out, ws, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)
