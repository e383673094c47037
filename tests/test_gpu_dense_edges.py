"""Dense layers at the ends of what a plan takes."""
import pytest
import torch

import image_stencil_amd as isa
from gpu_util import say

pytestmark = pytest.mark.gpu
F16 = torch.float16


def test_a_sum_of_almost_2_to_the_31_inputs_in_parts():
    """The last of 16 parts ends before 2^31, where its nominal end does not fit an int. Ones
    at both ends of every part count each part once; ones behind both rows count nothing."""
    k, part = 2147483000, 134217728
    say("dense inputs", k)
    x, w = (torch.zeros(k + 1024, dtype=F16, device="cuda") for _ in range(2))
    for t in (x, w):
        t[k:] = 1.0
        for at in range(0, k, part):
            t[at], t[at + 63], t[min(k, at + part) - 1] = 1.0, 1.0, 1.0
    xs, ws = x[:k].view(1, 1, k), w[:k].view(1, k)
    plan = isa.Dense(xs, ws)
    assert plan.info()["grid"] == (1, 16, 1) and plan.info()["kernel"] == "is_k13_dense"
    assert plan.forward(xs, ws).item() == 48.0


def test_more_entries_than_a_launch_of_few_rows_holds():
    """2^23 + 1 entries of two rows with gaps: as many workgroups of few rows would be 2^32
    threads. Small whole numbers, so that every sum is exact."""
    n, k, m = 2 ** 23 + 1, 8, 8
    say("dense entries", n)
    g = torch.Generator(device="cuda").manual_seed(0)
    whole = torch.randint(-4, 5, (n, 3 * k), generator=g, device="cuda", dtype=torch.int8).to(F16)
    x = whole.as_strided((n, 2, k), (3 * k, k, 1))
    w = torch.randint(-4, 5, (m, k), generator=g, device="cuda", dtype=torch.int8).to(F16)
    plan = isa.Dense(x, w)
    assert plan.info()["kernel"] == "is_k13_dense"
    got = plan.forward(x, w)
    assert torch.equal(got.view(2 * n, m), torch.matmul(x.reshape(2 * n, k).float(), w.float().t().contiguous()).to(F16))
