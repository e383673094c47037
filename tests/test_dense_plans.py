"""Which form a dense layer's plan takes (host only): calls that no form may refuse."""
import pytest
import torch

import image_stencil_amd as isa

BF16 = torch.bfloat16


def _info(n, length, k, m, gap=0):
    x = torch.empty_strided((n, length, k), (length * k + gap, k, 1), dtype=BF16, device="meta")
    return isa.Dense(x, torch.empty((m, k), dtype=BF16, device="meta")).info()


@pytest.mark.parametrize("n,length,k,m", [(100000, 4, 128, 4096), (200000, 4, 64, 2048), (2 ** 20, 2, 8, 512),
                                          (2 ** 23 + 1, 2, 8, 8), (2 ** 23 + 1, 250, 64, 8)])
def test_many_entries_of_few_rows(n, length, k, m):
    """Entries with gaps between them, whose few-rows form would need 2^32 threads or more:
    the tiles take them, walking all entries with as many workgroups as run at a time."""
    info = _info(n, length, k, m, gap=8)
    assert info["kernel"] == "is_k13_dense"
    features, rows = info["tile"]
    assert info["grid"][0] == n * -(-length // rows) * -(-m // features) <= 2147483000


def test_entries_just_within_a_launch_keep_their_form():
    assert _info(60000, 4, 16, 4096, gap=8)["kernel"] == "is_k13_dense_few"
    assert _info(2 ** 23 - 1, 2, 8, 8, gap=8)["kernel"] == "is_k13_dense_few"
