"""Which keys cross attention adds up, counted: queries of zeros give every
visible key the weight 1, so that the log-sum-exp is the logarithm of their number
and values that mark tiles or places are their shares. A single key that is lost
or taken twice shows among tens of thousands, where random data hides it in the
rounding of long sums."""
import math

import pytest
import torch

import image_stencil_amd as isa
from gpu_util import say

F16, BF16 = torch.float16, torch.bfloat16

# Weights of 1 and counts below 2^24 are exact in 32 bits. What is not: 1 / l and
# its product (2 roundings), and where keys are split over workgroups the
# logarithms of up to 2^16 in each part (off by 2^-23 * 16, and as much again in
# the difference to the largest), the weights 2^x made of them (ln 2 times that),
# sums of at most 128 parts (2^-24 each) and the last logarithm: together less
# than 2^-18 + 2^-17 of a share, and of the logarithm.
SLACK = 2.0 ** -16

# few queries over long keys: own tiles, split over workgroups and not; queries
# in the hundreds: shared tiles; many row tiles over few keys: kept keys.
SHAPES = [(1, 1, 40000, 8, 1, 128), (3, 2, 9001, 4, 4, 64), (1, 3, 20011, 2, 2, 256), (1, 130, 9001, 1, 1, 40),
          (1, 40, 16384, 1, 1, 128), (2, 1, 1000, 4, 2, 64), (2, 5, 333, 2, 1, 96), (1, 1, 33, 1, 1, 32),
          (2, 300, 1543, 2, 1, 96), (2, 300, 700, 2, 2, 64), (4, 4000, 200, 8, 8, 40), (1, 1000, 20011, 2, 2, 160)]


def _sees(n, lk):
    """Visible keys: all; a mask with a part left empty as a whole and the last key
    visible; lengths."""
    g = torch.Generator().manual_seed(lk)
    mask = torch.rand(n, lk, generator=g) < 0.5
    mask[:, lk // 3:] = False
    mask[:, -1] = True
    lengths = torch.tensor([max(1, lk - 37), lk // 2, 1, 0][:n], dtype=torch.int32)
    everywhere = torch.ones(n, lk, dtype=torch.bool)
    return [("all", everywhere, None, None), ("mask", mask, mask, None),
            ("lengths", torch.arange(lk)[None] < lengths[:, None], None, lengths)]


def _marks(lk, d, kind):
    """lk x d values: element e marks the tiles of 32 keys with that number, or the
    places in them (numbers modulo d)."""
    j = torch.arange(lk)
    number = j // 32 if kind == "tile" else j
    return (number[:, None] % d == torch.arange(d)[None]).double()


def _shares(weight, marks):
    """weight: n x lk, how often a key is added. Returns n x d shares and n logarithms."""
    total = weight.sum(-1)
    return (weight @ marks) / total.clamp_min(1)[:, None], torch.log(total)


def _accepts(out, lse, see, marks, dtype):
    want, log = _shares(see.double(), marks)
    bound = torch.finfo(dtype).eps / 2 * want.clamp_min(torch.finfo(dtype).smallest_normal) + SLACK * want
    lse_ok = (lse == log) | ((lse - log).abs() <= SLACK)
    return bool(((out - want).abs() <= bound).all()) and bool(lse_ok.all())


@pytest.mark.parametrize("n,lq,lk,hq,hkv,d", SHAPES)
def test_a_lost_or_doubled_tile_is_seen(n, lq, lk, hq, hkv, d):
    """On the CPU: exact results pass, the same with one tile of 32 keys left out or
    taken twice, or with one key, do not."""
    for dtype in (F16, BF16):
        for label, see, _, _ in _sees(n, lk):
            for kind in ("tile", "place"):
                marks = _marks(lk, d, kind)
                out, lse = _shares(see.double(), marks)
                assert _accepts(out.to(dtype).double(), lse.float().double(), see, marks, dtype)
                for b in range(n):
                    at = torch.nonzero(see[b]).flatten()
                    for key in at[[0, len(at) // 2, -1]].tolist() if len(at) else []:
                        for first, last in ((key // 32 * 32, key // 32 * 32 + 32), (key, key + 1)):
                            for times in (0.0, 2.0):
                                weight = see.double()
                                weight[b, first:last] *= times
                                out, lse = _shares(weight, marks)
                                assert not _accepts(out.to(dtype).double(), lse.float().double(), see, marks,
                                                    dtype), (label, kind, b, key, times)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,lq,lk,hq,hkv,d", SHAPES)
def test_every_visible_key_counts_once(n, lq, lk, hq, hkv, d, dtype):
    say("counts", dtype, n, lq, lk, hq, hkv, d)
    q = torch.zeros(n, lq, hq, d, dtype=dtype, device="cuda")
    k = torch.randn(n, lk, hkv, d, generator=torch.Generator().manual_seed(d)).to(dtype).cuda()
    for label, see, mask, lengths in _sees(n, lk):
        for kind in ("tile", "place"):
            marks = _marks(lk, d, kind)
            v = marks.to(dtype).cuda()[None, :, None].expand(n, lk, hkv, d).contiguous()
            out, lse = isa.cross_attention(q, k, v, None if mask is None else mask.cuda(),
                                           None if lengths is None else lengths.cuda(), return_lse=True)
            out, lse = out.cpu().double(), lse.cpu().double()
            # every row and head alike, to the bit
            assert (out == out[:, :1, :1]).all() and (lse == lse[:, :1, :1]).all(), (label, kind)
            assert _accepts(out[:, 0, 0], lse[:, 0, 0], see, marks, dtype), (label, kind)
