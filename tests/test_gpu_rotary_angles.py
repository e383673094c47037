"""Rotary angles on the GPU against exact ones: frequencies from 60-digit
arithmetic, positions times frequencies as integers of 2^-120 turns, so that the
comparison has no rounding of its own at any position."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

import attention_oracle as ao
import image_stencil_amd as isa
from gpu_util import say

ONE = 1 << 120


def _pi():
    """By Machin's formula."""
    def arctan_of_inverse(n):
        total = term = Decimal(1) / n
        k = 1
        while abs(term) > Decimal(10) ** -62:
            term = -term / (n * n)
            k += 2
            total += term / k
        return total
    return 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))


def _turns(rot, base, scaling, factor, original_len):
    """Each pair's turns per position in units of 1 / ONE."""
    getcontext().prec = 60
    two_pi, per, base, factor = 2 * _pi(), rot // 2, Decimal(base), Decimal(factor)
    if scaling == "ntk":
        base *= factor ** (Decimal(per) / (per - 1))
    out = []
    for i in range(per):
        f = base ** (Decimal(-i) / per)
        if scaling == "linear":
            f /= factor
        elif scaling == "ramp":
            keep = min(max((original_len * f / two_pi - 1) / 31, Decimal(0)), Decimal(1))
            f = f * keep + f / factor * (1 - keep)
        out.append(int(f / two_pi * ONE))
    return out


def test_exact_turns_of_a_known_pair():
    """One radian per position is 0.159154943091895335768883763... turns."""
    t = _turns(4, 10000, "none", 1, 0)
    assert abs(t[0] / ONE - 0.15915494309189535) < 1e-17
    assert str(_pi()).startswith("3.14159265358979323846264338327950288419716939937510")
    assert abs(t[1] / t[0] - 0.01) < 1e-17


@pytest.mark.gpu
@pytest.mark.parametrize("most", [1000, 2 ** 23, 2 ** 31 - 1])
@pytest.mark.parametrize("rot,base,scaling", [(256, 10000, "none"), (96, 500000, "none"), (96, 10000, "linear"),
                                              (96, 500000, "ntk"), (128, 10000, "ramp")])
def test_angles_keep_their_bits_at_any_position(rot, base, scaling, most):
    """Pairs (1, 0) turn into the cosine and the sine themselves. The angle is off by
    2^-53 of itself (the frequency's rounding to 64 bits; 2^-59 for what led to it
    in 80) and, when its rest is rounded to 32 bits, by 2^-24 of that, 2^-26 turns
    at most; the sine by its own error. Where the rest is small the first shows
    alone."""
    say("angles", rot, base, scaling, most)
    g = torch.Generator().manual_seed(most % 1000003)
    pos = torch.randint(most // 2, most, (1, 4096, 1), generator=g)
    pos[:, ::2] *= -1
    pos[0, 0], pos[0, 1] = -most - 1, most
    turns = _turns(rot, base, scaling, 8, 2048)
    rest = torch.tensor([[((p * t + ONE // 2) % ONE - ONE // 2) / ONE for t in turns] for p in pos.flatten().tolist()],
                        dtype=torch.float64)
    whole = pos[0].double().abs() * torch.tensor([t / ONE for t in turns], dtype=torch.float64)[None]
    x = torch.zeros(1, pos.shape[1], 1, rot)
    x[..., :rot // 2] = 1
    plan = isa.Rotary(rot, base=float(base), scaling=scaling, factor=8.0, original_len=2048)
    y = plan.apply(x.cuda(), pos.to(torch.int32).cuda()).cpu().double()[0, :, 0]
    cos, sin = torch.cos(2 * math.pi * rest), torch.sin(2 * math.pi * rest)
    angle = 2 * math.pi * (whole * (2.0 ** -53 + 2.0 ** -59) + rest.abs() * 2.0 ** -24 + 2.0 ** -53)
    for name, got, want, bound in (("cosine", y[:, :rot // 2], cos, angle + ao.SINE_ERROR),
                                   ("sine", y[:, rot // 2:], sin, angle + ao.SINE_ERROR)):
        assert ((got - want).abs() <= bound).all(), "%s off by %.2f U" % (name, ((got - want).abs().max() / ao.U).item())
    small = (rest.abs() < 2.0 ** -7) & (rest != 0)
    assert small.sum() > 100
    off = (y[:, rot // 2:] - sin).abs()[small] / (angle + ao.SINE_ERROR * sin.abs())[small]
    assert (off <= 1).all(), "small rests off by %.2f of the bound" % off.max().item()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("base", [1e-3, 1e-30, 1e-150, 1e300])
def test_frequencies_of_any_size_turn(dtype, base):
    """A base below 1 turns its pairs by more than a radian per position, beyond all
    bits of the angle: the pairs still turn, and keep their length."""
    x = torch.zeros(1, 64, 1, 64, dtype=dtype)
    x[..., :32] = 1
    pos = torch.arange(-2 ** 31, 2 ** 31, 2 ** 26, dtype=torch.int64).to(torch.int32)[None, :, None]
    y = isa.Rotary(64, base=base).apply(x.cuda(), pos.cuda()).cpu().double()[0, :, 0]
    length = y[:, :32] ** 2 + y[:, 32:] ** 2
    assert ((length - 1).abs() <= 4 * (ao.SINE_ERROR + ao.half(dtype))).all()
