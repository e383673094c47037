"""Plain 64-bit forms of the attention operators, with the error bounds of the
kernels. CPU tensors in, float64 out; written from the formulas of
include/imgstencil.h, sharing no code with the library.
"""
import math

import torch

U = 2.0 ** -24           # half a step of fp32
UM = 2.0 ** -23          # the same for a sum on the matrix cores (directed rounding allowed)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(y, dtype):
    """How far y may move when it is rounded to dtype: half a step, which below
    the smallest normal number no longer shrinks with y."""
    f = torch.finfo(dtype)
    return (f.eps / 2) * y.abs().clamp_min(f.smallest_normal)


# Largest error of a sine or cosine given an angle in turns (measured over 2^22
# angles: 2.1 U the hardware's, for 16-bit data, and 0.9 U sincospi's, for fp32).
SINE_ERROR = 4 * U


def frequencies(rot, axes, base=10000.0, scaling="none", factor=1.0, original_len=0, ramp=(1.0, 32.0)):
    per = rot // 2 // axes
    if scaling == "ntk":
        base = base * factor ** (per / (per - 1))
    out = []
    for i in range(per):
        f = base ** (-i / per)
        if scaling == "linear":
            f = f / factor
        elif scaling == "ramp":
            turns = original_len / (2 * math.pi / f)
            share = min(max((turns - ramp[0]) / (ramp[1] - ramp[0]), 0.0), 1.0)
            f = (1 - share) * f / factor + share * f
        out.append(f)
    return out


def rotate(x, pos, rot, axes, layout, freqs, magnitude=1.0):
    """x: float64 n x len x heads x d; pos: n x len x axes. Returns (y, scale):
    the sum of the magnitudes of each element's terms."""
    n, length, heads, d = x.shape
    y, m = x.clone(), x.abs()
    pairs, per = rot // 2, rot // 2 // axes
    for p in range(pairs):
        angle = pos[:, :, p // per].double() * freqs[p % per]
        c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
        i, j = (p, p + pairs) if layout == "half" else (2 * p, 2 * p + 1)
        u, v = x[..., i].clone(), x[..., j].clone()
        y[..., i], y[..., j] = magnitude * (u * c - v * s), magnitude * (u * s + v * c)
        m[..., i] = m[..., j] = magnitude * (u.abs() + v.abs())
    return y, m


def rotary_bound(y, m, dtype):
    """Rounding of the result, plus per term: the angle (2 pi 2^-26 < 1.6 U), the
    sine, the magnitude (rounded and multiplied), the product and the sum."""
    return rounding(y, dtype) + (1.6 * U + SINE_ERROR + 4 * U) * (1 + half(dtype)) * m


def norm(x, w, eps, kind):
    """Returns (norm(x) * w, scale): the scale counts |x| (layer norm: and the
    mean of |x|) in place of x."""
    size = x.abs()
    if kind == "layer":
        size = size + size.mean(-1, keepdim=True)
        x = x - x.mean(-1, keepdim=True)
    inv = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * inv * w, size * inv * w.abs()


def norm_error(d, kind):
    """Relative error of a normed element in units of its scale: a sum of d
    squares in any order (half of it after the root), the division by d, eps,
    root, reciprocal and two products; layer norm: the mean's sum of d terms,
    which reaches the element and, twice, the variance."""
    e = (0.5 * (d + 4) + 6) * U
    return e if kind == "rms" else e + 3 * (d + 4) * U


def attention(q, k, v, scale, see=None):
    """q: n x lq x hq x d, k and v: n x lk x hkv x d (float64); see: n x lk truth
    values or None. Returns out, lse and what the bounds need: sum p |v|, the
    largest |score| error base (sum |q k| * scale), sum |v| over the row's keys."""
    n, lq, hq, d = q.shape
    lk, hkv = k.shape[1], k.shape[2]
    out = torch.zeros(n, lq, hq, d, dtype=torch.float64)
    pav, sav = out.clone(), out.clone()
    lse = torch.full((n, hq, lq), -math.inf, dtype=torch.float64)
    qk = torch.zeros(n, hq, lq, dtype=torch.float64)
    for b in range(n):
        at = torch.arange(lk) if see is None else torch.nonzero(see[b]).flatten()
        if at.numel() == 0:
            continue
        for h in range(hq):
            kk, vv = k[b, at, h // (hq // hkv)], v[b, at, h // (hq // hkv)]
            z = scale * (q[b, :, h] @ kk.T)
            qk[b, h] = (abs(scale) * (q[b, :, h].abs() @ kk.abs().T)).amax(-1)
            lse[b, h] = torch.logsumexp(z, -1)
            p = torch.exp(z - lse[b, h][:, None])
            out[b, :, h] = p @ vv
            pav[b, :, h] = p @ vv.abs()
            sav[b, :, h] = vv.abs().sum(0)
    return out, lse, pav, qk, sav


def attention_bounds(out, lse, pav, qk, sav, lk, d, dtype):
    """(bound on out, bound on lse). A score is a sum of d products in fp32 times
    the factor: off by at most delta = (d + 4) UM sum|q k|; it is read again in the
    exponent (UM of it, twice). p is rounded to the data type (below fp16's
    smallest normal by at most 2^-25 of the largest), the sums of lk terms run
    in fp32, the exponential and the logarithm are good to 4 UM, and the result
    is rounded."""
    h = half(dtype)
    delta = ((d + 4) * UM + 2 * UM) * qk
    every = (2 * delta + (2 * lk + 24) * UM).permute(0, 2, 1)[..., None]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    bound = rounding(out, dtype) + (1 + h) * ((h + every) * pav + tiny * sav)
    finite = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    return bound, delta + (lk + 12) * UM + 4 * UM * finite.abs()
