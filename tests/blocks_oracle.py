"""Plain 64-bit forms of the operators around attention, with the error bounds of the
kernels. CPU tensors in, float64 out; written from the formulas of
include/imgstencil.h, sharing no code with the library.
"""
import math

import torch

from attention_oracle import U, UM, half, norm_error, rounding  # noqa: F401

BLOCK = 32


# ------------------------------------------------------- sum and norm of a block
def _normed(x, kind, eps):
    """(normed x, its scale: |x| (layer: and the mean of |x|) over the root)."""
    size = x.abs()
    if kind == "layer":
        size = size + size.mean(-1, keepdim=True)
        x = x - x.mean(-1, keepdim=True)
    inv = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * inv, size * inv, inv


def _row(t, like):
    return None if t is None else t.double()[:, None].expand(-1, 1, -1)


def block_norm(x, y=None, norm="rms", post=None, eps=1e-6, residual_scale=1.0, gate=None, post_weight=None, weight=None,
               bias=None, scale=None, shift=None):
    """(x_out, bound, out, bound); None where absent. Bounds to first order, with a
    hundredth on top for the rest.

    What multiplies y per channel is the product of up to three factors (2 U), and its
    product and sum take U each. An error e of the summed stream reaches the normed value
    directly, through the mean (layer) and through the root, which takes its
    mean square: |normed| * rms(e) * inv. The factor w (1 + scale) is two roundings, the
    term shift + bias one, product and sum one each."""
    dtype, c = x.dtype, x.shape[-1]
    x = x.double()
    err = torch.zeros_like(x)
    if y is not None:
        y = y.double()
        h, size, e_post = y, y.abs(), 0.0
        if post is not None:
            h, size, _ = _normed(y, post, eps)
            e_post = norm_error(c, post)
        g = residual_scale * torch.ones(1, 1, c, dtype=torch.float64)
        if post_weight is not None:
            g = g * post_weight.double()
        if gate is not None:
            g = g * _row(gate, x)
        x = x + g * h
        err = 1.01 * ((e_post + 3 * U) * size * g.abs() + U * (x.abs() + (g * h).abs()))
    x_bound = err + rounding(x, dtype) * 1.01
    if norm is None:
        return x, x_bound, None, None
    n, size, inv = _normed(x, norm, eps)
    spread = err + (err.mean(-1, keepdim=True) if norm == "layer" else 0.0)
    n_err = norm_error(c, norm) * size + spread * inv + n.abs() * torch.sqrt((spread * spread).mean(-1, keepdim=True)) * inv
    a = torch.ones(1, 1, c, dtype=torch.float64) if weight is None else weight.double()[None, None]
    b = torch.zeros(1, 1, c, dtype=torch.float64)
    b_size = b
    if scale is not None:
        a = a * (1.0 + _row(scale, x))
        # 1 + scale is rounded against its own size
    if shift is not None:
        b, b_size = b + _row(shift, x), b_size + _row(shift, x).abs()
    if bias is not None:
        b, b_size = b + bias.double()[None, None], b_size + bias.double().abs()[None, None]
    z = n * a + b
    bound = 1.01 * (n_err * a.abs() + 3 * U * (n * a).abs() + 2 * U * (b_size + z.abs())) + rounding(z, dtype) * 1.01
    return x, x_bound, z, bound


# ------------------------------------------------------------------ dense layers
def activate(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _activation_error(z, act):
    """How far the kernel's activation of z itself may be off. gelu: its tail |z|
    Phi(-|z|) by the polynomial (4.7e-6), the exponent's argument z^2 / 2 (three
    roundings of it) and 12 U for the hardware's reciprocal and exponential, products and
    sums; beyond 14 the tail is under 1e-43. The others: the exponent's argument u (five
    roundings of it) and 12 U."""
    if act == "gelu":
        t = z.abs().clamp_max(14.0)
        tail = t * 0.5 * torch.erfc(t / math.sqrt(2.0))
        return (4.7e-6 + 1.5 * z.clamp(-14, 14) ** 2 * U + 12 * U) * tail + 2 * U * activate(z, act).abs() + 1e-38
    if act in ("gelu_tanh", "silu"):
        u = z if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)
        return (5 * u.abs().clamp_max(200.0) + 12) * U * activate(z, act).abs() + 1e-37
    return 0.0


SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "gelu_tanh": 1.14, "silu": 1.1}   # largest derivatives


def dense(x, w, bias=None, activation="none", residual=None):
    """(out, bound): sums of k products in fp32 on the matrix cores, in any order and in
    parts; bias, activation, residual; one rounding."""
    dtype, k = x.dtype, x.shape[-1]
    x, w = x.double(), w.double()
    z, m = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, m = z + bias.double(), m + bias.double().abs()
    err = (k + 24) * UM * m
    out = activate(z, activation)
    err = SLOPE[activation] * err + _activation_error(z, activation)
    if residual is not None:
        out = out + residual.double()
    return out, 1.01 * (err + U * out.abs()) + (1 + U) * rounding(out, dtype)


# -------------------------------------------------------------- states in 8 bits
def _e4m3():
    """The non-negative e4m3 numbers, in order."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:-1], dtype=torch.float64)     # the last code is NaN


E4M3 = _e4m3()


def nearest_e4m3(u):
    """The nearest number of the table, ties to the even code; |u| <= 448."""
    a = u.abs()
    hi = torch.searchsorted(E4M3, a).clamp_max(len(E4M3) - 1)
    lo = (hi - 1).clamp_min(0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    pick = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    return torch.sign(u) * E4M3[pick]


def held(x, seen=None):
    """x (n x len x heads x d, stored from a block's start) as the states hold it, in
    64 bits; seen: n x len truth values or None."""
    n, length, heads, d = x.shape
    most = torch.finfo(x.dtype).max
    y = x.double().clone()
    if seen is not None:
        y[~seen] = 0.0
    for at in range(0, length, BLOCK):
        part = y[:, at:at + BLOCK]
        finite = torch.where(torch.isfinite(part), part.abs(), torch.zeros_like(part))
        for b in range(n):
            for h in range(heads):
                top, e = float(finite[b, :, h].max()), -120
                while top > 448.0 * 2.0 ** e:
                    e += 1
                p = part[b, :, h]
                q = nearest_e4m3(torch.where(torch.isfinite(p), p, torch.zeros_like(p)) / 2.0 ** e) * 2.0 ** e
                q = torch.where(q.abs() > most, torch.sign(q) * 240.0 * 2.0 ** e, q)
                part[b, :, h] = torch.where(torch.isfinite(p), q, torch.full_like(q, math.nan))
    return y
