"""A transformer block between two convolution layers that attends to a reference frame
whose states are held in 8 bits.

    reference -> 5x5 layer -> norm -> k, v (dense) -> k: norm, rotation -> held in 8 bits, once
    frame     -> 5x5 layer -> x
        x -> norm -> q (dense) -> norm, rotation -> attention to the held states -> y (dense)
        x, y -> x + gate y, normed and modulated -> wide layer, GELU (dense)
             -> back into x (dense with the stream as its residual) -> 3x3 layer

gate, scale and shift come per frame from a condition (here a noise level). Several
frames attend to one reference without its states being computed or kept in 16 bits again.
Run on an MI355X: python examples/held_reference_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import image_stencil_amd as isa  # noqa: E402

CHANNELS, HEADS, WIDE = 64, 2, 256


def weights(seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, fan_in, scale=2.0):
        return (torch.randn(shape, generator=g) * (scale / fan_in) ** 0.5).to(device)

    c = CHANNELS
    w = {"head": normal(c, 1, 5, 5, fan_in=25).half(), "tail": normal(c, c, 3, 3, fan_in=9 * c).half(),
         "q": normal(c, c, fan_in=c), "kv": normal(2 * c, c, fan_in=c), "o": normal(c, c, fan_in=c),
         "up": normal(WIDE, c, fan_in=c), "down": normal(c, WIDE, fan_in=WIDE), "condition": normal(3 * c, 8, fan_in=8)}
    w = {k: v.half() for k, v in w.items()}
    for name, n in (("head_b", c), ("tail_b", c), ("o_b", c), ("up_b", WIDE), ("down_b", c)):
        w[name] = torch.zeros(n, device=device)
    for name, n in (("norm_1", c), ("norm_2", c), ("norm_r", c), ("norm_q", c // HEADS), ("norm_k", c // HEADS)):
        w[name] = torch.ones(n, device=device)
    return w


def grid(h, w, device="cuda"):
    """Row and column of every pixel: 1 x h w x 2."""
    y, x = torch.meshgrid(torch.arange(h), torch.arange(w), indexing="ij")
    return torch.stack([y, x], -1).reshape(1, h * w, 2).to(torch.int32).to(device)


class HeldReferenceBlock:
    """For frames n x h x w and references n x hr x wr (fp16)."""

    def __init__(self, w, n, h, wd, hr, wr):
        self.w, self.n, d = w, n, CHANNELS // HEADS
        self.rotary, self.norm = isa.Rotary(d, axes=2), isa.BlockNorm(CHANNELS, "rms")
        self.at, self.at_ref = grid(h, wd), grid(hr, wr)
        self.none = torch.empty((n, 0, HEADS, d), dtype=torch.float16, device="cuda")
        self.nowhere = torch.empty((1, 0, 2), dtype=torch.int32, device="cuda")
        self.held = isa.HeldStates(n, hr * wr, HEADS, d)

    def tokens(self, frame):
        f = isa.conv2d(frame[..., None], self.w["head"], self.w["head_b"], relu=True)      # n x h x w x c
        return f.reshape(f.shape[0], -1, CHANNELS)

    def hold(self, reference):
        """Keys and values of the reference into the held states."""
        w, d = self.w, CHANNELS // HEADS
        _, r = self.norm.apply(self.tokens(reference), weight=w["norm_r"])
        kv = isa.dense(r, w["kv"]).view(self.n, -1, 2, HEADS, d)
        k, v = kv[:, :, 0], kv[:, :, 1]
        self.rotary.apply_qk_norm(self.none, k, self.nowhere, self.at_ref, w["norm_q"], w["norm_k"], q_out=self.none,
                                  k_out=k)
        self.held.put(k, v)

    def __call__(self, frame, condition):
        """condition: n x 1 x 8 (fp16)."""
        w, n, d = self.w, self.n, CHANNELS // HEADS
        gate, scale, shift = isa.dense(condition, w["condition"]).view(n, 3, CHANNELS).unbind(1)
        x = self.tokens(frame)
        _, z = self.norm.apply(x, weight=w["norm_1"])
        q = isa.dense(z, w["q"]).view(n, -1, HEADS, d)
        self.rotary.apply_qk_norm(q, self.none, self.at, self.nowhere, w["norm_q"], w["norm_k"], q_out=q, k_out=self.none)
        y = isa.held_attention(q, self.held).reshape(n, -1, CHANNELS)
        y = isa.dense(y, w["o"], w["o_b"])
        x, z = self.norm.apply(x, y, gate=gate, weight=w["norm_2"], scale=scale, shift=shift, x_out=x)
        z = isa.dense(z, w["up"], w["up_b"], activation="gelu")
        x = isa.dense(z, w["down"], w["down_b"], residual=x)
        h, wd = frame.shape[1:]
        return isa.conv2d(x.view(n, h, wd, CHANNELS), w["tail"], w["tail_b"], relu=True)


def main():
    n, h, w, hr, wr = 2, 90, 160, 72, 128
    block = HeldReferenceBlock(weights(), n, h, w, hr, wr)
    g = torch.Generator().manual_seed(1)
    frame, ref = (torch.rand((n, *s), generator=g).half().cuda() for s in ((h, w), (hr, wr)))
    condition = torch.randn((n, 1, 8), generator=g).half().cuda()
    block.hold(ref)
    y = block(frame, condition)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        y = block(frame, condition)
    b.record()
    torch.cuda.synchronize()
    print("features %s, mean %.4f, %.3f ms per frame, reference held in %.2f MB" % (
        tuple(y.shape), y.float().mean().item(), a.elapsed_time(b) / 20, block.held.bytes / 1e6))


if __name__ == "__main__":
    main()
