"""A frame's features attend to a reference frame's, between two convolution layers.

    frame (1 channel) -> 5x5 layer -> fp16 NHWC features --+-> q --norm, rotation--+
                                                           |                       v
    reference frame   -> 5x5 layer -> fp16 NHWC features --+-> k --norm, rotation--> cross attention
                                                           +-> v ------------------^      |
                                    features + attended features -> 3x3 layer <-----------+

Queries are the frame's pixels, keys and values the reference's (of any other
size); positions are row and column. Projections are 1x1, as plain matrix
products of torch. Run on an MI355X: python examples/attend_reference.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import image_stencil_amd as isa  # noqa: E402

CHANNELS, HEADS = 64, 2


def weights(seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, fan_in):
        return (torch.randn(shape, generator=g) * (2.0 / fan_in) ** 0.5).to(device)

    c = CHANNELS
    return {"head": normal(c, 1, 5, 5, fan_in=25), "head_b": torch.zeros(c, device=device),
            "q": normal(c, c, fan_in=c).half(), "kv": normal(c, 2 * c, fan_in=c).half(),
            "q_norm": torch.ones(c // HEADS, device=device), "k_norm": torch.ones(c // HEADS, device=device),
            "tail": normal(c, c, 3, 3, fan_in=9 * c), "tail_b": torch.zeros(c, device=device)}


def grid(h, w, device="cuda"):
    """Row and column of every pixel: 1 x h w x 2."""
    y, x = torch.meshgrid(torch.arange(h), torch.arange(w), indexing="ij")
    return torch.stack([y, x], -1).reshape(1, h * w, 2).to(torch.int32).to(device)


class AttendReference:
    """The block for frames n x h x w and references n x hr x wr (fp16)."""

    def __init__(self, w, h, wd, hr, wr):
        self.w, d = w, CHANNELS // HEADS
        self.rotary = isa.Rotary(d, axes=2)
        self.at, self.at_ref = grid(h, wd), grid(hr, wr)

    def features(self, frame):
        return isa.conv2d(frame[..., None], self.w["head"].half(), self.w["head_b"], relu=True)   # n x h x w x c

    def attend(self, f, r):
        """f: n x h x w x c features, r: n x hr x wr x c of the reference."""
        n, d = f.shape[0], CHANNELS // HEADS
        tokens, ref = f.reshape(n, -1, CHANNELS), r.reshape(n, -1, CHANNELS)
        q = (tokens @ self.w["q"]).view(n, -1, HEADS, d)
        kv = (ref @ self.w["kv"]).view(n, -1, 2, HEADS, d)
        k, v = kv[:, :, 0], kv[:, :, 1]
        # in place: k is a slice of the packed projection
        self.rotary.apply_qk_norm(q, k, self.at, self.at_ref, self.w["q_norm"], self.w["k_norm"], q_out=q, k_out=k)
        return f + isa.cross_attention(q, k, v).view_as(f)

    def __call__(self, frame, reference):
        z = self.attend(self.features(frame), self.features(reference))
        return isa.conv2d(z, self.w["tail"].half(), self.w["tail_b"], relu=True)


def main():
    h, w, hr, wr = 90, 160, 72, 128
    block = AttendReference(weights(), h, w, hr, wr)
    g = torch.Generator().manual_seed(1)
    frame, ref = (torch.rand((2, *s), generator=g).half().cuda() for s in ((h, w), (hr, wr)))
    y = block(frame, ref)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        y = block(frame, ref)
    b.record()
    torch.cuda.synchronize()
    print("features %s, mean %.4f, %.3f ms per pass" % (tuple(y.shape), y.float().mean().item(),
                                                        a.elapsed_time(b) / 20))


if __name__ == "__main__":
    main()
