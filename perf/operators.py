"""Cases of the library's attention operators: rotary positions, the norm of
queries and keys with the rotation in the same pass, and cross attention.

Each case has a plain form in elementary torch operations (`own` false) and the
library's call (`own` true). Tokens are n x length x heads x d tensors whose
last dimension is contiguous: an fp16 NHWC feature map of the convolution layers
is one (length = H * W, heads * d = C) without a copy.

With P = rot / 2 pairs per head, A position axes and Pa = P / A, pair p of a
token turns by the angle  pos[p // Pa] * f[p % Pa],  f[i] = base^(-i / Pa),
rescaled for long contexts. Pair p is the elements (p, p + P) in the "half"
layout and (2p, 2p + 1) in the "interleaved" one; elements from rot on pass
through. The norm of a head is x * rsqrt(mean(x^2) + eps) * w. Attention is
softmax(scale * q k^T) v over the keys that the mask or the lengths leave, and a
row without keys gives zeros (lse: -infinity).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _rotary(name, dtype, n, length, heads, d, rot, axes, layout, scaling, first):
    return {"name": name, "op": "rotary", "dtype": dtype, "n": n, "length": length, "heads": heads, "d": d,
            "rot": rot, "axes": axes, "layout": layout, "scaling": scaling, "first": first}


def _qk(name, dtype, n, lq, lk, hq, hkv, d, rot, axes, layout, scaling, first, packed):
    return {"name": name, "op": "qk", "dtype": dtype, "n": n, "lq": lq, "lk": lk, "hq": hq, "hkv": hkv, "d": d,
            "rot": rot, "axes": axes, "layout": layout, "scaling": scaling, "first": first, "packed": packed}


def _cross(name, dtype, n, lq, lk, hq, hkv, d, mask, packed, lse):
    return {"name": name, "op": "cross", "dtype": dtype, "n": n, "lq": lq, "lk": lk, "hq": hq, "hkv": hkv, "d": d,
            "mask": mask, "packed": packed, "lse": lse}


def listed():
    return [
        # One new token of a decoder, far into its sequence: latency.
        _rotary("rotary_one_token", "f16", 1, 1, 16, 64, 64, 1, "half", "none", 70000),
        # A batch of 128 x 128 feature maps as tokens, row and column positions: bandwidth.
        _rotary("rotary_feature_maps", "bf16", 16, 128 * 128, 16, 64, 64, 2, "interleaved", "none", 0),
        # Half of an 80-element head turned, positions beyond the trained length, fp32.
        _rotary("rotary_part_scaled", "f32", 2, 8191, 6, 80, 40, 1, "half", "ramp", 100000),
        # One new token for each of 16 sequences, shared key heads.
        _qk("qk_one_token", "bf16", 16, 1, 1, 16, 4, 128, 128, 1, "half", "linear", 5000, False),
        # A 1280 x 720 frame in 16 x 16 patches: 45 x 80 tokens, q and k out of one packed projection.
        _qk("qk_frame_patches", "f16", 2, 3600, 3600, 8, 8, 64, 64, 2, "half", "none", 0, True),
        # Many image tokens and a reference of another length, shared key heads: bandwidth.
        _qk("qk_two_lengths", "bf16", 4, 128 * 128, 5000, 16, 4, 128, 96, 1, "interleaved", "ntk", 0, False),
        # One query token over a short encoder output: latency.
        _cross("cross_one_token_short", "f16", 1, 1, 257, 8, 8, 64, "none", False, False),
        # One query token for each of 4 sequences over a long encoder output: the read of k and v.
        _cross("cross_one_token_long", "bf16", 4, 1, 32771, 16, 2, 128, "none", False, False),
        # 64 x 64 image tokens over a padded prompt, one of them empty, 40-element heads.
        _cross("cross_prompt", "f16", 8, 4096, 120, 8, 8, 40, "lengths", True, False),
        # A frame's patches over a reference frame's, with the log-sum for joining two references.
        _cross("cross_reference_frame", "f16", 2, 3600, 3600, 8, 8, 64, "none", True, True),
        # Odd lengths, 96-element heads, holes in the reference, shared key heads.
        _cross("cross_odd_masked", "bf16", 3, 1021, 1543, 6, 3, 96, "mask", False, False),
        # 128 x 128 tokens over 128 x 128: the matrix cores.
        _cross("cross_large", "bf16", 1, 128 * 128, 128 * 128, 16, 4, 128, "none", False, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "qk", "cross", "cross"])
    if op == "cross":
        d = 8 * rng.randint(4, 16)
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 1, 2, 3, 4, 8])
        n = rng.randint(1, 8)
        lq = 1 if rng.random() < 0.3 else _log(rng, 2, 16384)
        most = 16 * 16384.0 * 16384.0 / (n * hq * float(lq))   # the largest listed case's scores
        lk = _log(rng, 1, max(1, int(min(40000, most))))
        c = _cross("", rng.choice(["f16", "bf16"]), n, lq, lk, hq, hkv, d, rng.choice(["none", "lengths", "mask"]),
                   rng.random() < 0.5, rng.random() < 0.3)
    else:
        dtype = rng.choice(["f32", "f16", "bf16"])
        axes = rng.choice([1, 1, 2, 3])
        d = 8 * rng.randint(4, 32)
        rot = 2 * axes * (d // (2 * axes) if rng.random() < 0.5 else rng.randint(2, d // (2 * axes)))
        layout = rng.choice(["half", "interleaved"])
        scaling = rng.choice(["none", "linear", "ntk", "ramp"])
        first = 0 if rng.random() < 0.5 else _log(rng, 1, 1000000)
        n, heads = rng.randint(1, 16), _log(rng, 1, 32)
        room = 16.0 * 16384 * 16 * 64 * 2 / (n * heads * d * (4 if dtype == "f32" else 2))
        length = 1 if rng.random() < 0.2 else _log(rng, 2, max(2, int(min(65536, room))))
        if op == "rotary":
            c = _rotary("", dtype, n, length, heads, d, rot, axes, layout, scaling, first)
        else:
            hkv = rng.choice([h for h in (1, 2, 4, heads) if h <= heads])
            length = max(1, length // 2)
            same = rng.random() < 0.5
            lk = length if same else _log(rng, 1, length + 1)
            c = _qk("", dtype, n, length, lk, heads, hkv, d, rot, axes, layout, scaling, first, same)
    del c["name"]
    return c


# ----------------------------------------------------------------- the inputs
# Frequencies, in 64 bits: base 10000; the long-context forms stretch by 4
# beyond 2048 positions ("ramp": per frequency, by the turns it makes there).
BASE, FACTOR, ORIGINAL, RAMP_LO, RAMP_HI, MAGNITUDE = 10000.0, 4.0, 2048, 1.0, 32.0, 0.1 * math.log(4.0) + 1.0


def _magnitude(c):
    return MAGNITUDE if c["scaling"] == "ramp" else 1.0


def _positions(n, length, axes, first, device):
    """Positions n x length x axes: running numbers, or the place in a grid of the
    nearest square's width for two axes and more; `first` shifts them all."""
    i = torch.arange(length, device=device)
    if axes == 1:
        p = i[:, None]
    else:
        w = max(1, int(math.sqrt(length)))
        p = torch.stack([i // w, i % w] + [torch.zeros_like(i)] * (axes - 2), 1)
    p = p[None] + first + 17 * torch.arange(n, device=device)[:, None, None]
    return p.to(torch.int32).contiguous()


def _lengths(c):
    """Visible keys of each batch entry: from all of them down to none."""
    n, lk = c["n"], c["lk"]
    return [lk if n == 1 else (lk * (n - 1 - b)) // (n - 1) for b in range(n)]


def prepare(case, seed):
    c, dev = dict(case), torch.device("cuda")
    t = DTYPES[c["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    s = {"case": c}
    if c["op"] == "rotary":
        s["x"] = normal(c["n"], c["length"], c["heads"], c["d"]).to(t)
        s["pos"] = _positions(c["n"], c["length"], c["axes"], c["first"], dev)
    elif c["op"] == "qk":
        n, lq, lk, hq, hkv, d = (c[k] for k in ("n", "lq", "lk", "hq", "hkv", "d"))
        if c["packed"]:   # q, k and v of one projection
            qkv = (3.0 * normal(n, lq, hq + 2 * hkv, d)).to(t)
            s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv]
        else:
            s["q"], s["k"] = (3.0 * normal(n, lq, hq, d)).to(t), (3.0 * normal(n, lk, hkv, d)).to(t)
        s["wq"], s["wk"] = 1.0 + 0.1 * normal(d), 1.0 + 0.1 * normal(d)
        s["pos_q"] = _positions(n, lq, c["axes"], c["first"], dev)
        s["pos_k"] = s["pos_q"] if lk == lq else _positions(n, lk, c["axes"], 0, dev)
    else:
        n, lq, lk, hq, hkv, d = (c[k] for k in ("n", "lq", "lk", "hq", "hkv", "d"))
        s["q"] = (1.5 * normal(n, lq, hq, d)).to(t)
        if c["packed"]:   # k and v of one projection
            kv = normal(n, lk, 2, hkv, d).to(t)
            s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        else:
            s["k"], s["v"] = normal(n, lk, hkv, d).to(t), normal(n, lk, hkv, d).to(t)
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev) if c["mask"] == "lengths" else None
        s["mask"] = torch.rand((n, lk), generator=g, device=dev) < 0.75 if c["mask"] == "mask" else None
    if own:
        import image_stencil_amd as isa
        if c["op"] == "cross":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((n, hq, lq), dtype=torch.float32, device=dev) if c["lse"] else None
            s["plan"] = isa.CrossAttention(s["q"], s["k"], s["v"], s["out"])
            s["workspace"] = s["plan"].new_workspace()
        else:
            s["rotary"] = isa.Rotary(c["d"], c["rot"], axes=c["axes"], layout=c["layout"], base=BASE,
                                     scaling=c["scaling"], factor=FACTOR, original_len=ORIGINAL,
                                     ramp=(RAMP_LO, RAMP_HI), magnitude=_magnitude(c))
            if c["op"] == "rotary":
                s["out"] = torch.empty_like(s["x"])
            else:
                s["q_out"] = torch.empty((n, lq, hq, d), dtype=t, device=dev)
                s["k_out"] = torch.empty((n, lk, hkv, d), dtype=t, device=dev)
    return s


# ------------------------------------------------------------- the plain form
def _angles(c, pos):
    """pos: n x length x axes. Angles n x length x 1 x pairs, in 64 bits: far
    positions times a frequency lose the angle in 32."""
    pairs = c["rot"] // 2
    per = pairs // c["axes"]
    i = torch.arange(per, dtype=torch.float64, device=pos.device)
    base = BASE * FACTOR ** (per / (per - 1.0)) if c["scaling"] == "ntk" else BASE
    f = base ** (-i / per)
    if c["scaling"] == "linear":
        f = f / FACTOR
    elif c["scaling"] == "ramp":
        keep = ((ORIGINAL * f / (2.0 * math.pi) - RAMP_LO) / (RAMP_HI - RAMP_LO)).clamp(0.0, 1.0)
        f = f * keep + f / FACTOR * (1.0 - keep)
    a = pos.to(torch.float64)[..., None] * f
    return a.reshape(pos.shape[0], pos.shape[1], 1, pairs)


def _turn(c, x, pos):
    """The rotation of a 32-bit x."""
    a, rot = _angles(c, pos), c["rot"]
    cos, sin = (_magnitude(c) * torch.cos(a)).float(), (_magnitude(c) * torch.sin(a)).float()
    y = x.clone()
    if c["layout"] == "half":
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = u * cos - v * sin, u * sin + v * cos
    else:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * cos - v * sin, u * sin + v * cos
    return y


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _visible(s):
    """n x lk truth values, or None where every key is visible."""
    c = s["case"]
    if s["mask"] is not None:
        return s["mask"]
    if s["lengths"] is not None:
        return torch.arange(c["lk"], device=s["q"].device)[None, :] < s["lengths"][:, None]
    return None


def _cross_plain(s):
    c = s["case"]
    n, lq, lk, hq, hkv, d = (c[k] for k in ("n", "lq", "lk", "hq", "hkv", "d"))
    group = hq // hkv
    q = s["q"].float().reshape(n, lq, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * lq, d)
    kt = s["k"].float().permute(0, 2, 3, 1).contiguous()
    v = s["v"].float().permute(0, 2, 1, 3).contiguous()
    see = _visible(s)
    scores = torch.matmul(q, kt).mul_(1.0 / math.sqrt(d))
    if see is not None:
        scores.masked_fill_(~see[:, None, None, :], -math.inf)
        v = v * 1.0
        v.masked_fill_(~see[:, None, :, None], 0.0)
    top = scores.amax(-1, keepdim=True)
    top.masked_fill_(top == -math.inf, 0.0)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores, v) / total.masked_fill(total == 0, 1.0)
    out = out.reshape(n, hkv, group, lq, d).permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d).to(s["q"].dtype)
    return (out, (torch.log(total) + top).reshape(n, hq, lq)) if c["lse"] else out


def run(state):
    s, c = state, state["case"]
    if own:
        if c["op"] == "rotary":
            return s["rotary"].apply(s["x"], s["pos"], out=s["out"])
        if c["op"] == "qk":
            return s["rotary"].apply_qk_norm(s["q"], s["k"], s["pos_q"], s["pos_k"], s["wq"], s["wk"], eps=EPS,
                                             q_out=s["q_out"], k_out=s["k_out"])
        out = s["plan"].forward(s["q"], s["k"], s["v"], s["out"], key_mask=s["mask"], key_lengths=s["lengths"],
                                lse=s["lse"], workspace=s["workspace"])
        return (out, s["lse"]) if c["lse"] else out
    if c["op"] == "rotary":
        return _turn(c, s["x"].float(), s["pos"]).to(s["x"].dtype)
    if c["op"] == "qk":
        return (_turn(c, _norm(s["q"].float(), s["wq"]), s["pos_q"]).to(s["q"].dtype),
                _turn(c, _norm(s["k"].float(), s["wk"]), s["pos_k"]).to(s["k"].dtype))
    return _cross_plain(s)


# ----------------------------------------------------- the work and the values
def _visible_keys(c):
    if c["mask"] == "lengths":
        return sum(_lengths(c))
    return c["n"] * c["lk"] * (0.75 if c["mask"] == "mask" else 1.0)


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rotary":
        tokens = c["n"] * c["length"]
        return {"bytes": 2 * size * tokens * c["heads"] * c["d"] + 4 * c["axes"] * tokens,
                "flops": 3 * tokens * c["heads"] * c["rot"]}
    if c["op"] == "qk":
        rows = c["n"] * (c["lq"] * c["hq"] + c["lk"] * c["hkv"])
        tokens = c["n"] * (c["lq"] if c["lq"] == c["lk"] else c["lq"] + c["lk"])
        return {"bytes": 2 * size * rows * c["d"] + 4 * c["axes"] * tokens + 8 * c["d"],
                "flops": rows * (4 * c["d"] + 3 * c["rot"])}
    keys = _visible_keys(c)
    small = {"none": 0, "lengths": 4 * c["n"], "mask": c["n"] * c["lk"]}[c["mask"]]
    return {"bytes": size * (2 * c["n"] * c["lq"] * c["hq"] * c["d"] + 2 * keys * c["hkv"] * c["d"]) + small
            + (4 * c["n"] * c["hq"] * c["lq"] if c["lse"] else 0),
            "flops": 4.0 * c["lq"] * c["hq"] * c["d"] * keys}


def _exact_rotation(c, x, pos):
    """Pairs as complex numbers times magnitude * exp(i angle), one axis at a time."""
    per, y = c["rot"] // 2 // c["axes"], x.clone()
    for p in range(c["rot"] // 2):
        axis, i = divmod(p, per)
        if c["scaling"] == "ntk":
            f = (BASE * FACTOR ** (per / (per - 1.0))) ** (-i / per)
        else:
            f = BASE ** (-i / per)
            if c["scaling"] == "linear":
                f /= FACTOR
            elif c["scaling"] == "ramp":
                turns = ORIGINAL * f / (2.0 * math.pi)
                keep = min(1.0, max(0.0, (turns - RAMP_LO) / (RAMP_HI - RAMP_LO)))
                f = keep * f + (1.0 - keep) * f / FACTOR
        a, b = (p, p + c["rot"] // 2) if c["layout"] == "half" else (2 * p, 2 * p + 1)
        z = torch.polar(torch.full_like(pos[..., axis], _magnitude(c), dtype=torch.float64),
                        pos[..., axis].double() * f)[:, :, None] * torch.complex(x[..., a], x[..., b])
        y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rotary":
        return _exact_rotation(c, s["x"].double(), s["pos"])
    if c["op"] == "qk":
        both = []
        for x, w, pos in ((s["q"], s["wq"], s["pos_q"]), (s["k"], s["wk"], s["pos_k"])):
            x = x.double()
            x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["d"] + EPS) * w.double()
            both.append(_exact_rotation(c, x, pos))
        return tuple(both)
    out = torch.zeros((c["n"], c["lq"], c["hq"], c["d"]), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((c["n"], c["hq"], c["lq"]), -math.inf, dtype=torch.float64, device=out.device)
    see = _visible(s)
    for b in range(c["n"]):
        at = torch.arange(c["lk"], device=out.device) if see is None else torch.nonzero(see[b])[:, 0]
        if at.numel() == 0:
            continue
        for h in range(c["hq"]):
            kh = s["k"][b, at, h * c["hkv"] // c["hq"]].double()
            vh = s["v"][b, at, h * c["hkv"] // c["hq"]].double()
            z = s["q"][b, :, h].double() @ kh.t().contiguous() / c["d"] ** 0.5
            lse[b, h] = torch.logsumexp(z, -1)
            out[b, :, h] = torch.exp(z - lse[b, h][:, None]) @ vh
    return (out, lse) if c["lse"] else out
