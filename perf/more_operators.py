"""Cases of the operators around the library's cross attention: the sum and norm
between two blocks, dense layers on tokens, and attention over states held in
8 bits. Each has a plain form in elementary torch operations (`own` false) and
the library's call (`own` true).

Tokens are n x length x c (or x heads x d) tensors with a contiguous last
dimension: an fp16 NHWC feature map of the convolution layers is one.

norm:  x' = x + s g post(y),  z = norm(x') w (1 + scale) + shift + b: the stream x
       takes a block's output y (itself normed, gated per entry and channel, and
       scaled), and the next block's input z is normed and modulated.
dense: out = residual + act(x w^T + b), w of out x in features.
hold:  keys and values kept as e4m3 numbers times a power of two for each block of
       32 tokens and head: 2^e, the smallest with max |x| <= 448 * 2^e and e >= -120;
       a value past the data type's largest number becomes the largest below it.
       Tokens beyond an entry's length count for nothing and are held as zeros.
held:  softmax(scale * q k^T) v over the held keys that lengths or mask leave; a row
       without keys gives zeros (lse: -infinity).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
BLOCK = 32          # tokens that share a scale
RESIDUAL_SCALE = 0.5


# ------------------------------------------------------------------ the cases
def _norm(name, dtype, n, length, c, norm, post, modulated, block):
    return {"name": name, "op": "norm", "dtype": dtype, "n": n, "length": length, "c": c, "norm": norm, "post": post,
            "modulated": modulated, "block": block}


def _dense(name, dtype, n, length, k, m, act, bias, residual, packed):
    return {"name": name, "op": "dense", "dtype": dtype, "n": n, "length": length, "k": k, "m": m, "act": act,
            "bias": bias, "residual": residual, "packed": packed}


def _hold(name, dtype, n, lk, hkv, d, lengths, packed):
    return {"name": name, "op": "hold", "dtype": dtype, "n": n, "lk": lk, "hkv": hkv, "d": d,
            "mask": "lengths" if lengths else "none", "packed": packed}


def _held(name, dtype, n, lq, lk, hq, hkv, d, mask, lse):
    return {"name": name, "op": "held", "dtype": dtype, "n": n, "lq": lq, "lk": lk, "hq": hq, "hkv": hkv, "d": d,
            "mask": mask, "lse": lse}


def listed():
    return [
        # One new token between two blocks: latency.
        _norm("norm_one_token", "bf16", 1, 1, 1024, "rms", "none", False, True),
        # An odd channel count in fp32, mean and variance.
        _norm("norm_odd", "f32", 3, 1021, 1001, "layer", "none", False, True),
        # A batch of 128 x 128 maps: block output normed, gated, added; next input normed and modulated.
        _norm("norm_feature_maps", "bf16", 8, 128 * 128, 1024, "rms", "rms", True, True),
        # One new token into the wide layer of a block: latency.
        _dense("dense_one_token", "f16", 1, 1, 1024, 4096, "gelu", True, False, False),
        # One token of each of 16 sequences through a large square layer: the read of the weights.
        _dense("dense_batch_of_tokens", "bf16", 16, 1, 8192, 8192, "none", True, True, False),
        # Odd sizes everywhere.
        _dense("dense_odd", "bf16", 3, 1021, 344, 777, "silu", True, True, False),
        # Two 1280 x 720 frames in 16 x 16 patches, the wide layer.
        _dense("dense_frame_patches", "f16", 2, 3600, 512, 2048, "gelu_tanh", True, False, False),
        # Four 128 x 128 maps back from the wide layer into the stream: the matrix cores.
        _dense("dense_feature_maps", "bf16", 4, 128 * 128, 4096, 1024, "none", True, True, False),
        # A padded prompt for each of 8 entries, one of them empty, 40-element heads: latency.
        _hold("hold_prompt", "f16", 8, 120, 8, 40, True, True),
        # Reference maps of 128 x 128 tokens.
        _hold("hold_feature_maps", "bf16", 4, 128 * 128, 4, 128, False, False),
        # One query token for each of 4 sequences over long states: the read of the held bytes.
        _held("held_one_token_long", "bf16", 4, 1, 32771, 16, 2, 128, "none", False),
        # A frame's patches over a reference frame's, with the log-sum for joining two references.
        _held("held_reference_frame", "f16", 2, 3600, 3600, 8, 8, 64, "none", True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "dense", "dense", "hold", "held", "held"])
    if op == "norm":
        dtype = rng.choice(["f32", "f16", "bf16"])
        n, c = rng.randint(1, 16), _log(rng, 8, 16384)
        room = 8.0 * 16384 * 1024 * 2 / (n * c * (4 if dtype == "f32" else 2))
        length = 1 if rng.random() < 0.2 else _log(rng, 1, max(1, int(min(65536, room))))
        block = rng.random() < 0.8
        norm = rng.choice(["rms", "layer", "none"]) if block else rng.choice(["rms", "layer"])
        c = _norm("", dtype, n, length, c, norm, rng.choice(["none", "rms", "layer"]) if block else "none",
                  rng.random() < 0.5, block)
    elif op == "dense":
        k, m = 8 * _log(rng, 2, 1024), _log(rng, 1, 8192)
        n = rng.choice([1, 1, 2, 3, 4, 8, 16])
        most = 4.0 * 16384 * 4096 * 1024 / (float(n) * k * m)
        length = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, int(min(65536 // n, most))))
        c = _dense("", rng.choice(["f16", "bf16"]), n, length, k, m,
                   rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.7,
                   rng.random() < 0.4, rng.random() < 0.4)
    else:
        dtype = rng.choice(["f16", "bf16"])
        d, n, hkv = 8 * rng.randint(1, 32), rng.randint(1, 8), rng.choice([1, 2, 3, 4, 8])
        if op == "hold":
            most = 4.0 * 16384 * 4 * 128 / (n * hkv * d)
            c = _hold("", dtype, n, _log(rng, 1, max(1, int(min(40000, most)))), hkv, d, rng.random() < 0.5,
                      rng.random() < 0.5)
        else:
            hq = hkv * rng.choice([1, 1, 2, 3, 4, 8])
            lq = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
            most = 2.0 * 8 * 3600 * 3600 * 64 / (n * hq * float(lq) * d)
            lk = _log(rng, 1, max(1, int(min(40000, most))))
            c = _held("", dtype, n, lq, lk, hq, hkv, d, rng.choice(["none", "lengths", "mask"]), rng.random() < 0.3)
    del c["name"]
    return c


# ----------------------------------------------------------------- the inputs
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
    if c["op"] == "norm":
        n, length, ch = c["n"], c["length"], c["c"]
        s["x"] = (2.0 * normal(n, length, ch) + 0.5).to(t)
        s["y"] = (0.7 * normal(n, length, ch)).to(t) if c["block"] else None
        s["weight"] = 1.0 + 0.1 * normal(ch) if c["norm"] != "none" else None
        s["bias"] = 0.1 * normal(ch) if c["norm"] == "layer" else None
        s["post_weight"] = 1.0 + 0.1 * normal(ch) if c["post"] != "none" else None
        # gate, scale and shift of every entry out of one projection of its condition
        packed = (0.5 * normal(n, 3, ch)).to(t) if c["modulated"] else None
        s["gate"] = packed[:, 0] if c["modulated"] and c["block"] else None
        s["scale"], s["shift"] = (packed[:, 1], packed[:, 2]) if c["modulated"] and c["norm"] != "none" else (None, None)
        if own:
            import image_stencil_amd as isa
            s["plan"] = isa.BlockNorm(ch, norm=None if c["norm"] == "none" else c["norm"],
                                      post=None if c["post"] == "none" else c["post"], eps=EPS,
                                      residual_scale=RESIDUAL_SCALE)
            s["x_out"] = torch.empty_like(s["x"]) if c["block"] else None
            s["out"] = torch.empty_like(s["x"]) if c["norm"] != "none" else None
    elif c["op"] == "dense":
        n, length, k, m = c["n"], c["length"], c["k"], c["m"]
        s["x"] = normal(n, length, 2 * k).to(t)[:, :, k:] if c["packed"] else normal(n, length, k).to(t)
        s["w"] = (normal(m, k) * (1.5 / math.sqrt(k))).to(t)
        s["bias"] = 0.5 * normal(m) if c["bias"] else None
        s["residual"] = normal(n, length, m).to(t) if c["residual"] else None
        if own:
            import image_stencil_amd as isa
            s["out"] = torch.empty((n, length, m), dtype=t, device=dev)
            s["plan"] = isa.Dense(s["x"], s["w"], out=s["out"], residual=s["residual"], activation=c["act"])
            s["workspace"] = s["plan"].new_workspace()
    else:
        n, lk, hkv, d = (c[k] for k in ("n", "lk", "hkv", "d"))
        if c["op"] == "hold" and c["packed"]:   # k and v of one projection
            kv = normal(n, lk, 2, hkv, d).to(t)
            s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        else:
            s["k"], s["v"] = normal(n, lk, hkv, d).to(t), normal(n, lk, hkv, d).to(t)
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev) if c["mask"] == "lengths" else None
        s["mask"] = torch.rand((n, lk), generator=g, device=dev) < 0.75 if c["mask"] == "mask" else None
        if own:
            import image_stencil_amd as isa
            s["held"] = isa.HeldStates(n, lk, hkv, d, dtype=t, device=dev)
        if c["op"] == "hold":
            if own:
                s["k_out"], s["v_out"] = torch.empty((n, lk, hkv, d), dtype=t, device=dev), \
                    torch.empty((n, lk, hkv, d), dtype=t, device=dev)
        else:
            s["q"] = (1.5 * normal(n, c["lq"], c["hq"], d)).to(t)
            # What a program keeps in hand between calls: the held states, not the full ones.
            k, v = s.pop("k"), s.pop("v")
            if own:
                s["held"].put(k, v)
                s["out"] = torch.empty_like(s["q"])
                s["lse"] = torch.empty((n, c["hq"], c["lq"]), dtype=torch.float32, device=dev) if c["lse"] else None
                s["plan"] = isa.HeldAttention(s["q"], s["held"], s["out"])
                s["workspace"] = s["plan"].new_workspace()
            else:
                s["k8"], s["k_scale"] = _to_8_bits(k, None)
                s["v8"], s["v_scale"] = _to_8_bits(v, None)
    return s


# ------------------------------------------------------------- the plain form
def _normed(x, kind, w):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return y if w is None else y * w


def _norm_plain(s):
    c, x = s["case"], s["x"].float()
    if c["block"]:
        y = s["y"].float()
        if c["post"] != "none":
            y = _normed(y, c["post"], s["post_weight"])
        if s["gate"] is not None:
            y = y * s["gate"].float()[:, None]
        x = x + RESIDUAL_SCALE * y
    z = None
    if c["norm"] != "none":
        z = _normed(x, c["norm"], s["weight"])
        if s["scale"] is not None:
            z = z * (1.0 + s["scale"].float()[:, None]) + s["shift"].float()[:, None]
        if s["bias"] is not None:
            z = z + s["bias"]
        z = z.to(s["x"].dtype)
    return (x.to(s["x"].dtype) if c["block"] else None, z)


def _activated(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _dense_plain(s):
    c = s["case"]
    z = torch.matmul(s["x"].float().reshape(-1, c["k"]), s["w"].float().t())
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _activated(z, c["act"]).reshape(c["n"], c["length"], c["m"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(s["x"].dtype)


def _to_8_bits(x, lengths):
    """x: n x length x heads x d. The e4m3 numbers, n x blocks x BLOCK x heads x d,
    and the scales, n x blocks x 1 x heads x 1."""
    n, length, heads, d = x.shape
    y = x.float()
    if lengths is not None:
        seen = torch.arange(length, device=x.device)[None, :] < lengths[:, None]
        y = y.masked_fill(~seen[:, :, None, None], 0.0)
    blocks = (length + BLOCK - 1) // BLOCK
    full = torch.zeros((n, blocks * BLOCK, heads, d), dtype=torch.float32, device=x.device)
    full[:, :length] = y
    full = full.reshape(n, blocks, BLOCK, heads, d)
    mantissa, exponent = torch.frexp(full.abs().amax((2, 4), keepdim=True))   # 448 = 0.875 * 2^9
    e = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8).clamp_min(-120)
    scale = ((e + 127) << 23).view(torch.float32)   # 2^e
    q = (full / scale).to(torch.float8_e4m3fn).float()
    over = q.abs() * scale > torch.finfo(x.dtype).max
    q = torch.where(over, 240.0 * torch.sign(q), q)
    return q.to(torch.float8_e4m3fn), scale


def _from_8_bits(q, scale, length):
    return (q.float() * scale).reshape(q.shape[0], -1, q.shape[3], q.shape[4])[:, :length]


def _visible(s):
    """n x lk truth values, or None where every key is visible."""
    if s["mask"] is not None:
        return s["mask"]
    if s["lengths"] is not None:
        return torch.arange(s["case"]["lk"], device=s["lengths"].device)[None, :] < s["lengths"][:, None]
    return None


def _held_plain(s):
    c = s["case"]
    n, lq, lk, hq, hkv, d = (c[k] for k in ("n", "lq", "lk", "hq", "hkv", "d"))
    group = hq // hkv
    q = s["q"].float().reshape(n, lq, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * lq, d)
    kt = _from_8_bits(s["k8"], s["k_scale"], lk).permute(0, 2, 3, 1).contiguous()
    v = _from_8_bits(s["v8"], s["v_scale"], lk).permute(0, 2, 1, 3).contiguous()
    see = _visible(s)
    scores = torch.matmul(q, kt).mul_(1.0 / math.sqrt(d))
    if see is not None:
        scores.masked_fill_(~see[:, None, None, :], -math.inf)
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
        if c["op"] == "norm":
            x, z = s["plan"].apply(s["x"], s["y"], gate=s["gate"], post_weight=s["post_weight"], weight=s["weight"],
                                   bias=s["bias"], scale=s["scale"], shift=s["shift"], x_out=s["x_out"], out=s["out"])
            return (x if c["block"] else None, z)
        if c["op"] == "dense":
            return s["plan"].forward(s["x"], s["w"], bias=s["bias"], residual=s["residual"], out=s["out"],
                                     workspace=s["workspace"])
        if c["op"] == "hold":
            s["held"].put(s["k"], s["v"], key_lengths=s["lengths"])
            return s["held"].get(k_out=s["k_out"], v_out=s["v_out"])
        out = s["plan"].forward(s["q"], s["held"], s["out"], key_mask=s["mask"], key_lengths=s["lengths"],
                                lse=s["lse"], workspace=s["workspace"])
        return (out, s["lse"]) if c["lse"] else out
    if c["op"] == "norm":
        return _norm_plain(s)
    if c["op"] == "dense":
        return _dense_plain(s)
    if c["op"] == "hold":
        return tuple(_from_8_bits(*_to_8_bits(s[name], s["lengths"]), c["lk"]).to(s[name].dtype) for name in ("k", "v"))
    return _held_plain(s)


# ----------------------------------------------------- the work and the values
def _visible_keys(c):
    if c["mask"] == "lengths":
        return sum(_lengths(c))
    return c["n"] * c["lk"] * (0.75 if c["mask"] == "mask" else 1.0)


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "norm":
        elements, ends = c["n"] * c["length"] * c["c"], c["norm"] != "none"
        moved = 1 + 2 * c["block"] + ends       # x, (y, x'), z
        vectors = ends + (c["norm"] == "layer") + (c["post"] != "none")
        per_entry = c["modulated"] * (c["block"] + 2 * ends)
        return {"bytes": size * (moved * elements + per_entry * c["n"] * c["c"]) + 4 * vectors * c["c"],
                "flops": elements * (3 * c["block"] + 5 * ends + 4 * (c["post"] != "none") + 2 * c["modulated"])}
    if c["op"] == "dense":
        rows, k, m = c["n"] * c["length"], c["k"], c["m"]
        return {"bytes": size * (rows * k + m * k + rows * m * (2 if c["residual"] else 1)) + 4 * m * c["bias"],
                "flops": 2.0 * rows * k * m}
    keys = _visible_keys(c)
    small = {"none": 0, "lengths": 4 * c["n"], "mask": c["n"] * c["lk"]}[c["mask"]]
    if c["op"] == "hold":   # visible states read; 8 bits written and read; all values written
        every = 2 * c["n"] * c["lk"] * c["hkv"] * c["d"]
        scales = 8 * c["n"] * c["hkv"] * ((c["lk"] + BLOCK - 1) // BLOCK)
        return {"bytes": size * 2 * keys * c["hkv"] * c["d"] + 2 * (every + scales) + size * every + small,
                "flops": 4.0 * every}
    return {"bytes": size * 2 * c["n"] * c["lq"] * c["hq"] * c["d"]
            + 2 * keys * c["hkv"] * (c["d"] + 4.0 / BLOCK) + small
            + (4 * c["n"] * c["hq"] * c["lq"] if c["lse"] else 0),
            "flops": 4.0 * c["lq"] * c["hq"] * c["d"] * keys}


def _exact_norm(x, kind, w):
    if kind == "layer":
        x = x - x.sum(-1, keepdim=True) / x.shape[-1]
    x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS)
    return x * w.double()


def _exact_8_bits(x, lengths):
    """Every value's neighbour among the e4m3 numbers times the block's scale, by
    the spacing of the numbers where it lies."""
    x, most = x.double(), torch.finfo(x.dtype).max
    powers = torch.tensor([2.0 ** i for i in range(-200, 200)], dtype=torch.float64, device=x.device)
    for b, length in enumerate([] if lengths is None else lengths.tolist()):
        x[b, length:] = 0.0
    for at in range(0, x.shape[1], BLOCK):
        part = x[:, at:at + BLOCK]
        e = torch.ceil(torch.log2(part.abs().amax((1, 3), keepdim=True) / 448.0)).clamp_min(-120.0)
        scale = powers[e.long() + 200]
        unit = part / scale
        spacing = powers[torch.floor(torch.log2(unit.abs().clamp_min(2.0 ** -6))).long() - 3 + 200]
        held = torch.round(unit / spacing) * spacing * scale
        x[:, at:at + BLOCK] = torch.where(held.abs() > most, torch.sign(held) * 240.0 * scale, held)
    return x


def exact(case, seed):
    c = dict(case)
    if c["op"] == "held":   # the full states of the same draws
        s = prepare(dict(c, op="hold", packed=False), seed)
        k, v = (_exact_8_bits(s[name], None) for name in ("k", "v"))
        s = prepare(c, seed)
        out = torch.zeros((c["n"], c["lq"], c["hq"], c["d"]), dtype=torch.float64, device=k.device)
        lse = torch.full((c["n"], c["hq"], c["lq"]), -math.inf, dtype=torch.float64, device=k.device)
        see = _visible(s)
        for b in range(c["n"]):
            at = torch.arange(c["lk"], device=k.device) if see is None else torch.nonzero(see[b])[:, 0]
            if at.numel() == 0:
                continue
            for h in range(c["hq"]):
                kh, vh = k[b, at, h * c["hkv"] // c["hq"]], v[b, at, h * c["hkv"] // c["hq"]]
                z = s["q"][b, :, h].double() @ kh.t().contiguous() / c["d"] ** 0.5
                lse[b, h] = torch.logsumexp(z, -1)
                out[b, :, h] = torch.exp(z - lse[b, h][:, None]) @ vh
        return (out, lse) if c["lse"] else out
    s = prepare(c, seed)
    if c["op"] == "hold":
        return tuple(_exact_8_bits(s[name], s["lengths"]) for name in ("k", "v"))
    if c["op"] == "dense":
        z = s["x"].double() @ s["w"].double().t().contiguous()
        if s["bias"] is not None:
            z += s["bias"].double()
        if c["act"] == "relu":
            z = torch.where(z > 0, z, torch.zeros_like(z))
        elif c["act"] == "gelu":
            z *= 0.5 * torch.erfc(-z / 2.0 ** 0.5)
        elif c["act"] == "gelu_tanh":
            z /= 1.0 + torch.exp(-2.0 * (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
        elif c["act"] == "silu":
            z /= 1.0 + torch.exp(-z)
        return z if s["residual"] is None else z + s["residual"].double()
    x, z = s["x"].double(), None
    if c["block"]:
        y = s["y"].double()
        if c["post"] != "none":
            y = _exact_norm(y, c["post"], s["post_weight"])
        if s["gate"] is not None:
            y *= s["gate"].double()[:, None]
        x = x + RESIDUAL_SCALE * y
    if c["norm"] != "none":
        z = _exact_norm(x, c["norm"], s["weight"])
        if s["scale"] is not None:
            z = z + s["scale"].double()[:, None] * z + s["shift"].double()[:, None]
        if s["bias"] is not None:
            z = z + s["bias"].double()
    return (x if c["block"] else None, z)
