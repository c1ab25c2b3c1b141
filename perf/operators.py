"""The operators around the attention of a transformer block in primal-tangent form:
their plain forms, the library's calls, and the sizes that they are measured at.

The block is the one the library's attention serves: tokens [B, N, width] of a video
(frames of 1560 tokens, 12 heads of 128 channels, width 1536), projected to q, k, v,
normalised and rotated, attended to, projected back, and passed through a feed-forward
pair of 1536 -> 6144 -> 1536. Four operators:

  rope_table   cosines and sines of rotary angles from integer positions (several axes,
               frequencies scaled for long contexts)
  norm_rope    norm of queries and keys over each head (or token) and their rotation, in
               primal, primal-tangent and backward form
  linear       matrix product with bias, activation and residual in its epilogue, in
               primal, primal-tangent and backward form
  ckpt8        activation checkpoints in 8 bits, which norm_rope's and linear's backward
               read and linear's forward writes

An 8-bit checkpoint of a row holds blocks of 32 values: each value as a whole number c in
[-127, 127] times 2^(s - 127), with one byte s per block, the smallest s with
max|value| <= 127 * 2^(s - 127). Codes are padded with zeros to whole blocks and scale
bytes to whole groups of four.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the angles of one 30 x 52 latent frame, made for each new frame of a stream
        {"name": "rope_table_frame", "kind": "rope_table", "n": 1560, "axes": 3, "pairs": 64,
         "start": 20, "factor": 1.0, "mscale": 1.0},
        # positions far into a long context, frequencies scaled by parts
        {"name": "rope_table_long", "kind": "rope_table", "n": 131072, "axes": 1, "pairs": 64,
         "start": 1000003, "factor": 8.0, "mscale": 1.2079},
        # one frame of a stream, served: the primal alone, q, k, v as slices of one projection
        {"name": "norm_rope_frame", "kind": "norm_rope", "b": 1, "n": 1560, "h": 12, "hk": 12, "d": 128,
         "pairs": 64, "layout": "interleaved", "norm": "head", "dtype": "bf16", "tangent": False, "fused": True},
        # a teacher-forcing sequence of two times 21 frames, in primal-tangent form
        {"name": "norm_rope_long_jvp", "kind": "norm_rope", "b": 1, "n": 65520, "h": 12, "hk": 12, "d": 128,
         "pairs": 32, "layout": "half", "norm": "head", "dtype": "bf16", "tangent": True, "fused": False},
        # its gradient, from inputs kept in 8 bits
        {"name": "norm_rope_long_bwd", "kind": "norm_rope_bwd", "b": 1, "n": 65520, "h": 12, "hk": 12, "d": 128,
         "pairs": 64, "layout": "interleaved", "norm": "head", "dtype": "bf16", "ckpt": True},
        # the feed-forward's first product for a single token
        {"name": "linear_token", "kind": "linear", "m": 1, "k": 1536, "c": 6144, "act": "gelu_tanh",
         "bias": True, "residual": False, "tangent": False, "pre": False},
        # the attention block's output product of one frame with its residual, primal and tangent
        {"name": "linear_frame_jvp", "kind": "linear", "m": 1560, "k": 1536, "c": 1536, "act": "none",
         "bias": True, "residual": True, "tangent": True, "pre": False},
        # the feed-forward's first product of 21 frames, with its activation's tangent and an 8-bit checkpoint
        {"name": "linear_long_jvp", "kind": "linear", "m": 32760, "k": 1536, "c": 6144, "act": "gelu_tanh",
         "bias": True, "residual": False, "tangent": True, "pre": True},
        # gradients of the feed-forward's second product, one frame
        {"name": "linear_frame_bwd", "kind": "linear_bwd", "m": 1560, "k": 6144, "c": 1536, "act": "none",
         "bias": True, "ckpt": False},
        # gradients of its first product over 21 frames, input and pre-activation kept in 8 bits
        {"name": "linear_long_bwd", "kind": "linear_bwd", "m": 32760, "k": 1536, "c": 6144, "act": "gelu_tanh",
         "bias": True, "ckpt": True},
        # a block's input of 21 frames put away in 8 bits
        {"name": "ckpt8_pack_long", "kind": "ckpt8_pack", "m": 32760, "c": 1536, "dtype": "bf16"},
        # one frame's fetched back
        {"name": "ckpt8_unpack_frame", "kind": "ckpt8_unpack", "m": 1560, "c": 1544, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope_table", "norm_rope", "norm_rope_bwd", "linear", "linear", "linear_bwd",
                       "linear_bwd", "ckpt8_pack", "ckpt8_unpack"])
    if kind == "rope_table":
        axes = rng.choice([1, 3])
        return {"kind": kind, "n": _log(rng, 1, 131072), "axes": axes, "pairs": rng.randrange(8, 65),
                "start": _log(rng, 1, 4000000) if axes == 1 else rng.randrange(0, 200),
                "factor": rng.choice([1.0, 2.0, 8.0, 32.0]), "mscale": rng.choice([1.0, 1.2079])}
    if kind in ("norm_rope", "norm_rope_bwd"):
        b, d = rng.choice([1, 1, 2, 3]), rng.choice([64, 128])
        h = rng.choice([1, 3, 8, 12, 16])
        c = {"kind": kind, "b": b, "n": _log(rng, 1, max(2, 65520 * 12 * 128 // (b * h * d * 2))), "h": h, "hk": h,
             "d": d, "pairs": rng.choice([d // 8, d // 4, d // 2]), "layout": rng.choice(["interleaved", "half"]),
             "norm": rng.choice(["head", "head", "token"]), "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        if h % 2 == 0 and rng.random() < 0.3:
            c["hk"] = h // 2
        if kind == "norm_rope":
            c["tangent"], c["fused"] = rng.random() < 0.5, rng.random() < 0.5
        else:
            c["ckpt"] = rng.random() < 0.5
        return c
    if kind in ("linear", "linear_bwd"):
        k, c = 8 * _log(rng, 16, 768), 8 * _log(rng, 16, 768)
        m = _log(rng, 1, max(2, min(65520, 32760 * 1536 * 6144 // (k * c))))
        act = rng.choice(["none", "gelu_tanh", "gelu", "silu"])
        if kind == "linear":
            return {"kind": kind, "m": m, "k": k, "c": c, "act": act, "bias": rng.random() < 0.7,
                    "residual": rng.random() < 0.4, "tangent": rng.random() < 0.5, "pre": rng.random() < 0.4}
        return {"kind": kind, "m": m, "k": k, "c": c, "act": act, "bias": rng.random() < 0.7,
                "ckpt": rng.random() < 0.5}
    c = rng.randrange(1, 6145)
    return {"kind": kind, "m": _log(rng, 1, max(2, 32760 * 1536 // c)), "c": c, "dtype": rng.choice(["bf16", "bf16", "fp32"])}


def _size(dtype):
    return 4 if dtype == "fp32" else 2


def _ckpt_bytes(rows, c):
    nb = -(-c // BLOCK)
    return rows * (nb * BLOCK + 4 * -(-nb // 4))


def work(case):
    k = case["kind"]
    if k == "rope_table":
        return {"bytes": case["n"] * (8 * case["axes"] + 8 * case["pairs"]) + 8 * case["pairs"],
                "flops": 20 * case["n"] * case["pairs"]}
    if k in ("norm_rope", "norm_rope_bwd"):
        rows, d, s = case["b"] * case["n"], case["d"], _size(case["dtype"])
        qk, v = rows * (case["h"] + case["hk"]) * d, rows * case["hk"] * d
        tab = case["n"] * case["pairs"] * 8
        if k == "norm_rope":
            t = 2 if case["tangent"] else 1
            return {"bytes": 2 * s * t * (qk + v) + tab, "flops": 12 * t * qk}
        x = sum(_ckpt_bytes(rows, h * d) for h in (case["h"], case["hk"])) if case["ckpt"] else qk * s
        return {"bytes": 2 * s * (qk + v) + x + tab, "flops": 20 * qk}
    if k == "linear":
        m, kk, c, t = case["m"], case["k"], case["c"], 2 if case["tangent"] else 1
        n = 2 * t * (m * kk + m * c) + 2 * kk * c + (2 * c if case["bias"] else 0)
        n += 2 * t * m * c if case["residual"] else 0
        n += _ckpt_bytes(m, c) + 2 * m * c if case["pre"] else 0  # written, and read back as values
        return {"bytes": n, "flops": 2 * t * m * kk * c}
    if k == "linear_bwd":
        m, kk, c = case["m"], case["k"], case["c"]
        n = 2 * m * c + 4 * kk * c + 2 * m * kk + (4 * c if case["bias"] else 0)
        n += _ckpt_bytes(m, kk) if case["ckpt"] else 2 * m * kk
        n += _ckpt_bytes(m, c) if case["act"] != "none" else 0
        return {"bytes": n, "flops": 4 * m * kk * c}
    m, c = case["m"], case["c"]
    values = (2 if k == "ckpt8_pack" else 1) * m * c * _size(case["dtype"])  # packed and read back, or read back alone
    return {"bytes": values + _ckpt_bytes(m, c), "flops": 3 * m * c}


# --------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _activations(g, m, c, dtype):
    """Values as the layers of a trained network hand them on: most channels near one
    in size, one in 64 a good deal larger."""
    gain = torch.where(torch.rand(c, generator=g, device=DEV) < 1 / 64, 12.0, 1.0)
    return (torch.randn(m, c, generator=g, device=DEV) * gain).to(dtype)


def _frequencies(case):
    """Angle per position of each pair, 64 bits, and the axis each pair turns with. With a
    factor above one the slow pairs are slowed down by it, the fast ones are kept, and those
    between are blended (by how often they turn within an original length of 4096)."""
    pairs, axes = case["pairs"], case["axes"]
    axis = torch.arange(pairs, dtype=torch.int32, device=DEV) % axes
    per = -(-pairs // axes)
    i = (torch.arange(pairs, device=DEV) // axes).double()
    freq = 10000.0 ** (-i / per)
    if case["factor"] > 1:
        turns = freq * 4096 / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        freq = freq * keep + freq / case["factor"] * (1 - keep)
    return freq, axis


def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _tables(g, n, pairs):
    theta = torch.rand(n, pairs, generator=g, device=DEV, dtype=torch.float64) * 400.0
    return theta.cos().float(), theta.sin().float()


def _pack(x):
    """Codes and scale bytes of the rows of x, as plain tensor operations."""
    m, c = x.shape
    nb = -(-c // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - c)).view(m, nb, BLOCK)
    bits = v.abs().amax(-1).view(torch.int32)  # of a value that is no less than 0
    s = ((bits >> 23) - 6 + ((bits & 0x7FFFFF) > 0x7E0000)).clamp(min=0)
    up = ((254 - s) << 23).view(torch.float32)  # 2^(127 - s), by its bits
    codes = torch.round(v * up.unsqueeze(-1)).to(torch.int8).view(m, nb * BLOCK)
    scales = torch.nn.functional.pad(s, (0, -nb % 4)).to(torch.uint8)
    return codes, scales


def _unpack(codes, scales, c):
    """The values that codes and scale bytes stand for, in 32 bits."""
    m, w = codes.shape
    s = scales[:, :w // BLOCK].to(torch.int32)
    unit = torch.where(s > 0, s << 23, 0x400000).view(torch.float32)  # 2^(s - 127), by its bits
    return (codes.view(m, w // BLOCK, BLOCK).float() * unit.unsqueeze(-1)).view(m, w)[:, :c].contiguous()


def prepare(case, seed):
    g, k = _gen(seed), case["kind"]
    st = {"case": case}
    if k == "rope_table":
        n = case["n"]
        if case["axes"] == 1:
            pos = case["start"] + int(seed) % 1000 + torch.arange(n, device=DEV).unsqueeze(1)
        else:
            i = torch.arange(n, device=DEV)
            pos = torch.stack([case["start"] + int(seed) % 50 + i // 1560, i % 1560 // 52, i % 52], 1)
        st["pos"] = pos.to(torch.int64).contiguous()
        st["freq"], st["axis"] = _frequencies(case)
        return st
    if k in ("norm_rope", "norm_rope_bwd"):
        b, n, h, hk, d, dt = case["b"], case["n"], case["h"], case["hk"], case["d"], _dtype(case)
        st["cos"], st["sin"] = _tables(g, n, case["pairs"])
        st["gq"] = 1 + 0.1 * torch.randn(d if case["norm"] == "head" else h * d, generator=g, device=DEV)
        st["gk"] = 1 + 0.1 * torch.randn(d if case["norm"] == "head" else hk * d, generator=g, device=DEV)
        widths = (h * d, hk * d, hk * d)
        if k == "norm_rope":
            for t in ("x", "tx")[:2 if case["tangent"] else 1]:
                if case["fused"]:
                    parts = _randn(g, b, n, sum(widths), dtype=dt, std=1.5).split(widths, -1)
                else:
                    parts = [_randn(g, b, n, w, dtype=dt, std=1.5) for w in widths]
                st.update({t + s: p for s, p in zip("qkv", parts)})
            return st
        for s, heads in zip("qkv", (h, hk, hk)):
            st["d" + s] = _randn(g, b, heads, n, d, dtype=dt)
        for s, w in zip("qk", widths):
            x = _randn(g, b, n, w, dtype=dt, std=1.5)
            st["x" + s] = _pack(x.view(b * n, w)) if case["ckpt"] else x
        return st
    if k in ("linear", "linear_bwd"):
        m, kk, c = case["m"], case["k"], case["c"]
        st["w"] = _randn(g, c, kk, std=kk ** -0.5)
        if k == "linear":
            st["x"] = _randn(g, m, kk)
            st["bias"] = _randn(g, c, std=0.3) if case["bias"] else None
            st["res"] = _randn(g, m, c) if case["residual"] else None
            st["tx"] = _randn(g, m, kk, std=0.5) if case["tangent"] else None
            st["tres"] = _randn(g, m, c, std=0.5) if case["tangent"] and case["residual"] else None
            return st
        x = _randn(g, m, kk)
        st["dy"] = _randn(g, m, c)
        st["x"] = _pack(x) if case["ckpt"] else x
        st["pre"] = _pack(_randn(g, m, c, std=1.2)) if case["act"] != "none" else None
        return st
    x = _activations(g, case["m"], case["c"], _dtype(case))
    if k == "ckpt8_pack":
        st["x"] = x
    else:
        st["codes"], st["scales"] = _pack(x)
    return st


# ---------------------------------------------------------- plain forms

def _act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    a = (2 / math.pi) ** 0.5
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 0.134145 * z * z)


def _turn(x, cos, sin, layout, sign):
    """Rotates the first 2 P channels of x [B, N, H, D] by angles [N, P] (sign -1: back)."""
    p = cos.shape[1]
    c, s = cos[:, None], sign * sin[:, None]
    if layout == "half":
        a, b = x[..., :p], x[..., p:2 * p]
        return torch.cat([a * c - b * s, a * s + b * c, x[..., 2 * p:]], -1)
    a, b = x[..., 0:2 * p:2], x[..., 1:2 * p:2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), x[..., 2 * p:]], -1)


_EPS = 1e-6


def _rms(x, norm):
    over = (-1,) if norm == "head" else (-2, -1)
    return over, torch.sqrt((x * x).mean(over, keepdim=True) + _EPS)


def _norm_rope(st, s, heads):
    case = st["case"]
    d, norm, dt = case["d"], case["norm"], _dtype(case)
    x = st["x" + s].float().unflatten(-1, (heads, d))
    gain = st["g" + s].view(-1, d)
    over, r = _rms(x, norm)
    y = [gain * x / r]
    if case["tangent"]:
        tx = st["tx" + s].float().unflatten(-1, (heads, d))
        y.append(gain * (tx / r - x * (x * tx).mean(over, keepdim=True) / r ** 3))
    return [_turn(t, st["cos"], st["sin"], case["layout"], 1).transpose(1, 2).to(dt).contiguous() for t in y]


def _norm_rope_bwd(st, s, heads):
    case = st["case"]
    b, n, d, norm, dt = case["b"], case["n"], case["d"], case["norm"], _dtype(case)
    x = _unpack(*st["x" + s], heads * d) if case["ckpt"] else st["x" + s].float()
    x = x.view(b, n, heads, d)
    gain = st["g" + s].view(-1, d)
    dy = _turn(st["d" + s].float().transpose(1, 2), st["cos"], st["sin"], case["layout"], -1)
    over, r = _rms(x, norm)
    gdy = gain * dy
    dx = gdy / r - x * (x * gdy).mean(over, keepdim=True) / r ** 3
    dg = dy * x / r
    dg = dg.sum((0, 1, 2)) if norm == "head" else dg.sum((0, 1)).flatten()
    return dx.to(dt).view(b, n, heads * d), dg


def _plain(st):
    case = st["case"]
    k = case["kind"]
    if k == "rope_table":
        angle = st["pos"].double()[:, st["axis"].long()] * st["freq"]
        return [(angle.cos() * case["mscale"]).float(), (angle.sin() * case["mscale"]).float()]
    if k == "norm_rope":
        b, n, hk, d = case["b"], case["n"], case["hk"], case["d"]
        q, kk = _norm_rope(st, "q", case["h"]), _norm_rope(st, "k", hk)
        vs = [st[t].reshape(b, n, hk, d).transpose(1, 2).contiguous() for t in ("xv", "txv")[:len(q)]]
        return [t for three in zip(q, kk, vs) for t in three]
    if k == "norm_rope_bwd":
        dxq, dgq = _norm_rope_bwd(st, "q", case["h"])
        dxk, dgk = _norm_rope_bwd(st, "k", case["hk"])
        return [dxq, dxk, st["dv"].transpose(1, 2).contiguous().flatten(2), dgq, dgk]
    if k == "linear":
        w = st["w"].float().t()
        z = st["x"].float() @ w
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y, slope = _act(z, case["act"])
        out = {"y": (y if st["res"] is None else y + st["res"].float()).to(torch.bfloat16)}
        if st["tx"] is not None:
            ty = slope * (st["tx"].float() @ w)
            out["ty"] = (ty if st["tres"] is None else ty + st["tres"].float()).to(torch.bfloat16)
        if case["pre"]:
            out["pre"] = _unpack(*_pack(z), case["c"]).to(torch.bfloat16)
        return out
    if k == "linear_bwd":
        dz = st["dy"].float()
        if st["pre"] is not None:
            dz = dz * _act(_unpack(*st["pre"], case["c"]), case["act"])[1]
        x = _unpack(*st["x"], case["k"]) if case["ckpt"] else st["x"].float()
        out = {"dx": (dz @ st["w"].float()).to(torch.bfloat16), "dw": (dz.t() @ x).to(torch.bfloat16)}
        if case["bias"]:
            out["db"] = dz.sum(0)
        return out
    if k == "ckpt8_pack":
        return _unpack(*_pack(st["x"]), case["c"]).to(_dtype(case))
    return _unpack(st["codes"], st["scales"], case["c"]).to(_dtype(case))


# ------------------------------------------------------- the library's

def _own(st):
    import masked_attention_jvp_b200 as caj
    case = st["case"]
    k = case["kind"]
    if k == "rope_table":
        return list(caj.rope_table(st["pos"], st["freq"], st["axis"], mscale=case["mscale"]))
    if k == "norm_rope":
        return list(caj.qk_norm_rope_fwd(st["xq"], st["xk"], st["xv"], st["gq"], st["gk"], st["cos"], st["sin"],
                                         case["h"], case["hk"], eps=_EPS, norm=case["norm"], layout=case["layout"],
                                         txq=st.get("txq"), txk=st.get("txk"), txv=st.get("txv")))
    if k == "norm_rope_bwd":
        x = [st["xq"], st["xk"]]
        if case["ckpt"]:
            x = [caj.Ckpt8(*p, (case["b"], case["n"], heads * case["d"]))
                 for p, heads in zip(x, (case["h"], case["hk"]))]
        return list(caj.qk_norm_rope_bwd(st["dq"], st["dk"], st["dv"], *x, st["gq"], st["gk"], st["cos"], st["sin"],
                                         eps=_EPS, norm=case["norm"], layout=case["layout"]))
    if k == "linear":
        y, ty, pre = caj.linear_act_fwd(st["x"], st["w"], st["bias"], act=case["act"], residual=st["res"],
                                        tx=st["tx"], tresidual=st["tres"], save_pre=case["pre"])
        out = {"y": y}
        if ty is not None:
            out["ty"] = ty
        if pre is not None:
            out["pre"] = caj.ckpt8_unpack(pre, torch.bfloat16)
        return out
    if k == "linear_bwd":
        x = caj.Ckpt8(*st["x"], (case["m"], case["k"])) if case["ckpt"] else st["x"]
        pre = None if st["pre"] is None else caj.Ckpt8(*st["pre"], (case["m"], case["c"]))
        dx, dw, db = caj.linear_act_bwd(st["dy"], x, st["w"], act=case["act"], pre=pre, bias=case["bias"])
        return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}
    if k == "ckpt8_pack":
        return caj.ckpt8_unpack(caj.ckpt8_pack(st["x"]), _dtype(case))
    return caj.ckpt8_unpack(caj.Ckpt8(st["codes"], st["scales"], (case["m"], case["c"])), _dtype(case))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------- definitions, 64 bits

def _two_to(e):
    """2^e in 64 bits for whole numbers e (a device's pow may be an ulp off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales, c):
    m, w = codes.shape
    unit = _two_to(scales[:, :w // BLOCK].long() - 127)
    return (codes.double().reshape(m, -1, BLOCK) * unit[..., None]).reshape(m, w)[:, :c]


def _exact_ckpt(x):
    """x rounded to the values an 8-bit checkpoint can hold."""
    m, c = x.shape
    nb = -(-c // BLOCK)
    v = x.new_zeros(m, nb * BLOCK)
    v[:, :c] = x
    v = v.view(m, nb, BLOCK)
    frac, ex = torch.frexp(v.abs().max(-1, keepdim=True).values)  # frac in [1/2, 1)
    unit = _two_to(torch.clamp(ex - 7 + (frac > 127 / 128).int(), min=-127))
    return (torch.round(v / unit) * unit).view(m, -1)[:, :c]


def _exact_rotation(n, p, d, layout, cos, sin):
    """The rotation of each position as indexes of each channel's partner, its own factor
    and its partner's: out[i] = own[i] x[i] + other[i] x[partner[i]]."""
    partner = torch.arange(d, device=DEV)
    mine = torch.ones(n, d, dtype=torch.float64, device=DEV)
    other = torch.zeros(n, d, dtype=torch.float64, device=DEV)
    i = torch.arange(p, device=DEV)
    first, second = (i, i + p) if layout == "half" else (2 * i, 2 * i + 1)
    partner[first], partner[second] = second, first
    mine[:, first], mine[:, second] = cos, cos
    other[:, first], other[:, second] = -sin, sin
    return partner, mine, other


def exact(case, seed):
    st = prepare(case, seed)
    k = case["kind"]
    if k == "rope_table":
        pos = torch.stack([st["pos"][:, a] for a in st["axis"].tolist()], 1).double()
        theta = pos * st["freq"][None]
        return [case["mscale"] * torch.cos(theta), case["mscale"] * torch.sin(theta)]
    if k in ("norm_rope", "norm_rope_bwd"):
        b, n, d, head = case["b"], case["n"], case["d"], case["norm"] == "head"
        part, mine, other = _exact_rotation(n, case["pairs"], d, case["layout"], st["cos"].double(), st["sin"].double())
        res = {}
        for s, h in (("q", case["h"]), ("k", case["hk"])):
            gain = st["g" + s].double()
            gain = gain.repeat(h) if head else gain
            if k == "norm_rope":
                x = st["x" + s].double()
            else:
                x = _exact_values(*st["x" + s], h * d) if case["ckpt"] else st["x" + s].double()
            groups, wide = (b * n * h, d) if head else (b * n, h * d)
            x = x.reshape(groups, wide)
            inv = ((x * x).sum(1, keepdim=True) / wide + _EPS) ** -0.5
            if k == "norm_rope":
                ys = [x * inv]
                if case["tangent"]:
                    tx = st["tx" + s].double().reshape(groups, wide)
                    ys.append(inv * tx - inv ** 3 * x * (x * tx).sum(1, keepdim=True) / wide)
                for t, y in zip(("", "t"), ys):
                    y = (y.reshape(b * n, h * d) * gain).reshape(b, n, h, d).permute(0, 2, 1, 3)
                    res[t + s] = mine * y + other * y[..., part]
                continue
            dq = st["d" + s].double()
            back = (mine * dq + (other * dq)[..., part]).permute(0, 2, 1, 3).reshape(b * n, h * d)
            xhat = x * inv
            dg = (back * xhat.reshape(b * n, h * d)).sum(0)
            res["dg" + s] = dg.reshape(h, d).sum(0) if head else dg
            u = (back * gain).reshape(groups, wide)
            res["dx" + s] = (inv * (u - xhat * (u * xhat).sum(1, keepdim=True) / wide)).reshape(b, n, h * d)
        if k == "norm_rope_bwd":
            dv = st["dv"].double().permute(0, 2, 1, 3).reshape(b, n, case["hk"] * d)
            return [res["dxq"], res["dxk"], dv, res["dgq"], res["dgk"]]
        for t in ("", "t")[:2 if case["tangent"] else 1]:
            res[t + "v"] = st[t + "xv"].double().reshape(b, n, case["hk"], d).permute(0, 2, 1, 3)
        return [res[t + s] for t in ("", "t")[:2 if case["tangent"] else 1] for s in "qkv"]
    if k in ("linear", "linear_bwd"):
        w = st["w"].double()

        def slope_of(z):
            if case["act"] == "none":
                return z, torch.ones_like(z)
            with torch.enable_grad():
                u = z.detach().requires_grad_(True)
                f = torch.nn.functional
                v = {"silu": f.silu, "gelu": f.gelu,
                     "gelu_tanh": lambda a: f.gelu(a, approximate="tanh")}[case["act"]](u)
                return v.detach(), torch.autograd.grad(v.sum(), u)[0]

        if k == "linear":
            z = torch.einsum("mk,ck->mc", st["x"].double(), w)
            if st["bias"] is not None:
                z += st["bias"].double()
            v, slope = slope_of(z)
            out = {"y": v + st["res"].double() if st["res"] is not None else v}
            if st["tx"] is not None:
                out["ty"] = slope * torch.einsum("mk,ck->mc", st["tx"].double(), w)
                if st["tres"] is not None:
                    out["ty"] = out["ty"] + st["tres"].double()
            if case["pre"]:
                out["pre"] = _exact_ckpt(z)
            return out
        dz = st["dy"].double()
        if st["pre"] is not None:
            dz = dz * slope_of(_exact_values(*st["pre"], case["c"]))[1]
        x = _exact_values(*st["x"], case["k"]) if case["ckpt"] else st["x"].double()
        out = {"dx": torch.einsum("mc,ck->mk", dz, w), "dw": torch.einsum("mc,mk->ck", dz, x)}
        if case["bias"]:
            out["db"] = dz.sum(0)
        return out
    if k == "ckpt8_pack":
        return _exact_ckpt(st["x"].double())
    return _exact_values(st["codes"], st["scales"], case["c"])
