"""Plain 64-bit forms of the block operators, written from their formulas, for the tests.
Everything is torch float64 on the CPU; inputs are converted exactly."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


def d(t):
    return t.detach().cpu().double()


# ---------------------------------------------------------------- 8-bit checkpoints

def ckpt(x):
    """(codes int64 [rows, 32 nb], scale bytes int64 [rows, 4 ceil(nb/4)]) of x [rows, C],
    block by block from the definition: the smallest s >= 0 with max <= 127 * 2^(s - 127),
    at most 248, where magnitudes above 127 * 2^121 saturate."""
    x = d(x)
    rows, C = x.shape
    nb = -(-C // 32)
    codes = torch.zeros(rows, 32 * nb, dtype=torch.int64)
    scales = torch.zeros(rows, 4 * -(-nb // 4), dtype=torch.int64)
    for r in range(rows):
        for b in range(nb):
            v = x[r, 32 * b:32 * b + 32]
            if not torch.isfinite(v).all():
                scales[r, b] = 255
                continue
            top, s = float(v.abs().max()), 0
            if top > 0:
                s = max(0, math.frexp(top)[1] + 127 - 7 - 1)
                while top > 127 * 2.0 ** (s - 127):
                    s += 1
                while s > 0 and top <= 127 * 2.0 ** (s - 1 - 127):
                    s -= 1
            s = min(s, 248)
            scales[r, b] = s
            codes[r, 32 * b:32 * b + len(v)] = torch.round(v * 2.0 ** (127 - s)).clamp(-127, 127).long()
    return codes, scales


def unckpt(codes, scales, C):
    codes, scales = codes.cpu().long(), scales.cpu().long()
    rows, w = codes.shape
    s = scales[:, :w // 32].double().repeat_interleave(32, 1)
    v = codes.double() * torch.where(s == 255, torch.full_like(s, math.nan), 2.0 ** (s - 127))
    return v[:, :C]


# ---------------------------------------------------------------- norm and rotation

def turn(x, cos, sin, layout, back=False):
    """x [B, N, H, D]; cos, sin [N, P]."""
    P = cos.shape[1]
    y = x.clone()
    c, s = cos[None, :, None, :], (-sin if back else sin)[None, :, None, :]
    i = torch.arange(P)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + P)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def turn_abs(x, cos, sin, layout):
    """The sum of the magnitudes of the terms of turn()."""
    P = cos.shape[1]
    x, y = x.abs(), x.abs().clone()
    c, s = cos.abs()[None, :, None, :], sin.abs()[None, :, None, :]
    i = torch.arange(P)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + P)
    y[..., a] = x[..., a] * c + x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def _over(norm):
    return (-1,) if norm == "head" else (-2, -1)


def _gain(g, H, D):
    return g.view(-1, D) if g.numel() == D else g.view(H, D)


def norm_rope(x, tx, g, cos, sin, H, eps, norm, layout):
    """(y, ty, |y| terms, |ty| terms), each [B, H, N, D]; tx may be None."""
    B, N, C = x.shape
    D = C // H
    x = x.view(B, N, H, D)
    tx = None if tx is None else tx.view(B, N, H, D)
    if norm == "none":
        y, ty = x, tx
        ay, aty = x.abs(), None if tx is None else tx.abs()
    else:
        g = _gain(g, H, D)
        r = torch.sqrt((x * x).mean(_over(norm), keepdim=True) + eps)
        y = g * x / r
        ay = y.abs()
        if tx is not None:
            ty = g * (tx / r - x * (x * tx).mean(_over(norm), keepdim=True) / r ** 3)
            aty = g.abs() * (tx.abs() / r + x.abs() * (x * tx).abs().mean(_over(norm), keepdim=True) / r ** 3)
        else:
            ty = aty = None
    out = [turn(y, cos, sin, layout), None if ty is None else turn(ty, cos, sin, layout),
           turn_abs(ay, cos, sin, layout), None if ty is None else turn_abs(aty, cos, sin, layout)]
    return [None if t is None else t.transpose(1, 2) for t in out]


def norm_rope_bwd(dy, x, g, cos, sin, eps, norm, layout):
    """(dx, dg, |dx| terms, |dg| terms) from dy [B, H, N, D]."""
    B, H, N, D = dy.shape
    dy = dy.transpose(1, 2)
    u, au = turn(dy, cos, sin, layout, back=True), turn_abs(dy, cos, sin, layout)
    if norm == "none":
        return u.reshape(B, N, H * D), None, au.reshape(B, N, H * D), None
    x = x.view(B, N, H, D)
    gg = _gain(g, H, D)
    over = _over(norm)
    r = torch.sqrt((x * x).mean(over, keepdim=True) + eps)
    dx = gg * u / r - x * (x * gg * u).mean(over, keepdim=True) / r ** 3
    adx = gg.abs() * au / r + x.abs() * (x * gg).abs().mul(au).mean(over, keepdim=True) / r ** 3
    dg, adg = u * x / r, au * x.abs() / r
    keep = (0, 1, 2) if g.numel() == D else (0, 1)
    return (dx.reshape(B, N, H * D), dg.sum(keep).flatten(), adx.reshape(B, N, H * D), adg.sum(keep).flatten())


# -------------------------------------------------------------------- linear layers

def act(z, which):
    """act(z) and its derivative, from the formulas."""
    if which == "none":
        return z, torch.ones_like(z)
    if which == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if which == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)


def product_loss(depth):
    """What a sum of `depth` products may lose, relative to the sum of their magnitudes:
    products are exact, fp32 sums are truncated (2^-23), one after the other per 16 of them,
    and up to 32 parts, a bias and a few more are added."""
    return (depth / 16 + 40) * 2.0 ** -23


ACT_LOSS = 2.0 ** -19  # exponential, reciprocal (2^-22 each, arguments below 2^3 amplify) and products


def linear(x, w, bias, which, res, tx, tres):
    """{"y": (value, bound without the output's own rounding), "ty": ..., "z": ...}."""
    z, az = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, az = z + bias, az + bias.abs()
    ez = az * product_loss(x.shape[1])
    y, slope = act(z, which)
    ey = 1.2 * ez + ACT_LOSS * z.abs()  # |act'| < 1.13
    if res is not None:
        y, ey = y + res, ey + 2.0 ** -23 * (y.abs() + res.abs())
    out = {"y": (y, ey), "z": (z, ez)}
    if tx is not None:
        tz, atz = tx @ w.t(), tx.abs() @ w.abs().t()
        ty = slope * tz
        ety = 1.2 * atz * product_loss(x.shape[1]) + (1.2 * ez + ACT_LOSS * (1 + z.abs())) * tz.abs()  # |act''| < 1.2
        if which == "none":
            ety = atz * product_loss(x.shape[1])
        if tres is not None:
            ty, ety = ty + tres, ety + 2.0 ** -23 * (ty.abs() + tres.abs())
        out["ty"] = (ty, ety)
    return out


def linear_bwd(dy, x, w, z, which):
    """dx, dw, db with bounds (without the outputs' own rounding)."""
    dz, edz = dy, torch.zeros_like(dy)
    if which != "none":
        dz = dy * act(z, which)[1]
        edz = dy.abs() * ACT_LOSS * (1 + z.abs())
    rounded = dz.abs() * (2.0 ** -8 if which != "none" else 0.0) + edz
    out = {"db": (dz.sum(0), edz.sum(0) + dz.abs().sum(0) * (dy.shape[0] / 8 + 64) * 2.0 ** -24)}
    out["dx"] = (dz @ w, rounded @ w.abs() + dz.abs() @ w.abs() * product_loss(w.shape[0]))
    if x is not None:
        out["dw"] = (dz.t() @ x, rounded.t() @ x.abs() + dz.abs().t() @ x.abs() * product_loss(dy.shape[0]))
    return out
