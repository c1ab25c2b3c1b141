"""The operators around the attention of a transformer block (thin layer over the C-ABI
library; contracts in include/causaljvp.h):

    cos, sin = rope_table(pos, freq, axis)                   # angles from positions
    q, k, v = qk_norm_rope_fwd(xq, xk, xv, gq, gk, cos, sin, H)
    dxq, dxk, dxv, dgq, dgk = qk_norm_rope_bwd(dq, dk, dv, xq, xk, gq, gk, cos, sin)
    y, ty, pre = linear_act_fwd(x, w, bias, act="gelu_tanh", tx=tx, save_pre=True)
    dx, dw, db = linear_act_bwd(dy, x, w, act="gelu_tanh", pre=pre)
    c = ckpt8_pack(x); x = ckpt8_unpack(c)                   # activations kept in 8 bits

Tensors are CUDA tensors; calls run on the current stream of the tensors' device, whichever
device is current, and are asynchronous. Outputs are new tensors. Calls with no rows return
empty outputs (and zero gradients) without a launch.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch

from . import _lib

__all__ = ["Ckpt8", "ckpt8_pack", "ckpt8_unpack", "rope_frequencies", "rope_table", "qk_norm_rope_fwd",
           "qk_norm_rope_bwd", "linear_act_fwd", "linear_act_bwd"]

_DTYPES = {torch.float32: _lib.CAJ_DTYPE_F32, torch.bfloat16: _lib.CAJ_DTYPE_BF16}


# The calls are short, so what surrounds them is kept short too: addresses go to ctypes as plain
# ints, the current stream comes as a raw handle, and the device is switched only where it differs.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _run(name: str, device: torch.device, *args):
    """Calls the library's `name` on `device`'s current stream, with that device current."""
    fn, index = getattr(_lib.lib(), name), device.index
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _lib.check(st, name)


def _same_device(what: str, device: torch.device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"{what}: all tensors must be CUDA tensors on one device")


# ------------------------------------------------------------ 8-bit checkpoints

class Ckpt8(NamedTuple):
    """A tensor kept in 8 bits: codes int8 [rows, 32*nb], scales uint8 [rows, 4*ceil(nb/4)],
    nb = ceil(C/32) blocks a row, and the shape [..., C] it stands for."""
    codes: torch.Tensor
    scales: torch.Tensor
    shape: Tuple[int, ...]

    @property
    def rows(self) -> int:
        return math.prod(self.shape[:-1])

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _ckpt_widths(C: int) -> Tuple[int, int]:
    nb = -(-C // 32)
    return 32 * nb, 4 * -(-nb // 4)


def _check_ckpt(what: str, c: Ckpt8):
    w, ns = _ckpt_widths(c.shape[-1])
    rows, codes, scales = c.rows, c.codes, c.scales
    if not (codes.is_cuda and codes.dtype == torch.int8 and codes.shape == (rows, w) and codes.is_contiguous()
            and scales.is_cuda and scales.dtype == torch.uint8 and scales.shape == (rows, ns)
            and scales.is_contiguous()):
        raise ValueError(f"{what}: a checkpoint's codes are int8 [rows, {w}] and its scales uint8 "
                         f"[rows, {ns}], contiguous CUDA tensors")


def _rows(t: torch.Tensor) -> Optional[Tuple[int, int]]:
    """(rows, elements between rows) of t seen as rows of its last axis; None if its strides
    do not allow it."""
    rows = math.prod(t.shape[:-1])
    if t.is_contiguous():
        return rows, max(t.shape[-1], 1)
    if t.numel() == 0:
        return rows, max(t.shape[-1], 1)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        return None
    ld, inner = None, 1  # the distance of the innermost axis with more than one row; rows below
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != ld * inner:
            return None
        inner *= size
    if ld is None:
        ld = t.shape[-1]
    return (rows, ld) if ld >= t.shape[-1] else None


def ckpt8_pack(x: torch.Tensor) -> Ckpt8:
    """x [..., C] (bf16 or fp32, rows at one distance) in 8 bits: whole numbers in [-127, 127]
    times a power of two for each block of 32. An element is off by at most half a step, 1/127
    of its block's largest magnitude at worst; a block with inf or NaN decodes to NaN."""
    if not (x.is_cuda and x.dtype in _DTYPES and x.dim() >= 1 and x.shape[-1] >= 1):
        raise ValueError("ckpt8_pack: x must be a bf16 or fp32 CUDA tensor with at least one column")
    at = _rows(x)
    if at is None:
        x = x.contiguous()
        at = _rows(x)
    rows, ld = at
    C = x.shape[-1]
    w, ns = _ckpt_widths(C)
    codes = x.new_empty((rows, w), dtype=torch.int8)
    scales = x.new_empty((rows, ns), dtype=torch.uint8)
    _run("caj_ckpt_pack", x.device, x.data_ptr(), rows, C, ld, _DTYPES[x.dtype], codes.data_ptr(), scales.data_ptr())
    return Ckpt8(codes, scales, tuple(x.shape))


def ckpt8_unpack(c: Ckpt8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values a checkpoint stands for, contiguous [..., C] (exact in bf16 and fp32)."""
    _check_ckpt("ckpt8_unpack", c)
    if dtype not in _DTYPES:
        raise ValueError("ckpt8_unpack: dtype must be bf16 or fp32")
    device, C = c.codes.device, c.shape[-1]
    _same_device("ckpt8_unpack", device, c.scales)
    x = c.codes.new_empty(c.shape, dtype=dtype)
    _run("caj_ckpt_unpack", device, c.codes.data_ptr(), c.scales.data_ptr(), c.rows, C, C, _DTYPES[dtype],
         x.data_ptr())
    return x


# --------------------------------------------------------------- rotary positions

def rope_frequencies(dims: Union[int, Sequence[int]], base: float = 10000.0, factor: float = 1.0,
                     original_length: Optional[int] = None, fast: float = 32.0, slow: float = 1.0,
                     device: Union[str, torch.device] = "cuda"):
    """(freq, axis) for rope_table. dims: the rotated channels, one number or one for each
    position axis (even numbers, e.g. frames, rows, columns of a video); pair i of an axis of
    d channels turns by base^(-2i/d) a position.

    factor > 1 stretches positions for longer contexts: without original_length every
    frequency is divided by it (linear interpolation); with it, only pairs that turn at most
    `slow` times within original_length are, those that turn at least `fast` times are kept,
    and those between are blended linearly in their number of turns."""
    dims = [int(dims)] if isinstance(dims, int) else [int(d) for d in dims]
    if not dims or any(d <= 0 or d % 2 for d in dims):
        raise ValueError("rope_frequencies: dims must be positive even numbers")
    if not (base > 0 and factor >= 1 and fast > slow):
        raise ValueError("rope_frequencies: base > 0, factor >= 1 and fast > slow are needed")
    freq = torch.cat([float(base) ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in dims])
    axis = torch.cat([torch.full((d // 2,), a, dtype=torch.int32) for a, d in enumerate(dims)])
    if factor > 1:
        if original_length is None:
            freq = freq / factor
        else:
            keep = ((freq * original_length / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
            freq = freq * keep + freq / factor * (1 - keep)
    return freq.to(device), axis.to(device)


def rope_table(pos: torch.Tensor, freq: torch.Tensor, axis: Optional[torch.Tensor] = None,
               mscale: float = 1.0):
    """(cos, sin), each [N, P] fp32: mscale times the cosine and sine of
    pos[n, axis[i]] * freq[i]. pos: [N] or [N, axes] int32 or int64; freq: [P] fp64; axis: [P]
    int32 (None: all pairs turn with the first axis). Far positions lose nothing."""
    if not (pos.is_cuda and pos.dtype in (torch.int32, torch.int64) and pos.dim() in (1, 2) and pos.is_contiguous()):
        raise ValueError("rope_table: pos must be a contiguous int32 or int64 CUDA tensor [N] or [N, axes]")
    if not (freq.dtype == torch.float64 and freq.dim() == 1 and freq.is_contiguous() and freq.numel()):
        raise ValueError("rope_table: freq must be a contiguous fp64 tensor [P]")
    if axis is not None and not (axis.dtype == torch.int32 and axis.shape == freq.shape and axis.is_contiguous()):
        raise ValueError("rope_table: axis must be a contiguous int32 tensor [P]")
    _same_device("rope_table", pos.device, freq, axis)
    N, P, A = pos.shape[0], freq.shape[0], pos.shape[1] if pos.dim() == 2 else 1
    cos = pos.new_empty((N, P), dtype=torch.float32)
    sin = pos.new_empty((N, P), dtype=torch.float32)
    _run("caj_rope_table", pos.device, pos.data_ptr(), pos.dtype == torch.int64, freq.data_ptr(), _ptr(axis), N, A, P,
         mscale, cos.data_ptr(), sin.data_ptr())
    return cos, sin


def _token_rows(what: str, name: str, t: torch.Tensor, B: int, N: int, width: int, like: torch.Tensor):
    """t [B, N, width] with one distance between tokens: that distance. Raises otherwise."""
    if not (t.is_cuda and t.dtype == like.dtype and t.shape == (B, N, width)):
        raise ValueError(f"{what}: {name} must be a {like.dtype} CUDA tensor [{B}, {N}, {width}]")
    at = _rows(t)
    if at is None or at[1] * t.element_size() % 16 or t.data_ptr() % 16:
        raise ValueError(f"{what}: {name}'s tokens must lie at one distance, a multiple of 16 bytes, "
                         "16-byte aligned, with neighbouring channels side by side")
    return at[1]


def _rope_shape(what, B, N, Hq, Hk, D, dtype, gq, gk, rope_cos, rope_sin, eps, norm, layout):
    if norm not in _lib.NORMS or layout not in _lib.ROPE_LAYOUTS:
        raise ValueError(f"{what}: norm is one of {sorted(_lib.NORMS)}, layout one of {sorted(_lib.ROPE_LAYOUTS)}")
    for t in (rope_cos, rope_sin):
        if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and t.dim() == 2 and t.shape[0] == N
                and t.shape == rope_cos.shape):
            raise ValueError(f"{what}: rope tables must be contiguous fp32 CUDA tensors [N, pairs]")
    full = 0
    if norm == "none":
        if gq is not None or gk is not None:
            raise ValueError(f"{what}: norm 'none' takes no gains")
    else:
        for t in (gq, gk):
            if t is None or not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and t.dim() == 1):
                raise ValueError(f"{what}: gains must be contiguous fp32 CUDA tensors")
        full = int(norm == "token" or gq.numel() != D or gk.numel() != D)
        if full and (gq.numel() != Hq * D or gk.numel() != Hk * D):
            raise ValueError(f"{what}: gains hold D values (norm 'head', shared by the heads) or heads * D")
    return _lib.QkRopeShapeC(B, N, Hq, Hk, D, rope_cos.shape[1], _DTYPES[dtype], _lib.NORMS[norm],
                             _lib.ROPE_LAYOUTS[layout], full, float(eps))


def qk_norm_rope_fwd(xq, xk, xv, gq, gk, rope_cos, rope_sin, H: int, Hk: Optional[int] = None, eps: float = 1e-6,
                     norm: str = "head", layout: str = "interleaved", txq=None, txk=None, txv=None):
    """RMS norm of q and k, their rotation, and the attention's layout for q, k, v, in one pass.

    xq [B, N, H*D], xk and xv [B, N, Hk*D] (Hk None: H), bf16 or fp32; slices of one fused
    projection are fine. xv may be None. norm: "head" (gains [D] or [heads*D]), "token" (gains
    [heads*D]) or "none" (gains None). layout: pairs (2i, 2i+1) ("interleaved") or (i, i+P)
    ("half") of the first 2P channels of each head, P = rope_cos.shape[1]. With tangents txq,
    txk, txv also their JVP. Returns (q, k, v) or (q, k, v, tq, tk, tv), each
    [B, heads, N, D]; without xv, v and tv are left out."""
    what = "qk_norm_rope_fwd"
    Hk = H if Hk is None else Hk
    if xq.dim() != 3 or H <= 0 or Hk <= 0 or xq.shape[2] % H or xq.dtype not in _DTYPES:
        raise ValueError(f"{what}: xq must be a bf16 or fp32 tensor [B, N, H*D]")
    B, N, D = xq.shape[0], xq.shape[1], xq.shape[2] // H
    tangents = (txq, txk, txv)
    tan = txq is not None
    if (txk is None) == tan or (txv is not None) != (tan and xv is not None):
        raise ValueError(f"{what}: give the tangents of all inputs or of none")
    _same_device(what, xq.device, xk, xv, *tangents, gq, gk, rope_cos, rope_sin)
    shape = _rope_shape(what, B, N, H, Hk, D, xq.dtype, gq, gk, rope_cos, rope_sin, eps, norm, layout)
    shape.ldq = _token_rows(what, "xq", xq, B, N, H * D, xq)
    shape.ldk = _token_rows(what, "xk", xk, B, N, Hk * D, xq)
    if xv is not None:
        shape.ldv = _token_rows(what, "xv", xv, B, N, Hk * D, xq)
    if tan:
        shape.ldtq = _token_rows(what, "txq", txq, B, N, H * D, xq)
        shape.ldtk = _token_rows(what, "txk", txk, B, N, Hk * D, xq)
        if xv is not None:
            shape.ldtv = _token_rows(what, "txv", txv, B, N, Hk * D, xq)
    outs = [None if t is None else xq.new_empty((B, h, N, D))
            for t, h in ((xq, H), (xk, Hk), (xv, Hk), (txq, H), (txk, Hk), (txv, Hk))]
    if B * N:
        _run("caj_qk_rope_fwd", xq.device, xq.data_ptr(), xk.data_ptr(), _ptr(xv), _ptr(txq), _ptr(txk), _ptr(txv),
             _ptr(gq), _ptr(gk), rope_cos.data_ptr(), rope_sin.data_ptr(), ctypes.byref(shape),
             *[_ptr(t) for t in outs])
    return tuple(t for t in outs if t is not None)


def qk_norm_rope_bwd(dq, dk, dv, xq, xk, gq, gk, rope_cos, rope_sin, eps: float = 1e-6, norm: str = "head",
                     layout: str = "interleaved"):
    """Gradients of qk_norm_rope_fwd's primal: (dxq, dxk, dxv, dgq, dgk).

    dq [B, H, N, D], dk and dv [B, Hk, N, D] (dv None: no v, dxv None); xq, xk: the forward's
    inputs, or their 8-bit checkpoints (Ckpt8 of shape [B, N, heads*D]), read as they are; None
    with norm "none" (then dgq, dgk are None). dx [B, N, heads*D]; dg fp32, as long as the
    gains. Deterministic."""
    what = "qk_norm_rope_bwd"
    if dq.dim() != 4 or dk.dim() != 4 or dq.dtype not in _DTYPES:
        raise ValueError(f"{what}: dq, dk must be bf16 or fp32 tensors [B, heads, N, D]")
    B, H, N, D = dq.shape
    Hk = dk.shape[1]
    for t, h in ((dq, H), (dk, Hk), (dv, Hk)):
        if t is not None and not (t.is_cuda and t.is_contiguous() and t.dtype == dq.dtype
                                  and t.shape == (B, h, N, D)):
            raise ValueError(f"{what}: dq, dk, dv must be contiguous CUDA tensors [B, heads, N, D] of one dtype")
    shape = _rope_shape(what, B, N, H, Hk, D, dq.dtype, gq, gk, rope_cos, rope_sin, eps, norm, layout)
    ckpt = isinstance(xq, Ckpt8)
    xs, scales = [None, None], [None, None]
    if norm == "none":
        if xq is not None or xk is not None:
            raise ValueError(f"{what}: norm 'none' reads no inputs: give None")
    elif ckpt != isinstance(xk, Ckpt8):
        raise ValueError(f"{what}: xq and xk are both tensors or both checkpoints")
    else:
        for i, (name, x, h) in enumerate((("xq", xq, H), ("xk", xk, Hk))):
            if ckpt:
                if tuple(x.shape) != (B, N, h * D):
                    raise ValueError(f"{what}: {name}'s checkpoint must be of shape [{B}, {N}, {h * D}]")
                _check_ckpt(what, x)
                xs[i], scales[i] = x.codes, x.scales
            else:
                if x is None:
                    raise ValueError(f"{what}: {name} is needed")
                setattr(shape, ("ldq", "ldk")[i], _token_rows(what, name, x, B, N, h * D, dq))
                xs[i] = x
    _same_device(what, dq.device, dk, dv, *xs, *scales, gq, gk, rope_cos, rope_sin)
    dx = [None if t is None else dq.new_empty((B, N, h * D)) for t, h in ((dq, H), (dk, Hk), (dv, Hk))]
    dg = [None if g is None else torch.zeros_like(g) if B * N == 0 else torch.empty_like(g) for g in (gq, gk)]
    if B * N:
        nbytes = ctypes.c_size_t(0)
        _lib.check(_lib.lib().caj_qk_rope_bwd_workspace(ctypes.byref(shape), ctypes.byref(nbytes)),
                   "caj_qk_rope_bwd_workspace")
        ws = dq.new_empty(nbytes.value, dtype=torch.uint8)
        _run("caj_qk_rope_bwd", dq.device, dq.data_ptr(), dk.data_ptr(), _ptr(dv), _ptr(xs[0]), _ptr(xs[1]),
             _ptr(scales[0]), _ptr(scales[1]), _ptr(gq), _ptr(gk), rope_cos.data_ptr(), rope_sin.data_ptr(),
             ctypes.byref(shape), *[_ptr(t) for t in dx], _ptr(dg[0]), _ptr(dg[1]), ws.data_ptr(), nbytes.value)
    return (*dx, *dg)


# --------------------------------------------------------------------- linear layers

def _matrix(what: str, name: str, t: torch.Tensor, rows: Optional[int], cols: int) -> int:
    """t [..., cols] bf16 as rows at one distance, 16-byte aligned: that distance."""
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.dim() >= 1 and t.shape[-1] == cols
            and (rows is None or t.numel() == rows * cols)):
        raise ValueError(f"{what}: {name} must be a bf16 CUDA tensor with rows of {cols} elements"
                         + ("" if rows is None else f", {rows} of them"))
    at = _rows(t)
    if at is None or at[1] % 8 or t.data_ptr() % 16:
        raise ValueError(f"{what}: {name}'s rows must lie at one distance, a multiple of 16 bytes, 16-byte aligned")
    return at[1]


def _weight(what: str, w: torch.Tensor, bias: Optional[torch.Tensor]):
    if not (w.is_cuda and w.dtype == torch.bfloat16 and w.dim() == 2 and w.is_contiguous()):
        raise ValueError(f"{what}: w must be a contiguous bf16 CUDA tensor [C, K]")
    if w.shape[0] % 8 or w.shape[1] % 8 or 0 in w.shape:
        raise ValueError(f"{what}: C and K must be positive multiples of 8")
    if bias is not None and not (bias.is_cuda and bias.dtype == torch.bfloat16 and bias.is_contiguous()
                                 and tuple(bias.shape) == (w.shape[0],)):
        raise ValueError(f"{what}: bias must be a contiguous bf16 CUDA tensor [C]")


def linear_act_fwd(x, w, bias=None, act: str = "none", residual=None, tx=None, tresidual=None,
                   save_pre: bool = False):
    """(y, ty, pre): y = act(z) + residual with z = x W^T + bias, its tangent
    ty = act'(z) * (tx W^T) + tresidual, and z as an 8-bit checkpoint for linear_act_bwd.

    x, tx [..., K] and residual, tresidual [..., C] bf16 (rows at one distance: slices are
    fine); w [C, K], bias [C] bf16; act "none", "gelu_tanh", "gelu" or "silu". y, ty [..., C]
    bf16. Without tx, ty is None; without save_pre, pre is. Everything after the product is
    done in fp32 in its epilogue."""
    what = "linear_act_fwd"
    _weight(what, w, bias)
    if act not in _lib.ACTS:
        raise ValueError(f"{what}: act is one of {sorted(_lib.ACTS)}")
    if tresidual is not None and tx is None:
        raise ValueError(f"{what}: tresidual needs tx")
    C, K = w.shape
    ldx = _matrix(what, "x", x, None, K)
    M, lead = x.numel() // K, tuple(x.shape[:-1])
    for name, t in (("tx", tx), ("residual", residual), ("tresidual", tresidual)):
        if t is not None and tuple(t.shape[:-1]) != lead:
            raise ValueError(f"{what}: {name} must have x's leading shape")
    shape = _lib.LinearActShapeC(M, K, C, _lib.ACTS[act], ldx)
    if tx is not None:
        shape.ldtx = _matrix(what, "tx", tx, M, K)
    if residual is not None:
        shape.ldres = _matrix(what, "residual", residual, M, C)
    if tresidual is not None:
        shape.ldtres = _matrix(what, "tresidual", tresidual, M, C)
    _same_device(what, x.device, w, bias, residual, tx, tresidual)
    y = x.new_empty(lead + (C,))
    ty = x.new_empty(lead + (C,)) if tx is not None else None
    pre = None
    if save_pre:
        cw, sw = _ckpt_widths(C)
        pre = Ckpt8(x.new_empty((M, cw), dtype=torch.int8), x.new_empty((M, sw), dtype=torch.uint8), lead + (C,))
    if M:
        nbytes = ctypes.c_size_t(0)
        _lib.check(_lib.lib().caj_linear_act_fwd_workspace(ctypes.byref(shape), int(tx is not None),
                                                           ctypes.byref(nbytes)), "caj_linear_act_fwd_workspace")
        ws = x.new_empty(nbytes.value, dtype=torch.uint8) if nbytes.value else None
        _run("caj_linear_act_fwd", x.device, x.data_ptr(), _ptr(tx), w.data_ptr(), _ptr(bias), _ptr(residual),
             _ptr(tresidual), ctypes.byref(shape), y.data_ptr(), _ptr(ty), _ptr(pre.codes if pre else None),
             _ptr(pre.scales if pre else None), _ptr(ws), nbytes.value)
    return y, ty, pre


def linear_act_bwd(dy, x, w, act: str = "none", pre: Optional[Ckpt8] = None, bias: bool = True,
                   need: Tuple[bool, bool] = (True, True)):
    """Gradients (dx, dw, db) of linear_act_fwd's primal (the residual's is dy itself).

    dy [..., C] bf16; x [..., K] bf16 or its Ckpt8 (may be None if dw is not needed); w [C, K];
    pre: the forward's checkpoint of z, needed with an activation. need: whether dx and dw are
    wanted; bias: whether db is. dx [..., K] and dw [C, K] bf16, db [C] fp32 (None where not
    wanted). Deterministic."""
    what = "linear_act_bwd"
    _weight(what, w, None)
    if act not in _lib.ACTS:
        raise ValueError(f"{what}: act is one of {sorted(_lib.ACTS)}")
    if not (need[0] or need[1] or bias):
        raise ValueError(f"{what}: no gradient is wanted")
    C, K = w.shape
    ldy = _matrix(what, "dy", dy, None, C)
    M, lead = dy.numel() // C, tuple(dy.shape[:-1])
    shape = _lib.LinearActShapeC(M, K, C, _lib.ACTS[act], 0, 0, 0, 0, ldy)
    ckpt = isinstance(x, Ckpt8)
    if need[1]:
        if ckpt:
            if x.rows != M or x.shape[-1] != K:
                raise ValueError(f"{what}: x's checkpoint must be of {M} rows of {K}")
            _check_ckpt(what, x)
        elif x is None:
            raise ValueError(f"{what}: dw needs x")
        else:
            shape.ldx = _matrix(what, "x", x, M, K)
    if act == "none":
        if pre is not None:
            raise ValueError(f"{what}: without an activation no checkpoint is read")
    else:
        if pre is None or pre.rows != M or pre.shape[-1] != C:
            raise ValueError(f"{what}: an activation needs the checkpoint of z, {M} rows of {C}")
        _check_ckpt(what, pre)
    xs = x.codes if ckpt else x
    _same_device(what, dy.device, w, *(t for t in (xs if need[1] else None, x.scales if ckpt else None,
                                                   *(pre[:2] if pre else ()))))
    dx = dy.new_empty(lead + (K,)) if need[0] else None
    make = dy.new_empty if M else dy.new_zeros
    dw = make((C, K)) if need[1] else None
    db = make((C,), dtype=torch.float32) if bias else None
    if M:
        nbytes = ctypes.c_size_t(0)
        _lib.check(_lib.lib().caj_linear_act_bwd_workspace(ctypes.byref(shape), int(ckpt), ctypes.byref(nbytes)),
                   "caj_linear_act_bwd_workspace")
        ws = dy.new_empty(nbytes.value, dtype=torch.uint8) if nbytes.value else None
        _run("caj_linear_act_bwd", dy.device, dy.data_ptr(), _ptr(xs if need[1] else None),
             _ptr(x.scales if ckpt and need[1] else None), w.data_ptr(), _ptr(pre.codes if pre else None),
             _ptr(pre.scales if pre else None), ctypes.byref(shape), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws),
             nbytes.value)
    return dx, dw, db
