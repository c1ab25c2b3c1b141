"""Block operators without a GPU: the 64-bit reference forms against finite differences,
the host-side frequency helper, and every refusal (nothing is launched)."""
import ctypes
import math

import pytest
import torch

import block_reference as ref
import masked_attention_jvp_b200 as caj
from masked_attention_jvp_b200 import _lib

_NO_GPU = not torch.cuda.is_available()
INVALID, UNSUPPORTED, CUDA = _lib.CAJ_ERR_INVALID_ARG, _lib.CAJ_ERR_UNSUPPORTED, _lib.CAJ_ERR_CUDA
A = 1 << 20  # a fake, aligned device address: validation never reads it


# ------------------------------------------------------------------ reference forms

@pytest.mark.parametrize("norm", ["none", "head", "token"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_norm_rope_reference_against_differences(norm, layout):
    g = torch.Generator().manual_seed(3)
    B, N, H, D, P = 2, 3, 2, 32, 8
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, tx, dy = rnd(B, N, H * D), rnd(B, N, H * D), rnd(B, H, N, D)
    gain = None if norm == "none" else 1 + 0.1 * rnd(H * D if norm == "token" else D)
    th = rnd(N, P)
    cos, sin = th.cos(), th.sin()
    f = lambda x_, g_: ref.norm_rope(x_, None, g_, cos, sin, H, 1e-6, norm, layout)[0]  # noqa: E731
    h = 1e-5
    ty = ref.norm_rope(x, tx, gain, cos, sin, H, 1e-6, norm, layout)[1]
    num = (f(x + h * tx, gain) - f(x - h * tx, gain)) / (2 * h)
    # central differences: O(h^2) truncation and 2^-53 / h rounding, both near 1e-10
    assert torch.allclose(ty, num, rtol=0, atol=1e-8)
    dx, dg, _, _ = ref.norm_rope_bwd(dy, x, gain, cos, sin, 1e-6, norm, layout)
    assert abs(float((dx * tx).sum() - (dy * num).sum())) < 1e-7
    if norm != "none":
        dirn = rnd(gain.numel())
        num_g = (f(x, gain + h * dirn) - f(x, gain - h * dirn)) / (2 * h)
        assert abs(float((dg * dirn).sum() - (dy * num_g).sum())) < 1e-7


def test_ckpt_reference_holds_the_format():
    x = torch.tensor([[127.0, -1.0, 0.5, 1.5] + [0.0] * 28 + [127.5, 1.0]], dtype=torch.float64)
    codes, scales = ref.ckpt(x)
    assert scales.tolist() == [[127, 128, 0, 0]]
    assert codes[0, :4].tolist() == [127, -1, 0, 2]      # ties to even
    assert codes[0, 32:34].tolist() == [64, 0] and codes.shape == (1, 64)
    assert ref.unckpt(codes, scales, 34).shape == (1, 34)


def test_rope_frequencies():
    f, a = caj.rope_frequencies((44, 42, 42), device="cpu")
    assert f.dtype == torch.float64 and a.dtype == torch.int32 and f.shape == a.shape == (64,)
    assert a.tolist() == [0] * 22 + [1] * 21 + [2] * 21
    assert math.isclose(float(f[1]), 10000.0 ** (-2 / 44)) and float(f[22]) == 1.0
    lin, _ = caj.rope_frequencies(64, factor=4.0, device="cpu")
    plain, _ = caj.rope_frequencies(64, device="cpu")
    assert torch.equal(lin, plain / 4)
    parts, _ = caj.rope_frequencies(64, factor=4.0, original_length=4096, device="cpu")
    turns = plain * 4096 / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], plain[turns >= 32])
    assert torch.allclose(parts[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15)
    assert ((parts <= plain) & (parts >= plain / 4 * (1 - 1e-15))).all()
    for bad in (dict(dims=7), dict(dims=0), dict(dims=64, factor=0.5), dict(dims=64, base=0.0),
                dict(dims=64, fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            caj.rope_frequencies(device="cpu", **bad)


# ------------------------------------------------------------------------- refusals

def _pack(x=A, rows=4, cols=64, ld=64, dtype=1, codes=A, scales=A):
    return _lib.lib().caj_ckpt_pack(x, rows, cols, ld, dtype, codes, scales, None)


def _unpack(x=A, rows=4, cols=64, ld=64, dtype=1, codes=A, scales=A):
    return _lib.lib().caj_ckpt_unpack(codes, scales, rows, cols, ld, dtype, x, None)


@pytest.mark.parametrize("call", [_pack, _unpack])
@pytest.mark.parametrize("kw,want", [
    (dict(x=0), INVALID), (dict(codes=0), INVALID), (dict(scales=0), INVALID), (dict(x=A + 1), INVALID),
    (dict(codes=A + 8), INVALID), (dict(scales=A + 2), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(ld=63), INVALID), (dict(dtype=2), INVALID), (dict(x=A + 2, dtype=0), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(rows=1 << 62), UNSUPPORTED), (dict(rows=0, x=0), 0)])
def test_ckpt_refusals(call, kw, want):
    assert call(**kw) == want


def _table(pos=A, pos64=1, freq=A, axis=A, N=5, axes=3, pairs=64, mscale=1.0, cos=A, sin=A):
    return _lib.lib().caj_rope_table(pos, pos64, freq, axis, N, axes, pairs, mscale, cos, sin, None)


@pytest.mark.parametrize("kw,want", [
    (dict(pos=0), INVALID), (dict(pos=A + 4), INVALID), (dict(freq=0), INVALID), (dict(freq=A + 4), INVALID),
    (dict(axis=A + 2), INVALID), (dict(N=-1), INVALID), (dict(axes=0), INVALID), (dict(pairs=0), INVALID),
    (dict(mscale=float("nan")), INVALID), (dict(mscale=float("inf")), INVALID), (dict(cos=0), INVALID),
    (dict(sin=A + 1), INVALID), (dict(pos64=2), INVALID), (dict(N=1 << 40), UNSUPPORTED), (dict(N=0, pos=0), 0)])
def test_rope_table_refusals(kw, want):
    assert _table(**kw) == want


@pytest.mark.parametrize("kw", [dict(axes=(1 << 28) + 1), dict(pairs=(1 << 28) + 1)])
def test_rope_table_refuses_widths_past_32_bits(kw):
    assert _table(**kw) == UNSUPPORTED


@pytest.mark.parametrize("mscale", [2.0**126, -2.0**126, 1e300])
def test_rope_table_refuses_scales_past_fp32(mscale):
    assert _table(mscale=mscale) == INVALID
    assert _table(mscale=mscale, N=0) == INVALID
    assert _table(mscale=2.0**125, N=0) == 0


def _rope_shape(**kw):
    v = dict(B=1, N=5, Hq=4, Hk=2, D=64, pairs=32, dtype=1, norm=1, layout=0, gain_full=0, eps=1e-6, ldq=256,
             ldk=128, ldv=128, ldtq=256, ldtk=128, ldtv=128)
    v.update(kw)
    return _lib.QkRopeShapeC(*[v[n] for n, _ in _lib.QkRopeShapeC._fields_])


_FWD = ("xq", "xk", "xv", "txq", "txk", "txv", "gq", "gk", "cos", "sin")
_OUT = ("q", "k", "v", "tq", "tk", "tv")


def _fwd(ptrs=None, **kw):
    p = dict.fromkeys(_FWD + _OUT, A)
    p.update(ptrs or {})
    shape = _rope_shape(**kw)
    return _lib.lib().caj_qk_rope_fwd(*[p[n] for n in _FWD], ctypes.byref(shape), *[p[n] for n in _OUT], None)


_SHAPE_REFUSALS = [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID),
    (dict(D=0), INVALID), (dict(pairs=0), INVALID), (dict(pairs=40), INVALID), (dict(dtype=5), INVALID),
    (dict(norm=3), INVALID), (dict(norm=-1), INVALID), (dict(layout=2), INVALID), (dict(gain_full=2), INVALID),
    (dict(norm=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(D=96, pairs=32), UNSUPPORTED), (dict(D=512), UNSUPPORTED),
    (dict(pairs=20), UNSUPPORTED), (dict(Hq=129), UNSUPPORTED), (dict(B=1 << 16, N=1 << 16), UNSUPPORTED),
    (dict(B=1, N=(1 << 30) + 1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", _SHAPE_REFUSALS + [
    (dict(ldq=255), INVALID), (dict(ldq=248), INVALID), (dict(ldk=132), INVALID), (dict(ldv=64), INVALID),
    (dict(ldtq=128), INVALID), (dict(ldq=1 << 31), INVALID)])
def test_qk_rope_fwd_shape_refusals(kw, want):
    assert _fwd(**kw) == want


@pytest.mark.parametrize("ptrs", [dict(xq=0), dict(xk=0), dict(q=0), dict(k=A + 8), dict(xq=A + 8), dict(gq=0),
                                  dict(gk=A + 4), dict(cos=0), dict(sin=A + 8), dict(txk=0), dict(tq=0),
                                  dict(txv=0), dict(xv=0), dict(v=0), dict(xv=0, txv=0, tv=0)])
def test_qk_rope_fwd_pointer_refusals(ptrs):
    assert _fwd(ptrs) == INVALID


_BWD = ("dq", "dk", "dv", "xq", "xk", "sq", "sk", "gq", "gk", "cos", "sin")
_BOUT = ("dxq", "dxk", "dxv", "dgq", "dgk", "ws")


def _bwd(ptrs=None, ws_bytes=1 << 30, **kw):
    p = dict.fromkeys(_BWD + _BOUT, A)
    p.update(ptrs or {})
    shape = _rope_shape(**kw)
    return _lib.lib().caj_qk_rope_bwd(*[p[n] for n in _BWD], ctypes.byref(shape), *[p[n] for n in _BOUT], ws_bytes,
                                      None)


@pytest.mark.parametrize("kw,want", _SHAPE_REFUSALS)
def test_qk_rope_bwd_shape_refusals(kw, want):
    assert _bwd(**kw) == want
    size = ctypes.c_size_t(7)
    assert _lib.lib().caj_qk_rope_bwd_workspace(ctypes.byref(_rope_shape(**kw)), ctypes.byref(size)) == want


@pytest.mark.parametrize("ptrs", [dict(dq=0), dict(dk=A + 8), dict(dv=0), dict(dxq=0), dict(dxk=A + 8), dict(xq=0),
                                  dict(xk=A + 8), dict(sq=0), dict(dgq=0), dict(dgk=A + 2), dict(ws=0),
                                  dict(ws=A + 8), dict(gq=0)])
def test_qk_rope_bwd_pointer_refusals(ptrs):
    assert _bwd(ptrs) == INVALID


def test_qk_rope_bwd_workspace():
    size = ctypes.c_size_t(0)
    f = _lib.lib().caj_qk_rope_bwd_workspace
    assert f(ctypes.byref(_rope_shape()), ctypes.byref(size)) == 0 and size.value > 0
    assert _bwd(ws_bytes=size.value - 1) == INVALID
    assert f(ctypes.byref(_rope_shape(norm=0)), ctypes.byref(size)) == 0 and size.value == 0
    assert f(ctypes.byref(_rope_shape()), None) == INVALID


@pytest.mark.skipif(not _NO_GPU, reason="valid calls with fake pointers must not launch")
def test_valid_calls_reach_the_device_check():
    assert _pack() == _unpack() == _table() == _fwd() == _bwd() == CUDA
    assert _fwd(dict(txq=0, txk=0, txv=0, tq=0, tk=0, tv=0)) == CUDA
    assert _fwd(dict(gq=0, gk=0), norm=0) == CUDA
    assert _bwd(dict(xq=0, xk=0, sq=0, sk=0, gq=0, gk=0, dgq=0, dgk=0, ws=0), norm=0) == CUDA


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        caj.ckpt8_pack(x)
    with pytest.raises(ValueError):
        caj.ckpt8_unpack(caj.Ckpt8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 4, dtype=torch.uint8), (4, 64)))
    with pytest.raises(ValueError):
        caj.rope_table(torch.arange(4), torch.ones(8, dtype=torch.float64))
    t = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    tab = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        caj.qk_norm_rope_fwd(t, t, t, torch.ones(64), torch.ones(64), tab, tab, 2)
    h = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        caj.qk_norm_rope_bwd(h, h, h, t, t, torch.ones(64), torch.ones(64), tab, tab)


# --------------------------------------------------------------------- linear layers

@pytest.mark.parametrize("which", ["none", "gelu_tanh", "gelu", "silu"])
def test_linear_reference_against_differences(which):
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, tx, w, b, dy = rnd(5, 8), rnd(5, 8), rnd(16, 8), rnd(16), rnd(5, 16)
    f = lambda x_, w_, b_: ref.linear(x_, w_, b_, which, None, None, None)["y"][0]  # noqa: E731
    h = 1e-5
    num = (f(x + h * tx, w, b) - f(x - h * tx, w, b)) / (2 * h)
    assert torch.allclose(ref.linear(x, w, b, which, None, tx, None)["ty"][0], num, rtol=0, atol=1e-7)
    z = x @ w.t() + b
    got = ref.linear_bwd(dy, x, w, z, which)
    tw, tb = rnd(16, 8), rnd(16)
    assert abs(float((got["dx"][0] * tx).sum() - (dy * num).sum())) < 1e-6
    num_w = (f(x, w + h * tw, b) - f(x, w - h * tw, b)) / (2 * h)
    assert abs(float((got["dw"][0] * tw).sum() - (dy * num_w).sum())) < 1e-6
    num_b = (f(x, w, b + h * tb) - f(x, w, b - h * tb)) / (2 * h)
    assert abs(float((got["db"][0] * tb).sum() - (dy * num_b).sum())) < 1e-6


_LIN = ("x", "tx", "w", "bias", "res", "tres")
_LOUT = ("y", "ty", "codes", "scales", "ws")


def _lin_shape(**kw):
    v = dict(M=100, K=64, C=128, act=1, ldx=64, ldtx=64, ldres=128, ldtres=128, ldy=128)
    v.update(kw)
    return _lib.LinearActShapeC(*[v[n] for n, _ in _lib.LinearActShapeC._fields_])


def _lfwd(ptrs=None, ws_bytes=1 << 40, **kw):
    p = dict.fromkeys(_LIN + _LOUT, A)
    p.update(ptrs or {})
    return _lib.lib().caj_linear_act_fwd(*[p[n] for n in _LIN], ctypes.byref(_lin_shape(**kw)),
                                         *[p[n] for n in _LOUT], ws_bytes, None)


_LBWD = ("dy", "x", "xs", "w", "codes", "scales")
_LBOUT = ("dx", "dw", "db", "ws")


def _lbwd(ptrs=None, ws_bytes=1 << 40, **kw):
    p = dict.fromkeys(_LBWD + _LBOUT, A)
    p.update(ptrs or {})
    return _lib.lib().caj_linear_act_bwd(*[p[n] for n in _LBWD], ctypes.byref(_lin_shape(**kw)),
                                         *[p[n] for n in _LBOUT], ws_bytes, None)


_LIN_SHAPES = [(dict(M=0), INVALID), (dict(M=-5), INVALID), (dict(K=0), INVALID), (dict(C=0), INVALID),
               (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(K=60), UNSUPPORTED), (dict(C=129), UNSUPPORTED),
               (dict(M=1 << 31), UNSUPPORTED), (dict(K=1 << 25), UNSUPPORTED),
               (dict(M=1 << 30, C=1 << 20), UNSUPPORTED), (dict(K=1 << 24, C=1 << 24), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", _LIN_SHAPES)
def test_linear_shape_refusals(kw, want):
    size = ctypes.c_size_t(0)
    assert _lfwd(**kw) == want and _lbwd(**kw) == want
    assert _lib.lib().caj_linear_act_fwd_workspace(ctypes.byref(_lin_shape(**kw)), 0, ctypes.byref(size)) == want
    assert _lib.lib().caj_linear_act_bwd_workspace(ctypes.byref(_lin_shape(**kw)), 0, ctypes.byref(size)) == want


@pytest.mark.parametrize("kw", [dict(ldx=56), dict(ldx=68), dict(ldtx=63), dict(ldres=120), dict(ldtres=130),
                                dict(ldx=-64)])
def test_linear_fwd_row_refusals(kw):
    assert _lfwd(**kw) == INVALID


@pytest.mark.parametrize("ptrs", [dict(x=0), dict(w=0), dict(y=0), dict(x=A + 8), dict(tx=A + 2), dict(w=A + 8),
                                  dict(bias=A + 2), dict(res=A + 8), dict(tres=A + 8), dict(tx=0), dict(ty=0),
                                  dict(codes=0), dict(scales=0), dict(scales=A + 2), dict(codes=A + 16),
                                  dict(tx=0, ty=0)])
def test_linear_fwd_pointer_refusals(ptrs):
    assert _lfwd(ptrs) == INVALID  # the last: tres without tx


@pytest.mark.parametrize("ptrs", [dict(dy=0), dict(dy=A + 8), dict(w=0), dict(x=0), dict(x=A + 8), dict(xs=A + 1),
                                  dict(codes=0), dict(scales=0), dict(dx=A + 8), dict(dw=A + 8), dict(db=A + 2),
                                  dict(ws=0), dict(ws=A + 128), dict(dx=0, dw=0, db=0)])
def test_linear_bwd_pointer_refusals(ptrs):
    assert _lbwd(ptrs) == INVALID


def test_linear_workspaces():
    L, size = _lib.lib(), ctypes.c_size_t(0)
    assert L.caj_linear_act_fwd_workspace(ctypes.byref(_lin_shape(M=4)), 1, ctypes.byref(size)) == 0 and size.value == 0
    big = dict(M=256, K=8192, ldx=8192, ldtx=8192)
    assert L.caj_linear_act_fwd_workspace(ctypes.byref(_lin_shape(**big)), 0, ctypes.byref(size)) == 0
    assert size.value > 0  # one tile of a long contraction is split
    assert _lfwd(ws_bytes=size.value - 1, ptrs=dict(tx=0, ty=0, tres=0), **big) == INVALID
    assert L.caj_linear_act_fwd_workspace(ctypes.byref(_lin_shape()), 2, ctypes.byref(size)) == INVALID
    assert L.caj_linear_act_bwd_workspace(ctypes.byref(_lin_shape()), 1, None) == INVALID
    assert L.caj_linear_act_bwd_workspace(ctypes.byref(_lin_shape()), 1, ctypes.byref(size)) == 0
    assert _lbwd(ws_bytes=size.value - 1) == INVALID


@pytest.mark.skipif(not _NO_GPU, reason="valid calls with fake pointers must not launch")
def test_valid_linear_calls_reach_the_device_check():
    assert _lfwd() == _lbwd() == CUDA
    assert _lfwd(dict.fromkeys(("tx", "ty", "tres", "res", "bias", "codes", "scales"), 0)) == CUDA
    assert _lbwd(dict(xs=0)) == _lbwd(dict(xs=0, codes=0, scales=0), act=0) == CUDA
    assert _lbwd(dict(dx=0, w=0)) == _lbwd(dict(dw=0, x=0, xs=0)) == CUDA


def test_linear_python_refuses_host_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        caj.linear_act_fwd(x, w)
    with pytest.raises(ValueError):
        caj.linear_act_bwd(torch.zeros(4, 8, dtype=torch.bfloat16), x, w)
