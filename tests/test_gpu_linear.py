"""Linear layers with their epilogue on the GPU (values, tangents, gradients, checkpoints)
against their 64-bit forms. The reference returns, element by element, what fp32 arithmetic
may lose before the output's own rounding of half a step; nothing else is allowed."""
import pytest
import torch

import block_reference as ref
import masked_attention_jvp_b200 as caj
from masked_attention_jvp_b200 import _lib

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rnd(g, *s, std=1.0):
    return (torch.randn(*s, generator=g) * std).to(BF)


def close(got, pair):
    want, loss = pair
    assert got.shape == want.shape
    half = ref.HALF[got.dtype]
    bad = (ref.d(got) - want).abs() - (half * want.abs() + (1 + half) * loss)
    assert float(bad.max()) <= 0, (float(bad.max()), float((ref.d(got) - want).abs().max()))


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def run_fwd(M, K, C, which, bias, residual, tangent, pre, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, w = rnd(g, M, K), rnd(g, C, K, std=K ** -0.5)
    b = rnd(g, C, std=0.5) if bias else None
    res = rnd(g, M, C) if residual else None
    tx = rnd(g, M, K) if tangent else None
    tres = rnd(g, M, C) if tangent and residual else None
    xd, wd, bd, rd, txd, trd = cuda(x, w, b, res, tx, tres)
    y, ty, kept = caj.linear_act_fwd(xd, wd, bd, act=which, residual=rd, tx=txd, tresidual=trd, save_pre=pre)
    torch.cuda.synchronize()
    caj.device_status()
    want = ref.linear(*[None if t is None else ref.d(t) for t in (x, w, b)], which,
                      *[None if t is None else ref.d(t) for t in (res, tx, tres)])
    close(y, want["y"])
    assert (ty is None) == (not tangent) and (kept is None) == (not pre)
    if tangent:
        close(ty, want["ty"])
    if pre:
        z, ez = want["z"]
        nb = -(-C // 32)
        codes, scales = kept.codes.cpu().long(), kept.scales.cpu().long()
        assert codes.shape == (M, 32 * nb) and scales.shape == (M, 4 * -(-nb // 4))
        assert not codes[:, C:].any() and not scales[:, nb:].any()
        unit = (2.0 ** (scales[:, :nb].double() - 127)).repeat_interleave(32, 1)[:, :C]
        dec = ref.unckpt(kept.codes, kept.scales, C)
        assert bool(((dec - z).abs() <= unit / 2 + ez).all())
        top = torch.nn.functional.pad(z.abs() + ez, (0, 32 * nb - C)).view(M, nb, 32).amax(-1)
        # the smallest unit that holds the block: no more than twice what its largest needs
        assert bool((2.0 ** (scales[:, :nb].double() - 127) * 63.5 <= top + 1e-30).all())
        assert torch.equal(ref.d(caj.ckpt8_unpack(kept)), dec)
    return y, ty


FWD = [  # M, K, C, act, bias, residual, tangent, checkpoint
    (1, 8, 8, "none", False, False, False, False),
    (1, 1536, 1536, "gelu_tanh", True, False, False, True),
    (1, 264, 6000, "silu", True, True, True, False),
    (2, 2056, 2600, "gelu", True, True, True, True),
    (3, 72, 40, "gelu", False, True, True, True),
    (4, 512, 4800, "gelu_tanh", True, True, True, True),
    (5, 1000, 104, "silu", True, False, False, True),
    (8, 256, 264, "none", True, True, False, False),
    (5, 64, 96, "gelu_tanh", True, True, True, True),     # ten rows: the tile kernel
    (9, 8, 8, "none", False, False, False, True),
    (33, 72, 264, "gelu_tanh", True, True, False, True),
    (64, 128, 256, "silu", True, False, True, False),
    (127, 64, 40, "gelu", True, True, True, True),
    (128, 200, 512, "none", True, True, True, False),
    (129, 64, 520, "gelu_tanh", False, False, True, True),
    (257, 1536, 200, "gelu", True, True, False, False),
    (300, 4096, 256, "gelu_tanh", True, True, True, True),   # split contraction
    (100, 8192, 72, "silu", True, True, False, True),        # split contraction
    (70, 4104, 2056, "none", True, False, True, False),
    (1111, 64, 2568, "gelu_tanh", True, True, True, True),   # more tiles than pairs
    (2050, 128, 2560, "silu", True, True, False, True),
]


@pytest.mark.parametrize("case", FWD)
def test_forward(case):
    run_fwd(*case, seed=sum(case[:3]))


def test_some_sizes_split_and_some_do_not():
    import ctypes
    n = ctypes.c_size_t(0)
    got = []
    for M, K, C, tan in ((300, 4096, 256, 1), (100, 8192, 72, 0), (1111, 64, 2568, 1)):
        s = _lib.LinearActShapeC(M, K, C, 0, K)
        assert _lib.lib().caj_linear_act_fwd_workspace(ctypes.byref(s), tan, ctypes.byref(n)) == 0
        got.append(n.value > 0)
    assert got == [True, True, False]


BWD = [  # M, K, C, act, checkpoint of x
    (1, 8, 8, "none", False),
    (1, 256, 1536, "gelu_tanh", True),
    (7, 72, 40, "silu", True),
    (64, 64, 256, "gelu", False),
    (129, 264, 200, "gelu_tanh", True),
    (300, 512, 520, "none", True),
    (1000, 1536, 256, "silu", False),
    (5000, 256, 264, "gelu_tanh", True),      # a long contraction over the rows
    (700, 64, 5000, "gelu", True),
    (2100, 2560, 136, "none", False),
]


def bwd_inputs(M, K, C, which, kept, seed):
    g = torch.Generator().manual_seed(seed)
    dy, x, w = rnd(g, M, C), rnd(g, M, K), rnd(g, C, K, std=C ** -0.5)
    z = (torch.randn(M, C, generator=g) * 1.5).float()
    dyd, xd, wd = cuda(dy, x, w)
    seen = ref.d(x)
    if kept:
        xd = caj.ckpt8_pack(xd)
        seen = ref.unckpt(xd.codes, xd.scales, K)
    pre = caj.ckpt8_pack(z.cuda()) if which != "none" else None
    zs = ref.unckpt(pre.codes, pre.scales, C) if pre else None
    return dyd, xd, wd, pre, ref.linear_bwd(ref.d(dy), seen, ref.d(w), zs, which)


@pytest.mark.parametrize("case", BWD)
def test_backward(case):
    M, K, C, which, kept = case
    dyd, xd, wd, pre, want = bwd_inputs(*case, seed=sum(case[:3]))
    dx, dw, db = caj.linear_act_bwd(dyd, xd, wd, act=which, pre=pre)
    torch.cuda.synchronize()
    caj.device_status()
    close(dx, want["dx"])
    close(dw, want["dw"])
    close(db, want["db"])
    again = caj.linear_act_bwd(dyd, xd, wd, act=which, pre=pre)
    for a, b in zip((dx, dw, db), again):
        assert torch.equal(a, b)
    only = caj.linear_act_bwd(dyd, None, wd, act=which, pre=pre, need=(True, False), bias=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    only = caj.linear_act_bwd(dyd, xd, wd, act=which, pre=pre, need=(False, True), bias=False)
    assert only[0] is None and torch.equal(only[1], dw)
    only = caj.linear_act_bwd(dyd, None, wd, act=which, pre=pre, need=(False, False))
    assert only[0] is None and only[1] is None and torch.equal(only[2], db)


def test_strided_rows_and_leading_shapes():
    g = torch.Generator().manual_seed(1)
    wide = rnd(g, 2, 150, 400).cuda()
    w, b = rnd(g, 136, 128, std=0.1).cuda(), rnd(g, 136).cuda()
    x, tx, res, tres = wide[..., :128], wide[..., 128:256], wide[..., 8:144], wide[..., 256:392]
    got = caj.linear_act_fwd(x, w, b, "silu", res, tx, tres)
    want = caj.linear_act_fwd(*[t.contiguous() for t in (x, w, b)], "silu", res.contiguous(), tx.contiguous(),
                              tres.contiguous())
    assert got[0].shape == (2, 150, 136)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    few = caj.linear_act_fwd(x[:1, :2], w, b, "silu", res[:1, :2], tx[:1, :2], tres[:1, :2])
    ref_few = caj.linear_act_fwd(*[t[:1, :2].contiguous() if t.dim() == 3 else t for t in (x, w, b)], "silu",
                                 res[:1, :2].contiguous(), tx[:1, :2].contiguous(), tres[:1, :2].contiguous())
    assert torch.equal(few[0], ref_few[0]) and torch.equal(few[1], ref_few[1])
    dy = wide[..., 200:336]
    for a, c in zip(caj.linear_act_bwd(dy, x, w), caj.linear_act_bwd(dy.contiguous(), x.contiguous(), w)):
        assert torch.equal(a, c)


def test_no_rows():
    w = torch.zeros(16, 64, dtype=BF, device="cuda")
    x, dy = w.new_zeros(3, 0, 64), w.new_zeros(3, 0, 16)
    y, ty, pre = caj.linear_act_fwd(x, w, act="silu", tx=x, save_pre=True)
    assert y.shape == ty.shape == (3, 0, 16) and pre.codes.shape == (0, 32)
    dx, dw, db = caj.linear_act_bwd(dy, x, w, act="silu", pre=pre)
    assert dx.shape == (3, 0, 64) and not dw.any() and not db.any() and dw.shape == (16, 64)


@pytest.mark.parametrize("M", [2, 200])
def test_infinities_and_nans_stay_in_their_rows(M):
    g = torch.Generator().manual_seed(2)
    x, w = rnd(g, M, 128), rnd(g, 64, 128, std=0.1)
    clean, _, _ = caj.linear_act_fwd(x.cuda(), w.cuda(), act="gelu_tanh")
    x[1, 5], x[0, 3] = float("nan"), 3e38
    y, _, pre = caj.linear_act_fwd(x.cuda(), w.cuda(), act="gelu_tanh", save_pre=True)
    assert torch.isnan(y[1]).all() and torch.isnan(caj.ckpt8_unpack(pre)[1]).all()
    assert (pre.scales[1, :2] == 255).all()
    if M > 2:
        assert torch.equal(y[2:], clean[2:])


def test_few_rows_agree_with_tiles():
    """The streaming kernels (one row, up to 64) and the tile kernel sum in different orders:
    each is within its bound of the same reference."""
    for M in (1, 2, 8, 9, 17, 33, 64, 65):
        run_fwd(M, 520, 264, "gelu_tanh", True, True, False, True, seed=3)
        run_fwd(M, 1544, 72, "silu", True, True, True, True, seed=4)


def test_bounded_waits_report_and_the_context_survives():
    L = _lib.lib()
    g = torch.Generator().manual_seed(3)
    # more than 64 rows: the kernels with copies to wait for
    x, tx, w = rnd(g, 128, 64).cuda(), rnd(g, 128, 64).cuda(), rnd(g, 64, 64).cuda()
    pre = caj.ckpt8_pack(x)
    calls = [lambda: caj.linear_act_fwd(x, w, act="silu"), lambda: caj.linear_act_fwd(x, w, act="silu", tx=tx),
             lambda: caj.linear_act_bwd(x, x, w, act="silu", pre=pre, need=(True, False)),
             lambda: caj.linear_act_bwd(x, x, w, act="silu", pre=pre, need=(False, True))]
    want = [call() for call in calls]
    caj.device_status()
    assert L.caj_set_wait_timeout_ms(100.0) == _lib.CAJ_OK
    try:
        for call in calls:
            assert L.caj_debug_set_fault(1) == _lib.CAJ_OK
            call()
            with pytest.raises(caj.CajError) as err:
                caj.device_status()
            assert err.value.status == _lib.CAJ_ERR_DEVICE_TIMEOUT
            assert L.caj_last_device_error_code() & 0xFF0 == 0x120
            caj.device_status()
    finally:
        L.caj_debug_set_fault(0)
        L.caj_set_wait_timeout_ms(0.0)
    for call, w_ in zip(calls, want):
        for a, b in zip(call(), w_):
            assert a is None and b is None or torch.equal(a, b)
    caj.device_status()


def test_other_streams_and_graphs():
    g = torch.Generator().manual_seed(5)
    x, tx, w, b = rnd(g, 300, 1024).cuda(), rnd(g, 300, 1024).cuda(), rnd(g, 256, 1024, std=0.03).cuda(), rnd(g, 256).cuda()

    def step():  # split contractions: both directions use a workspace
        y, ty, pre = caj.linear_act_fwd(x, w, b, "gelu_tanh", tx=tx, save_pre=True)
        return (y, ty) + caj.linear_act_bwd(y, caj.ckpt8_pack(x), w, "gelu_tanh", pre)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for s, t in zip(want, got):
        assert torch.equal(s, t)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    x.mul_(0.5)
    want = step()
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    caj.device_status()
    for _, out in graphs:
        for s, t in zip(want, out):
            assert torch.equal(s, t)


def test_two_calls_at_once():
    """Two streams, each with its own workspace; both kernels take every SM that is free."""
    g = torch.Generator().manual_seed(11)
    a = [rnd(g, 700, 1024).cuda(), rnd(g, 512, 1024, std=0.03).cuda()]
    b = [rnd(g, 300, 4096).cuda(), rnd(g, 256, 4096, std=0.02).cuda()]
    want = [caj.linear_act_fwd(*t, act="silu", tx=t[0], save_pre=True) for t in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):
        for s, t in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(caj.linear_act_fwd(*t, act="silu", tx=t[0], save_pre=True))
    torch.cuda.synchronize()
    caj.device_status()
    for i, (y, ty, pre) in enumerate(got):
        w = want[i % 2]
        assert torch.equal(y, w[0]) and torch.equal(ty, w[1])
        assert torch.equal(pre.codes, w[2].codes) and torch.equal(pre.scales, w[2].scales)


def test_outputs_past_32_bits():
    """More than 2^31 outputs: the last rows must equal a call on them alone (one block of the
    contraction, so both sum alike)."""
    g = torch.Generator().manual_seed(12)
    M, K, C = 360_000, 64, 6144
    x, w = torch.zeros(M, K, dtype=BF, device="cuda"), rnd(g, C, K, std=0.2).cuda()
    tail = 128 * 2 + 128 + 64
    x[-tail:] = rnd(g, tail, K).cuda()
    y, ty, pre = caj.linear_act_fwd(x, w, act="gelu_tanh", tx=x, save_pre=True)
    assert y.numel() > 2 ** 31
    few = caj.linear_act_fwd(x[-tail:], w, act="gelu_tanh", tx=x[-tail:], save_pre=True)
    assert torch.equal(y[-tail:], few[0]) and torch.equal(ty[-tail:], few[1])
    assert torch.equal(pre.codes[-tail:], few[2].codes) and torch.equal(pre.scales[-tail:], few[2].scales)
    dx, dw, db = caj.linear_act_bwd(y, x, w, act="gelu_tanh", pre=pre, need=(True, False), bias=False)
    want = caj.linear_act_bwd(few[0], x[-tail:], w, act="gelu_tanh", pre=few[2], need=(True, False), bias=False)
    rel = float((dx[-tail:].float() - want[0].float()).norm() / want[0].float().norm())
    assert rel <= 2.0 ** -8  # the contraction may be split differently: one rounding apart
    caj.device_status()


@pytest.mark.parametrize("M,K,C", [(1560, 192, 1536), (1000, 256, 1480), (1560, 64, 1448)])
@pytest.mark.parametrize("tangent", [False, True])
def test_sizes_of_every_tile_width(M, K, C, tangent):
    """A frame's worth of rows, where the width of the tiles is chosen by their number."""
    run_fwd(M, K, C, "gelu_tanh", True, True, tangent, True, seed=9)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,K,C", [(64, 256, 512), (700, 512, 2568), (1560, 1536, 1536)])
def test_bias_gradients_back_to_back(M, K, C, act):
    """The bias's sums run beside the products: calls in a row, each on what the one before left
    and with its inputs overwritten at once, give what the same calls give one at a time."""
    g = torch.Generator().manual_seed(M)
    dys = [rnd(g, M, C).cuda() for _ in range(4)]
    x, w = rnd(g, M, K).cuda(), rnd(g, C, K, std=K ** -0.5).cuda()
    pre = caj.ckpt8_pack(rnd(g, M, C).cuda()) if act != "none" else None

    def run(alone):
        dy, outs = torch.empty_like(dys[0]), []
        for d in dys:
            dy.copy_(d)
            dx, dw, db = caj.linear_act_bwd(dy, x, w, act=act, pre=pre)
            if alone:
                torch.cuda.synchronize()
            # the library's own kernel reads dx right behind, its predecessor's inputs change
            y, _, _ = caj.linear_act_fwd(dx, w)
            again = caj.linear_act_bwd(y, x, w, act=act, pre=pre)
            dy.zero_()
            outs += [dx, dw, db, *again]
            if alone:
                torch.cuda.synchronize()
        return outs

    want, got = run(True), run(False)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(False)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # the sums themselves: fp32 over M rows, off by at most M steps of the sum of magnitudes
    if act == "none":
        for i, d in enumerate(dys):
            d = d.double()
            assert bool(((want[6 * i + 2] - d.sum(0)).abs() <= M * 2.0**-24 * d.abs().sum(0)).all())


@pytest.mark.parametrize("M,K,C,act,tangent", [(1700, 840, 2568, "none", True), (600, 3160, 4104, "silu", False),
                                               (2100, 4104, 1544, "none", False)])
def test_rows_at_odd_multiples_of_16_bytes(M, K, C, act, tangent):
    """Large products of such inputs run on copies in even rows: the same values, to the bit, as
    from inputs that lie in even rows, and the inputs stay as they are."""
    g = torch.Generator().manual_seed(C)
    x, tx, dy = rnd(g, M, K).cuda(), rnd(g, M, K).cuda() if tangent else None, rnd(g, M, C).cuda()
    w, b = rnd(g, C, K, std=K ** -0.5).cuda(), rnd(g, C).cuda()

    def even(t):
        if t is None:
            return None
        wide = torch.full((t.shape[0], -(-t.shape[1] // 64) * 64), float("nan"), dtype=BF, device="cuda")
        wide[:, :t.shape[1]] = t
        return wide[:, :t.shape[1]]

    want = caj.linear_act_fwd(even(x), w, b, act=act, tx=even(tx), save_pre=True)
    for _ in range(2):
        got = caj.linear_act_fwd(x, w, b, act=act, tx=tx, save_pre=True)
        assert torch.equal(got[0], want[0]) and (not tangent or torch.equal(got[1], want[1]))
        assert torch.equal(got[2].codes, want[2].codes) and torch.equal(got[2].scales, want[2].scales)
    pre = want[2] if act != "none" else None
    kept = x.clone(), dy.clone()
    for need in ((True, True), (True, False), (False, True)):
        a = caj.linear_act_bwd(even(dy), even(x), w, act=act, pre=pre, need=need)
        for s, t in zip(a, caj.linear_act_bwd(dy, x, w, act=act, pre=pre, need=need)):
            assert s is None and t is None or torch.equal(s, t)
    assert torch.equal(x, kept[0]) and torch.equal(dy, kept[1])
