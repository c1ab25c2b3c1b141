"""Block operators on the GPU against their 64-bit forms: rotary tables, norm + rotation
(forward, tangent, gradient), 8-bit checkpoints.

Tolerances, element by element: half a step of the output's type relative to the value, plus
what fp32 arithmetic may lose, K * 2^-24 times the sum of the magnitudes of the terms (which
the reference returns), K counting the roundings on the longest path to an element."""
import pytest
import torch

import block_reference as ref
import masked_attention_jvp_b200 as caj
from masked_attention_jvp_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def close(got, want, terms, K):
    assert got.shape == want.shape
    err = (ref.d(got) - want).abs()
    bound = ref.HALF[got.dtype] * want.abs() + K * U * terms
    worst = float((err - bound).max()) if err.numel() else 0.0
    assert worst <= 0, (worst, float(err.max()))


# ---------------------------------------------------------------- 8-bit checkpoints

def _rows(C, rows, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, C, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))
    x[:, ::7] *= 20
    return x.to(dtype)


def check_pack(x_dev):
    x = x_dev.cpu()
    c = caj.ckpt8_pack(x_dev)
    codes, scales = ref.ckpt(x.reshape(-1, x.shape[-1]))
    assert torch.equal(c.codes.cpu().long(), codes)
    assert torch.equal(c.scales.cpu().long(), scales)
    for dtype in (BF, F32):
        back = caj.ckpt8_unpack(c, dtype)
        want = ref.unckpt(codes, scales, x.shape[-1]).reshape(x.shape)
        assert back.shape == x.shape and back.dtype == dtype
        assert torch.equal(torch.isnan(back.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(ref.d(back)), torch.nan_to_num(want))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,C", [(1, 1), (1, 8), (3, 31), (5, 32), (4, 33), (7, 40), (2, 1000), (3, 1536),
                                    (70, 64), (1, 4104), (130, 7)])
def test_ckpt_codes_and_values(rows, C, dtype):
    check_pack(_rows(C, rows, dtype, 10 * rows + C).cuda())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ckpt_special_values(dtype):
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    rows = [torch.zeros(96), torch.full((96,), big), torch.full((96,), tiny), torch.full((96,), tiny / 4),
            torch.full((96,), -0.0), torch.arange(96).float() - 48, torch.full((96,), 127.5), torch.full((96,), 127.0),
            torch.arange(96) / 2 - 24.0]
    x = torch.stack(rows)
    x = torch.cat([x, x, x])
    x[9, 3], x[10, 40], x[11, 95], x[12, 0] = float("inf"), float("-inf"), float("nan"), big
    check_pack(x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ckpt_strided_and_unaligned_rows(dtype):
    base = _rows(200, 24, dtype, 5).cuda()
    check_pack(base[:, 8:136])            # a slice on a 16-byte boundary
    check_pack(base[:, 3:100])            # one that is not
    check_pack(base.view(4, 6, 200)[:, :, :64])
    check_pack(base.view(4, 6, 200)[:, 2:3])
    check_pack(base.t())                  # laid out anew by the call
    check_pack(base[:0].reshape(0, 200))


# ------------------------------------------------------------------------ rope table

@pytest.mark.parametrize("N,axes,P,start,dt", [(1, 1, 1, 0, torch.int64), (7, 3, 9, 5, torch.int32),
                                               (1560, 3, 64, 0, torch.int64), (333, 1, 64, 3999999, torch.int32),
                                               (65, 1, 32, (1 << 40) + 12345, torch.int64), (19, 2, 5, -400, torch.int64)])
def test_rope_table(N, axes, P, start, dt):
    dims = [2 * ((P + a) // axes) for a in range(axes)]
    freq, axis = caj.rope_frequencies(dims)
    pos = torch.stack([start + 3 * a + torch.arange(N) // (a + 1) for a in range(axes)], 1).to(dt).cuda()
    for m in (1.0, 1.25):
        cos, sin = caj.rope_table(pos, freq, axis, mscale=m)
        # angles in whole turns with Python's integers would do; 64-bit products suffice
        # below 2^30, beyond it the exact product is split
        import fractions
        import math
        two_pi = fractions.Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799")
        rows = range(0, N, max(1, N // 40))
        for n in rows:
            for i in range(P):
                a = fractions.Fraction(int(pos[n, int(axis[i])])) * fractions.Fraction(float(freq[i]))
                r = float(a - two_pi * round(a / two_pi))
                # the reduced angle and each series round a few times: 4 half-steps at 1
                assert abs(float(cos[n, i]) - m * math.cos(r)) <= m * 4 * U + U * m
                assert abs(float(sin[n, i]) - m * math.sin(r)) <= m * 4 * U + U * m


@pytest.mark.parametrize("P", [3, 61, 64])
@pytest.mark.parametrize("dt", [torch.int32, torch.int64])
def test_rope_table_long(P, dt):
    """More rows than threads at work: every thread walks, the last ones end early."""
    N, m = 30011, 1.2079
    freq, axis = caj.rope_frequencies([2 * ((P + a) // 3) for a in range(3)])
    pos = torch.stack([(torch.arange(N) * (7 + a)) % 65521 - 1000 * a for a in range(3)], 1).to(dt).cuda()
    cos, sin = caj.rope_table(pos, freq, axis, mscale=m)
    angle = pos[:, axis.long()].double() * freq  # below 2^17: off by 2^-37
    for got, want in ((cos, angle.cos() * m), (sin, angle.sin() * m)):
        # the reduced angle and each series round a few times: 4 half-steps at 1, and the result's own
        assert float((got - want).abs().max()) <= m * 5 * U
    assert float((cos.double() ** 2 + sin.double() ** 2 - m * m).abs().max()) <= 2 * m * m * 5 * U * 2


@pytest.mark.parametrize("N,P", [(1, 1), (7, 61), (9, 62), (6, 64), (10001, 3)])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_rope_table_writes_its_rows_alone(N, P, off):
    """Tables at any fp32 address: the same values, and nothing before or behind them."""
    freq, axis = caj.rope_frequencies(2 * P)
    pos = torch.arange(N, device="cuda") + 77
    want = caj.rope_table(pos, freq, axis)
    bufs = [torch.full((off + N * P + 8,), 7.0, device="cuda") for _ in range(2)]
    st = _lib.lib().caj_rope_table(pos.data_ptr(), 1, freq.data_ptr(), axis.data_ptr(), N, 1, P, 1.0,
                                   *[b.data_ptr() + 4 * off for b in bufs], torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for b, w in zip(bufs, want):
        assert torch.equal(b[off:off + N * P].view(N, P), w)
        assert bool((b[:off] == 7).all()) and bool((b[off + N * P:] == 7).all())


def test_rope_table_one_axis_and_bad_axis():
    freq, axis = caj.rope_frequencies(16)
    pos = torch.arange(5, device="cuda")
    a, b = caj.rope_table(pos, freq), caj.rope_table(pos[:, None].contiguous(), freq, axis)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    axis[3], axis[5] = 1, -1
    cos, sin = caj.rope_table(pos, freq, axis)
    bad = torch.zeros(8, dtype=torch.bool, device="cuda")
    bad[3] = bad[5] = True
    assert torch.equal(torch.isnan(cos), bad.expand(5, 8)) and torch.equal(torch.isnan(sin), bad.expand(5, 8))
    assert caj.rope_table(pos[:0], freq)[0].shape == (0, 8)


# ---------------------------------------------------------------- norm and rotation

CASES = [  # B, N, H, Hk, D, P, norm, layout, dtype, gains over all channels
    (1, 1, 1, 1, 64, 32, "head", "interleaved", BF, False),
    (1, 37, 12, 12, 128, 64, "head", "interleaved", BF, False),
    (2, 19, 12, 12, 128, 32, "head", "half", BF, True),
    (3, 5, 4, 2, 64, 8, "token", "half", BF, True),
    (1, 33, 12, 12, 128, 64, "token", "interleaved", F32, True),
    (2, 50, 8, 1, 64, 16, "head", "half", F32, False),
    (1, 9, 3, 5, 32, 16, "head", "half", BF, True),
    (1, 7, 32, 32, 256, 128, "token", "half", BF, True),
    (1, 6, 32, 4, 256, 64, "head", "interleaved", F32, False),
    (2, 11, 5, 5, 64, 24, "none", "interleaved", BF, False),
    (1, 13, 7, 3, 128, 56, "none", "half", F32, False),
    (1, 3000, 2, 2, 64, 32, "head", "half", BF, False),
    (1, 5, 32, 32, 256, 128, "token", "half", F32, True),     # the widest token, one token's copies at a time
    (2, 400, 64, 8, 128, 64, "head", "interleaved", BF, True),
    (1, 9, 256, 16, 32, 16, "token", "interleaved", BF, True),
    (3, 1, 12, 12, 128, 64, "head", "half", BF, False),       # single tokens of a batch
    (500, 2, 3, 3, 64, 32, "token", "half", F32, True),       # walks that cross many sequences
]


def make(case, seed, std=1.5):
    B, N, H, Hk, D, P, norm, layout, dtype, full = case
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = [(rnd(B, N, h * D) * std).to(dtype) for h in (H, Hk, Hk)]
    tx = [rnd(B, N, h * D).to(dtype) for h in (H, Hk, Hk)]
    gains = [None, None]
    if norm != "none":
        gains = [1 + 0.2 * rnd(h * D if full else D) for h in (H, Hk)]
    th = rnd(N, P) * 50
    return x, tx, gains, th.cos(), th.sin()


def dev(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("case", CASES)
def test_norm_rope_forward_and_tangent(case):
    B, N, H, Hk, D, P, norm, layout, dtype, full = case
    x, tx, gains, cos, sin = make(case, 1)
    args = [dev(t) for t in (*x, *gains, cos, sin)]
    kw = dict(eps=1e-5, norm=norm, layout=layout)
    got = caj.qk_norm_rope_fwd(*args, H, Hk, txq=dev(tx[0]), txk=dev(tx[1]), txv=dev(tx[2]), **kw)
    primal = caj.qk_norm_rope_fwd(*args, H, Hk, **kw)
    assert len(got) == 6 and len(primal) == 3
    for a, b in zip(got, primal):
        assert torch.equal(a, b)
    K = 96 + max(H, Hk)  # sums: 8 + 5 + heads in a row; then scales, products and the rotation
    for i, h in enumerate((H, Hk)):
        y, ty, ay, aty = ref.norm_rope(ref.d(x[i]), ref.d(tx[i]), None if norm == "none" else ref.d(gains[i]),
                                       ref.d(cos), ref.d(sin), h, 1e-5, norm, layout)
        close(got[i], y, ay, K)
        close(got[3 + i], ty, aty, K)
    for j, src in ((2, x[2]), (5, tx[2])):
        assert torch.equal(got[j].cpu(), src.view(B, N, Hk, D).transpose(1, 2))
    two = caj.qk_norm_rope_fwd(*args[:2], None, *args[3:], H, Hk, **kw)
    assert len(two) == 2 and torch.equal(two[0], got[0]) and torch.equal(two[1], got[1])


@pytest.mark.parametrize("kept", ["tensor", "ckpt8"])
@pytest.mark.parametrize("case", CASES)
def test_norm_rope_backward(case, kept):
    B, N, H, Hk, D, P, norm, layout, dtype, full = case
    if norm == "none" and kept == "ckpt8":
        pytest.skip("no inputs are read")
    x, _, gains, cos, sin = make(case, 2)
    g = torch.Generator().manual_seed(9)
    dy = [torch.randn(B, h, N, D, generator=g).to(dtype) for h in (H, Hk, Hk)]
    xs, seen = [None, None], [None, None]
    if norm != "none":
        for i in range(2):
            xs[i] = dev(x[i])
            seen[i] = ref.d(x[i])
            if kept == "ckpt8":
                xs[i] = caj.ckpt8_pack(xs[i])
                seen[i] = ref.unckpt(xs[i].codes, xs[i].scales, x[i].shape[-1]).view(x[i].shape)
    kw = dict(eps=1e-5, norm=norm, layout=layout)
    call = lambda dv: caj.qk_norm_rope_bwd(dev(dy[0]), dev(dy[1]), dv, *xs, dev(gains[0]), dev(gains[1]),  # noqa: E731
                                           dev(cos), dev(sin), **kw)
    got = call(dev(dy[2]))
    K = 96 + max(H, Hk)
    for i in range(2):
        dx, dg, adx, adg = ref.norm_rope_bwd(ref.d(dy[i]), seen[i], None if norm == "none" else ref.d(gains[i]),
                                             ref.d(cos), ref.d(sin), 1e-5, norm, layout)
        close(got[i], dx, adx, K)
        if norm == "none":
            assert got[3 + i] is None
        else:  # at most every token and head in a row
            close(got[3 + i], dg, adg, K + min(B * N * (1 if full else (H, Hk)[i]), 4096))
    assert torch.equal(got[2].cpu(), dy[2].transpose(1, 2).reshape(B, N, Hk * D))
    again = call(None)
    assert again[2] is None
    for a, b in zip(got[:2] + got[3:], again[:2] + again[3:]):
        assert a is None and b is None or torch.equal(a, b)  # the same sums in the same order


WIDE = [  # tokens whose heads are shared out between blocks, and those next to them
    (1, 700, 40, 40, 128, 64, "head", "interleaved", BF, False),
    (2, 301, 64, 8, 128, 64, "head", "half", BF, False),      # the second share has no key heads
    (1, 160, 33, 33, 128, 32, "head", "half", BF, True),      # shares of 17 and 16 heads
    (1, 450, 8, 48, 128, 64, "head", "half", F32, True),
    (3, 90, 127, 5, 64, 32, "head", "interleaved", F32, False),
    (1, 40, 32, 9, 256, 24, "none", "half", BF, False),
    (1, 333, 32, 8, 128, 64, "head", "half", BF, False),      # one block a token, 512 threads
    (1, 300, 20, 20, 128, 64, "head", "interleaved", BF, True),
    (1, 200, 48, 8, 128, 64, "token", "half", BF, True),      # a token's mean: no shares
    (1, 1, 64, 64, 128, 64, "head", "half", BF, True),
]


@pytest.mark.parametrize("case", WIDE)
def test_norm_rope_wide_tokens(case):
    test_norm_rope_forward_and_tangent(case)
    test_norm_rope_backward(case, "tensor")
    if case[6] != "none":
        test_norm_rope_backward(case, "ckpt8")


def test_norm_rope_fused_projection_slices():
    case = CASES[1]
    B, N, H, Hk, D, P, norm, layout, dtype, full = case
    x, tx, gains, cos, sin = make(case, 4)
    fused, tfused = torch.cat(x, -1).cuda(), torch.cat(tx, -1).cuda()
    rest = [dev(t) for t in (*gains, cos, sin)]
    a = caj.qk_norm_rope_fwd(*fused.split(H * D, -1), *rest, H, txq=tfused[..., :H * D],
                             txk=tfused[..., H * D:2 * H * D], txv=tfused[..., 2 * H * D:])
    b = caj.qk_norm_rope_fwd(*[dev(t) for t in x], *rest, H, txq=dev(tx[0]), txk=dev(tx[1]), txv=dev(tx[2]))
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    dy = [torch.randn_like(t) for t in b[:3]]
    c = caj.qk_norm_rope_bwd(*dy, fused[..., :H * D], fused[..., H * D:2 * H * D], *rest)
    e = caj.qk_norm_rope_bwd(*dy, dev(x[0]), dev(x[1]), *rest)
    for s, t in zip(c, e):
        assert torch.equal(s, t)


def test_norm_rope_agrees_with_the_prologue():
    """The full-width interleaved form against the library's primal-tangent prologue: the same
    formula, so at most an fp32 rounding apart before the one to bf16."""
    case = (2, 40, 4, 4, 128, 64, "token", "interleaved", BF, True)
    x, tx, gains, cos, sin = make(case, 8)
    a = caj.qk_norm_rope_jvp(*[dev(t) for t in (*x, *tx, *gains, cos, sin)], 4, eps=1e-6)
    b = caj.qk_norm_rope_fwd(*[dev(t) for t in (*x, *gains, cos, sin)], 4, eps=1e-6, norm="token",
                             txq=dev(tx[0]), txk=dev(tx[1]), txv=dev(tx[2]))
    for s, t in zip(a, b):
        assert float((s.float() - t.float()).abs().max()) <= 2.0 ** -7 * float(t.float().abs().max())


def test_zero_inputs_and_no_rows():
    case = CASES[1]
    B, N, H, Hk, D, P, norm, layout, dtype, full = case
    x, tx, gains, cos, sin = make(case, 4)
    rest = [dev(t) for t in (*gains, cos, sin)]
    z = torch.zeros(B, N, H * D, dtype=dtype, device="cuda")
    for t in caj.qk_norm_rope_fwd(z, z, z, *rest, H, txq=z, txk=z, txv=z):
        assert not t.any()
    e = z[:, :0]
    none = [*rest[:2], rest[2][:0], rest[3][:0]]
    for t in caj.qk_norm_rope_fwd(e, e, e, *none, H):
        assert t.shape == (B, H, 0, D)
    h = torch.zeros(B, H, 0, D, dtype=dtype, device="cuda")
    out = caj.qk_norm_rope_bwd(h, h, h, e, e, *none)
    assert out[0].shape == (B, 0, H * D) and not out[3].any() and out[3].shape == (D,)


def test_calls_on_another_stream_and_in_a_graph():
    case = CASES[1]
    B, N, H, Hk, D, P, norm, layout, dtype, full = case
    x, tx, gains, cos, sin = make(case, 6)
    xs, rest = [dev(t) for t in x], [dev(t) for t in (*gains, cos, sin)]
    freq, axis = caj.rope_frequencies(2 * P)
    pos = torch.arange(N, device="cuda")

    def step():
        c, s = caj.rope_table(pos, freq, axis)
        q, k, v = caj.qk_norm_rope_fwd(*xs, *rest[:2], c, s, H)
        kept = caj.ckpt8_pack(xs[0]), caj.ckpt8_pack(xs[1])
        return caj.qk_norm_rope_bwd(q, k, v, *kept, *rest[:2], c, s) + (caj.ckpt8_unpack(kept[0]),)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):  # each with its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
            pass
    for t in xs:
        t.mul_(-0.75)
    want = step()
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last tokens must equal a call on them alone."""
    H, D, N = 12, 128, 1_450_000
    x = torch.zeros(1, N, H * D, dtype=BF, device="cuda")
    tail = 300
    g = torch.Generator().manual_seed(1)
    x[:, -tail:] = torch.randn(1, tail, H * D, generator=g).to(BF).cuda()
    assert x.numel() > 2 ** 31
    gain = torch.ones(D, device="cuda")
    cos, sin = caj.rope_table(torch.arange(N, device="cuda"), caj.rope_frequencies(D)[0])
    q, k = caj.qk_norm_rope_fwd(x, x, None, gain, gain, cos, sin, H)
    small = caj.qk_norm_rope_fwd(*[x[:, -tail:].contiguous()] * 2, None, gain, gain, cos[-tail:].contiguous(),
                                 sin[-tail:].contiguous(), H)
    assert torch.equal(q[:, :, -tail:], small[0]) and torch.equal(k[:, :, -tail:], small[1])
    del k
    kept = caj.ckpt8_pack(x)
    assert torch.equal(caj.ckpt8_unpack(kept)[:, -tail:], caj.ckpt8_unpack(caj.ckpt8_pack(x[:, -tail:])))
    dxq, dxk, _, dgq, _ = caj.qk_norm_rope_bwd(q, q, None, kept, kept, gain, gain, cos, sin)
    few = caj.ckpt8_pack(x[:, -tail:].contiguous())
    want = caj.qk_norm_rope_bwd(*[q[:, :, -tail:].contiguous()] * 2, None, few, few, gain, gain,
                                cos[-tail:].contiguous(), sin[-tail:].contiguous())
    assert torch.equal(dxq[:, -tail:], want[0]) and torch.equal(dxk[:, -tail:], want[1])
    # zeros elsewhere: the same sums in another order, K roundings of at most the sum of magnitudes
    assert float((dgq - want[3]).abs().max()) <= 1e-4 * tail * H
