"""The block operators through autograd, alone and as the transformer block they make up
around the attention: values, tangents and gradients against 64-bit plain torch."""
import math

import pytest
import torch

import block_reference as ref
import masked_attention_jvp_b200 as caj
from masked_attention_jvp_b200.workloads import MaskDesc

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rnd(g, *s, std=1.0):
    return (torch.randn(*s, generator=g) * std).to(BF).cuda()


@pytest.mark.parametrize("ckpt8", [False, True])
@pytest.mark.parametrize("norm,v", [("head", True), ("token", False), ("none", True)])
def test_qk_norm_rope_gradients_are_the_kernels(norm, v, ckpt8):
    g = torch.Generator().manual_seed(1)
    B, N, H, D, P = 2, 33, 4, 64, 32
    xs = [rnd(g, B, N, H * D) for _ in range(3 if v else 2)] + ([] if v else [None])
    gains = [None, None] if norm == "none" else [(1 + 0.1 * torch.randn(D if norm == "head" else H * D, generator=g)).cuda()
                                                 for _ in range(2)]
    th = torch.rand(N, P, generator=g).cuda()
    leaves = [None if t is None else t.clone().requires_grad_() for t in (*xs, *gains)]
    out = caj.qk_norm_rope(*leaves, th.cos(), th.sin(), H, norm=norm, ckpt8=ckpt8)
    want = caj.qk_norm_rope_fwd(*xs, *gains, th.cos(), th.sin(), H, norm=norm)
    dys = [torch.randn_like(t) for t in want]
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    torch.autograd.backward(out, dys)
    kept = [None, None] if norm == "none" else [caj.ckpt8_pack(t) for t in xs[:2]] if ckpt8 else xs[:2]
    grads = caj.qk_norm_rope_bwd(*dys, *([] if v else [None]), *kept, *gains, th.cos(), th.sin(), norm=norm)
    for leaf, gr in zip(leaves, grads):
        assert leaf is None and gr is None or torch.equal(leaf.grad, gr)


@pytest.mark.parametrize("ckpt8", [False, True])
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_linear_act_gradients_are_the_kernels(act, ckpt8):
    g = torch.Generator().manual_seed(2)
    x, w, b, r = rnd(g, 3, 50, 64), rnd(g, 96, 64, std=0.1), rnd(g, 96), rnd(g, 3, 50, 96)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
    y, ty = caj.linear_act(*leaves[:3], act, leaves[3], ckpt8=ckpt8)
    assert ty is None
    want, _, pre = caj.linear_act_fwd(x, w, b, act, r, save_pre=act != "none")
    assert torch.equal(y, want)
    dy = torch.randn_like(y)
    y.backward(dy)
    dx, dw, db = caj.linear_act_bwd(dy, caj.ckpt8_pack(x) if ckpt8 else x, w, act, pre)
    assert torch.equal(leaves[0].grad, dx) and torch.equal(leaves[1].grad, dw)
    assert torch.equal(leaves[2].grad, db.to(BF)) and torch.equal(leaves[3].grad, dy)
    # an upstream gradient that is one number everywhere has no strides of its own
    y, ty = caj.linear_act(leaves[0], w, None, act, tx=x, ckpt8=ckpt8)
    assert not ty.requires_grad
    leaves[0].grad = None
    y.sum().backward()
    ones = torch.ones_like(y)
    _, _, pre = caj.linear_act_fwd(x, w, None, act, save_pre=act != "none")
    assert torch.equal(leaves[0].grad, caj.linear_act_bwd(ones, None, w, act, pre, bias=False, need=(True, False))[0])


def test_attention_from_8_bits_is_the_backward_of_the_kept_values():
    g = torch.Generator().manual_seed(3)
    mask = MaskDesc(50, 1, 4, 1)
    q, k, v, tq, tk, tv = [rnd(g, 1, 2, mask.seq_len, 64) for _ in range(6)]
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o, to, lse, tlse = caj.attention_jvp(*leaves, tq, tk, tv, mask, ckpt8=True)
    want = caj.attn_fwd_jvp(q, k, v, tq, tk, tv, mask)
    for a, b in zip((o, to, lse, tlse), want):
        assert torch.equal(a, b)
    do = torch.randn_like(o)
    o.backward(do)
    kept = [caj.ckpt8_unpack(caj.ckpt8_pack(t)) for t in (q, k, v, want[0])]
    dq, dk, dv, _ = caj.attn_bwd(*kept, do, want[2], mask)
    for leaf, gr in zip(leaves, (dq, dk, dv)):
        assert torch.equal(leaf.grad, gr)


# ------------------------------------------------------------------- the whole block

W, H, D, HID = 256, 2, 128, 512  # width = H * D
MASK = MaskDesc(20, 1, 3, 1)


def params(g):
    shapes = {"wqkv": (3 * W, W), "bqkv": (3 * W,), "wo": (W, W), "bo": (W,), "w1": (HID, W), "b1": (HID,),
              "w2": (W, HID), "b2": (W,)}
    p = {n: rnd(g, *s, std=s[-1] ** -0.5 if len(s) == 2 else 0.1) for n, s in shapes.items()}
    p["gq"], p["gk"] = [(1 + 0.1 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    return p


def block(x, tx, p, cos, sin, ckpt8):
    """One block through the library, (y, ty)."""
    qkv, tqkv = caj.linear_act(x, p["wqkv"], p["bqkv"], tx=tx, ckpt8=ckpt8)
    parts, tparts = qkv.split(W, -1), tqkv.split(W, -1)
    q, k, v, tq, tk, tv = caj.qk_norm_rope(*parts, p["gq"], p["gk"], cos, sin, H, layout="half", txq=tparts[0],
                                           txk=tparts[1], txv=tparts[2], ckpt8=ckpt8)
    o, to, _, _ = caj.attention_jvp(q, k, v, tq, tk, tv, MASK, ckpt8=ckpt8)
    o, to = [t.transpose(1, 2).reshape(x.shape) for t in (o, to)]
    h, th = caj.linear_act(o, p["wo"], p["bo"], residual=x, tx=to, tresidual=tx, ckpt8=ckpt8)
    f, tf = caj.linear_act(h, p["w1"], p["b1"], act="gelu_tanh", tx=th, ckpt8=ckpt8)
    return caj.linear_act(f, p["w2"], p["b2"], residual=h, tx=tf, tresidual=th, ckpt8=ckpt8)


def plain(x, p, cos, sin):
    """The same in plain torch, 64 bits."""
    B, N, _ = x.shape
    q, k, v = (x @ p["wqkv"].t() + p["bqkv"]).view(B, N, 3, H, D).unbind(2)
    out = []
    for t, g in ((q, p["gq"]), (k, p["gk"])):
        t = g * t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)
        a, b = t[..., :D // 2], t[..., D // 2:]
        c, s = cos[None, :, None], sin[None, :, None]
        out.append(torch.cat([a * c - b * s, a * s + b * c], -1).transpose(1, 2))
    L, T = MASK.n_frames * MASK.tokens_per_frame, MASK.tokens_per_frame
    i = torch.arange(N)
    noisy, frame = i >= L, i % L // T
    see = torch.where(noisy[None, :], noisy[:, None] & (frame[:, None] == frame[None, :]),
                      torch.where(noisy[:, None], frame[None, :] < frame[:, None], frame[None, :] <= frame[:, None]))
    s = (out[0] @ out[1].transpose(-1, -2) / math.sqrt(D)).masked_fill(~see, -math.inf)
    o = (torch.softmax(s, -1) @ v.transpose(1, 2)).transpose(1, 2).reshape(B, N, W)
    h = x + o @ p["wo"].t() + p["bo"]
    f = ref.act(h @ p["w1"].t() + p["b1"], "gelu_tanh")[0]
    return h + f @ p["w2"].t() + p["b2"]


@pytest.mark.parametrize("ckpt8", [False, True])
def test_block_values_tangents_and_gradients(ckpt8):
    """Against 64 bits, relative in the 2-norm over each tensor. Forward: nine tensors are
    rounded to bf16 between x and y (qkv, q, k, P inside the attention, o, h, f, y, and the
    attention's own operands), each by at most 2^-8 relative to its size, and the block maps
    relative errors of that order to themselves (norms and residuals): 9 * 2^-8 = 3.5e-2 is
    allowed. The gradient passes the same tensors back and rounds each of theirs once more:
    twice that. From 8 bits, a kept tensor is off by at most half a step, 2^-8 of the power of
    two above its block's largest magnitude, itself at most about 4 times the block's size:
    4 * 2^-7 each for the eight that are kept, of independent signs, so sqrt(8) times that
    on top."""
    g = torch.Generator().manual_seed(5)
    N = MASK.seq_len
    x, tx = rnd(g, 2, N, W), rnd(g, 2, N, W, std=0.5)
    p = params(g)
    freq, axis = caj.rope_frequencies((64, 32, 32))
    i = torch.arange(N) % (N // 2)
    pos = torch.stack([i // 20, i % 20 // 5, i % 5], 1).cuda()
    cos, sin = caj.rope_table(pos, freq, axis)
    leaves = {n: t.clone().requires_grad_() for n, t in p.items()}
    xl = x.clone().requires_grad_()
    y, ty = block(xl, tx, leaves, cos, sin, ckpt8)
    dy = rnd(g, *y.shape)
    y.backward(dy)
    torch.cuda.synchronize()
    caj.device_status()

    pd = {n: ref.d(t).requires_grad_() for n, t in p.items()}
    xd = ref.d(x).requires_grad_()
    f = lambda x_: plain(x_, pd, ref.d(cos), ref.d(sin))  # noqa: E731
    want, twant = torch.func.jvp(lambda x_: plain(x_, {n: t.detach() for n, t in pd.items()}, ref.d(cos), ref.d(sin)),
                                 (ref.d(x),), (ref.d(tx),))
    f(xd).backward(ref.d(dy))
    rel = lambda a, b: float((ref.d(a) - b).norm() / b.norm())  # noqa: E731
    fwd = 9 * 2.0 ** -8
    bwd = 2 * fwd + (math.sqrt(8) * 4 * 2.0 ** -7 if ckpt8 else 0.0)
    assert rel(y, want) <= fwd and rel(ty, twant) <= fwd
    assert rel(xl.grad, xd.grad) <= bwd
    for n in p:
        assert rel(leaves[n].grad, pd[n].grad) <= bwd, n


def test_block_from_8_bits_keeps_half_the_memory():
    g = torch.Generator().manual_seed(6)
    x = rnd(g, 4096, 512)
    w = rnd(g, 512, 512).requires_grad_()
    held = []
    for ckpt8 in (False, True):
        xl = x.clone().requires_grad_()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        h = xl * 1  # an activation that only the graph keeps
        y, _ = caj.linear_act(h, w, ckpt8=ckpt8)
        del h
        held.append(torch.cuda.memory_allocated() - before - y.numel() * 2)
        y.backward(torch.ones_like(y))
    # bf16: 4 MiB; 8 bits: one byte a value and four bytes each 128
    assert held[0] >= 2 * x.numel() and held[1] <= x.numel() * 1.04 + 4096


def test_backward_replays_in_a_graph():
    """Forward and backward of a layer captured together and replayed on new inputs, while
    another graph and eager results of other leaves are alive."""
    g = torch.Generator().manual_seed(7)
    w, b = rnd(g, 128, 256, std=0.06), rnd(g, 128)
    static_x, static_dy = rnd(g, 200, 256), rnd(g, 200, 128)

    def grads(x, dy):
        y, _, pre = caj.linear_act_fwd(x, w, b, "silu", save_pre=True)
        return (y,) + caj.linear_act_bwd(dy, caj.ckpt8_pack(x), w, "silu", pre)

    grads(static_x, static_dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = grads(static_x, static_dy)
    for seed in (8, 9):
        h = torch.Generator().manual_seed(seed)
        x, dy = rnd(h, 200, 256), rnd(h, 200, 128)
        static_x.copy_(x)
        static_dy.copy_(dy)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, grads(x, dy)):
            assert torch.equal(a, c)


def test_autograd_replays_in_a_graph():
    """Forward and gradients through autograd captured while an eager graph of the same tensors
    is alive, on leaves taken anew inside the capture, and replayed on new inputs."""
    g = torch.Generator().manual_seed(10)
    tensors = [rnd(g, 200, 256), rnd(g, 128, 256, std=0.06), rnd(g, 128)]
    eager = [t.requires_grad_() for t in tensors]
    dy = rnd(g, 200, 128)

    def grads():
        leaves = [t.detach().requires_grad_() for t in tensors]
        y, _ = caj.linear_act(*leaves, "gelu_tanh", ckpt8=True)
        return (y.detach(),) + torch.autograd.grad(y, leaves, dy)

    alive, _ = caj.linear_act(*eager, "silu")
    grads()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = grads()
    alive.backward(dy)  # the eager graph is none the worse
    with torch.no_grad():
        tensors[0].mul_(-0.5)
        dy.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(out, grads()):
        assert torch.equal(a, c)
    assert all(t.grad is not None for t in eager)
