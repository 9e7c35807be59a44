"""Linear attention and the layer norm run together: the differentiable functions, the block that is made of them, and the
example's stack of such blocks."""
import math

import numpy as np
import pytest
import torch

import block_reference
import linattn_reference as ref
from bidirectional_selective_scan_amd import autograd, recurrent_block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("packed", [False, True])
def test_linear_attention_gradients(packed):
    rng = np.random.default_rng(1)
    H, G, dk, dv = 4, 2, 12, 20
    if packed:
        lens = [30, 0, 64, 1, 55]
        off = np.concatenate([[0], np.cumsum(lens)]).tolist()
        shape, bounds, offsets = (1, off[-1]), list(zip(off[:-1], off[1:])), torch.tensor(off, dtype=torch.int32, device=DEV)
    else:
        shape, bounds, offsets = (3, 50), [(0, 50), (50, 100), (100, 150)], None

    def leaf(*s):
        return torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV).requires_grad_()

    q, k, v, h0 = leaf(*shape, G, dk), leaf(*shape, G, dk), leaf(*shape, H, dv), leaf(len(bounds), H, dk, dv)
    g = (-torch.rand(*shape, H, device=DEV)).requires_grad_()
    dy, dh = torch.randn(*shape, H, dv, device=DEV), torch.randn(len(bounds), H, dk, dv, device=DEV)
    y, h = autograd.linear_attention(q, k, v, g, 0.5, h0, offsets=offsets, reverse=packed)
    ((y * dy).sum() + (h * dh).sum()).backward()
    n = shape[0] * shape[1]
    rows = [f64(t).reshape(n, *t.shape[2:]) for t in (q, k, v, g, dy)]
    want = ref.linattn(*rows[:4], 0.5, bounds, f64(h0), packed, rows[4], f64(dh))
    for name, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dh0", h0)):
        block_reference.check(t.grad, want[name], False, name)


def test_broadcast_inputs_get_their_sums():
    """q and k expanded over the heads, a decay expanded over the tokens: their gradients are the sums over the copies. Both sides run the same
    kernels in fp32; the copies are added in another order, 8 or 60 additions of half an ulp each."""
    torch.manual_seed(0)
    one = torch.randn(2, 30, 1, 16, device=DEV, requires_grad=True)
    v, dy = torch.randn(2, 30, 8, 16, device=DEV), torch.randn(2, 30, 8, 16, device=DEV)
    g1 = (-torch.rand(8, device=DEV)).requires_grad_()
    y, _ = autograd.linear_attention(one.expand(2, 30, 8, 16), one.expand(2, 30, 8, 16), v, g1)
    wide = torch.autograd.grad(y, (one, g1), dy)
    y, _ = autograd.linear_attention(one, one, v, g1.expand(2, 30, 8).contiguous())
    shared = torch.autograd.grad(y, (one, g1), dy)
    for a, b in zip(wide, shared):
        assert (a - b).abs().max() <= 64 * 2.0 ** -24 * 16 * b.abs().max()


def test_only_one_output_used():
    q, k, v = (torch.randn(2, 40, 2, 16, device=DEV, requires_grad=True) for _ in range(3))
    g = (-torch.rand(2, device=DEV)).requires_grad_()
    _, h = autograd.linear_attention(q, k, v, g)
    h.sum().backward()
    rows = [f64(t).reshape(80, 2, 16) for t in (q, k, v)]
    want = ref.linattn(*rows, f64(g), 0.25, [(0, 40), (40, 80)], None, False, None, np.ones((2, 2, 16, 16)))
    for name, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g)):
        block_reference.check(t.grad, want[name], False, name)
    with pytest.raises(RuntimeError):
        y, _ = autograd.linear_attention(q, k, v, g)
        d, = torch.autograd.grad(y.sum(), q, create_graph=True)
        d.sum().backward()


def test_block_against_plain_torch():
    """A block's output and parameter gradients against the same block in torch operations, fp32: 1e-4 of a tensor's largest value
    covers the two's summation orders (products of 48 to 96 terms and sums over 90 tokens, 1e-6 each, through a few layers)."""
    torch.manual_seed(3)
    b = recurrent_block.LinearAttentionBlock(48, 64, 16, groups=2, dtype=torch.float32).to(DEV)
    n0 = torch.randn(2, 90, 48, device=DEV, requires_grad=True)
    r0 = torch.randn(2, 90, 48, device=DEV, requires_grad=True)

    def plain(n, res):
        q, k, v, z, decay = (n @ b.w_in).split(b.widths, -1)
        q, k, v = (t.unflatten(-1, (-1, 16)) for t in (q, k, v))
        q, k = (t.repeat_interleave(2, 2) for t in (q, k))
        a = torch.exp(-torch.exp(b.rate) * torch.nn.functional.softplus(decay))
        S, ys = torch.zeros(2, 4, 16, 16, device=DEV), []
        for t in range(90):
            S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
            ys.append((q[:, t, :, :, None] * S).sum(-2) * 0.25)
        y = torch.stack(ys, 1)

        def norm(v):
            c = v - v.mean(-1, keepdim=True)
            return c * torch.rsqrt(c.pow(2).mean(-1, keepdim=True) + 1e-5)

        res = res + (norm(y).flatten(-2) * torch.nn.functional.silu(z)) @ b.w_out
        return norm(res) * b.w_next + b.b_next, res

    params = [n0, r0] + list(b.parameters())
    go = torch.randn(2, 90, 48, device=DEV)
    got, want = [], []
    for f, out in ((b, got), (plain, want)):
        n, res = f(n0, r0)
        out += [n.detach(), res.detach()] + list(torch.autograd.grad((n * go).sum() + res.sum(), params))
    for a, w in zip(got, want):
        assert (a - w).abs().max() <= 1e-4 * w.abs().max()


def test_example_runs():
    """The example trains and decodes; what it decodes token by token is what the whole sequence gives, to a bf16 network's
    rounding (values of order one, 2^-8 each, over a handful of layers)."""
    first, last, diff = recurrent_block.main(steps=5, mixer="attention")
    assert math.isfinite(first) and math.isfinite(last)
    assert diff < 0.1
    with pytest.raises(ValueError):
        recurrent_block.RecurrentStack(8, 16, 32, 8, 1, bidirectional=True, mixer="attention")
