"""The differentiable functions and the recurrent block that runs them together, on the GPU."""
import numpy as np
import pytest
import torch

import block_reference as ref
from bidirectional_selective_scan_amd import autograd, recurrent_block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def leaf(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV).requires_grad_()


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("packed", [False, True])
def test_gated_recurrence_gradients(packed):
    rng = np.random.default_rng(1)
    d = 22
    if packed:
        lens = [30, 0, 64, 1, 55]
        off = np.concatenate([[0], np.cumsum(lens)]).tolist()
        shape, bounds = (1, off[-1], d), ref.bounds_of(0, 0, off)
        offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    else:
        shape, bounds, offsets = (3, 50, d), ref.bounds_of(3, 50), None
    x, r, i = (leaf(rng.standard_normal(shape)) for _ in range(3))
    lam, h0 = leaf(rng.standard_normal(d) - 3), leaf(rng.standard_normal((len(bounds), d)))
    dy, dh = rng.standard_normal(shape).astype(np.float32), rng.standard_normal((len(bounds), d)).astype(np.float32)
    y, h = autograd.gated_recurrence(x, r, i, lam, 8.0, h0, offsets=offsets, reverse=packed)
    ((y * torch.from_numpy(dy).to(DEV)).sum() + (h * torch.from_numpy(dh).to(DEV)).sum()).backward()
    rows = [f64(t).reshape(-1, d) for t in (x, r, i)]
    want = ref.gated(*rows, f64(lam), 8.0, bounds, f64(h0), packed, dy.astype(np.float64).reshape(-1, d),
                     dh.astype(np.float64), True)
    for name, t in (("dx", x), ("dr", r), ("di", i), ("dlam", lam), ("dh0", h0)):
        ref.check(t.grad, want[name], False, name)


def test_only_one_output_used():
    """No gradient of h_last (or of the sum): the missing one counts as zero."""
    rng = np.random.default_rng(2)
    x, r, i = (leaf(rng.standard_normal((2, 70, 12))) for _ in range(3))
    lam = leaf(rng.standard_normal(12) - 3)
    y, _ = autograd.gated_recurrence(x, r, i, lam)
    y.sum().backward()
    rows = [f64(t).reshape(-1, 12) for t in (x, r, i)]
    want = ref.gated(*rows, f64(lam), 8.0, ref.bounds_of(2, 70), None, False, np.ones((140, 12)), None, True)
    for name, t in (("dx", x), ("dr", r), ("di", i), ("dlam", lam)):
        ref.check(t.grad, want[name], False, name)
    x, w = leaf(rng.standard_normal((9, 40))), leaf(rng.standard_normal(40))
    _, n = autograd.block_norm(x, w_pre=w)
    n.sum().backward()
    want = ref.norm(f64(x), w_pre=f64(w), dn=np.ones((9, 40)), want_grads=True)
    ref.check(x.grad, want["dx"])
    ref.check(w.grad, want["dw_pre"])


def test_no_second_derivative():
    x = torch.randn(4, 16, device=DEV, requires_grad=True)
    w = torch.ones(16, device=DEV, requires_grad=True)
    _, n = autograd.block_norm(x, w_pre=w)
    g, = torch.autograd.grad(n.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("bidirectional", [False, True])
def test_block_against_plain_torch(bidirectional):
    """A block's output and parameter gradients against the same block in torch operations, fp32. The
    matrix products run in fp32 on both sides; 1e-4 of a tensor's largest value covers the longer of
    the two's summation orders (products of 48 to 192 terms, 1e-6 each, through two layers of them)."""
    torch.manual_seed(3)
    d, di = 48, 64
    b = recurrent_block.RecurrentBlock(d, di, bidirectional, dtype=torch.float32).to(DEV)
    n0 = torch.randn(2, 90, d, device=DEV, requires_grad=True)
    r0 = torch.randn(2, 90, d, device=DEV, requires_grad=True)

    def rms(v, w):
        return v * torch.rsqrt(v.pow(2).mean(-1, keepdim=True) + 1e-5) * w

    def plain(n, res):
        parts = (n @ b.w_in).split(di, -1)
        z, y = parts[-1], 0
        for k in range(b.directions):
            x, r, i = parts[3 * k:3 * k + 3]
            if k == 1:
                x, r, i = (t.flip(1) for t in (x, r, i))
            u = -b.c * torch.nn.functional.softplus(b.lam[k]) * torch.sigmoid(r)
            inp = torch.sqrt(-torch.expm1(2 * u)) * torch.sigmoid(i) * x
            h, hs = torch.zeros(2, di, device=DEV), []
            for t in range(90):
                h = torch.exp(u[:, t]) * h + inp[:, t]
                hs.append(h)
            hs = torch.stack(hs, 1)
            y = y + (hs.flip(1) if k == 1 else hs)
        g = rms(y * torch.nn.functional.silu(z), b.w_gated)
        res = res + b.gamma * rms(g @ b.w_out, b.w_post)
        return rms(res, b.w_next), res

    params = [n0, r0] + list(b.parameters())
    go = torch.randn(2, 90, d, device=DEV)
    got, want = [], []
    for f, out in ((b, got), (plain, want)):
        n, res = f(n0, r0)
        out += [n.detach(), res.detach()] + list(torch.autograd.grad((n * go).sum() + res.sum(), params))
    for a, w in zip(got, want):
        assert (a - w).abs().max() <= 1e-4 * w.abs().max()


def test_example_trains_and_decodes():
    """The example's loss falls by half, and decoding token by token gives the whole sequence's outputs
    to a bf16 network's rounding (values of order one, 2^-8 each, over a handful of layers)."""
    first, last, diff = recurrent_block.main(steps=60)
    assert last < 0.5 * first
    assert diff < 0.1
