"""The layer norm on the GPU (forward and backward) against its 64-bit form, element by element within the error
that 32-bit arithmetic may leave: ULP = 2^-23 relative for an operation, a row's sums added in a tree with at most 64
additions in a row per lane, errors carried to first order; outputs in bf16 add their rounding, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from block_reference import TINY, ULP, check
from bidirectional_selective_scan_amd import autograd, binding
from bidirectional_selective_scan_amd.binding import PreparedLayerNorm, PreparedLayerNormGrad

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
DEPTH = 64 + 16


def tensor(a, dtype=torch.float32):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def reference(x, residual, weight, bias, dsum, dn, eps=EPS):
    """All float64; a dict of name -> (value, bound)."""
    def mean(v):
        return v.mean(1, keepdims=True)

    rows = x.shape[0]
    w = np.ones(x.shape[1]) if weight is None else weight
    s = x if residual is None else x + residual
    se = ULP * np.abs(s)
    mu = mean(s)
    ce = se + mean(se) + ULP * (DEPTH * mean(np.abs(s)) + np.abs(mu))
    c = s - mu
    ce = ce + ULP * np.abs(c)
    ss = mean(c * c) + eps
    sse = mean(2 * np.abs(c) * ce + ce * ce) + ULP * (DEPTH + 4) * ss
    rho = 1 / np.sqrt(ss)
    rhoe = 0.5 * rho / ss * sse + 2 * ULP * rho
    xh = c * rho
    xhe = ce * rho + np.abs(c) * rhoe + ULP * np.abs(xh)
    b = 0.0 if bias is None else bias
    n = xh * w + b
    out = {"n": (n, np.abs(w) * xhe + 2 * ULP * (np.abs(xh * w) + np.abs(b)) + TINY)}
    if residual is not None:
        out["sum"] = (s, se + TINY)
    d = np.zeros_like(x) if dn is None else dn
    g = d * w
    mg, mge = mean(g), ULP * (DEPTH + 2) * mean(np.abs(g))
    mx = mean(g * xh)
    mxe = mean(np.abs(g) * xhe) + ULP * (DEPTH + 2) * mean(np.abs(g * xh))
    inner = g - mg - xh * mx
    innere = mge + xhe * np.abs(mx) + np.abs(xh) * mxe + 4 * ULP * (np.abs(g) + np.abs(mg) + np.abs(xh * mx))
    add = 0.0 if dsum is None else dsum
    ds = add + rho * inner
    dse = rhoe * np.abs(inner) + rho * innere + 2 * ULP * (np.abs(rho * inner) + np.abs(ds))
    out["dx"] = (ds, dse + TINY)
    if residual is not None:
        out["dresidual"] = (ds, dse + TINY)
    if weight is not None:
        out["dweight"] = ((d * xh).sum(0), (np.abs(d) * xhe).sum(0) + ULP * (64 + rows) * np.abs(d * xh).sum(0) + TINY)
    if bias is not None:
        out["dbias"] = (d.sum(0), ULP * (64 + rows) * np.abs(d).sum(0) + TINY)
    return out


class Problem:
    def __init__(self, rows, d, io="f32", res="f32", affine=True, seed=0, mean=0.3, std=1.0, strided=False, given=(True, True)):
        rng = np.random.default_rng(seed)
        dt = torch.bfloat16 if io == "bf16" else torch.float32
        rdt = {"f32": torch.float32, "io": dt, None: None}[res]

        def rnd(*shape, std=1.0, mean=0.0, dtype=dt):
            return tensor(rng.standard_normal(shape) * std + mean, dtype)

        self.x = rnd(rows, d + 3, std=std, mean=mean)[:, 1:d + 1] if strided else rnd(rows, d, std=std, mean=mean)
        self.residual = rnd(rows, d, std=2.0, dtype=rdt) if rdt else None
        self.weight = rnd(d, std=0.2, mean=1.0, dtype=torch.float32) if affine else None
        self.bias = rnd(d, dtype=torch.float32) if affine else None
        self.dsum = rnd(rows, d, dtype=rdt) if rdt and given[0] else None
        self.dn = rnd(rows, d) if given[1] else None
        self.bf, self.rbf = io == "bf16", (rdt or dt) == torch.bfloat16

    def args(self):
        return self.x, self.residual, self.weight, self.bias

    def check(self, what=""):
        want = reference(*(f64(t) for t in self.args()), f64(self.dsum), f64(self.dn))
        fwd = PreparedLayerNorm(*self.args(), eps=EPS)
        fwd()
        bwd = PreparedLayerNormGrad(*self.args(), self.dsum, self.dn, EPS)
        bwd()
        torch.cuda.synchronize()
        got = dict(sum=fwd.sum, n=fwd.n, dx=bwd.dx, dresidual=bwd.dresidual, dweight=bwd.dweight, dbias=bwd.dbias)
        assert {k for k, v in got.items() if v is not None} == set(want)
        for k in want:
            check(got[k], want[k], self.rbf if k in ("sum", "dresidual") else self.bf and k in ("n", "dx"), f"{what} {k}")
        return fwd, bwd


@pytest.mark.parametrize("io,res", [("f32", "f32"), ("f32", None), ("bf16", "f32"), ("bf16", "io"), ("bf16", None)])
@pytest.mark.parametrize("affine", [True, False])
def test_kinds(io, res, affine):
    for rows, d in ((1, 64), (7, 768), (33, 100), (5, 1531)):
        Problem(rows, d, io, res, affine, seed=rows).check(f"{rows} x {d}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1, 2, 3, 5, 63, 64, 65, 127, 129, 255, 256, 257, 511, 513, 767, 769, 1023, 1024, 1025, 2047, 2049,
                               4095, 4096, 4097, 4100, 8191, 8192, 8193, 16383, 16385, 32767, 32768])
def test_widths(io, d):
    Problem(3, d, io, "f32", seed=d).check(f"width {d}")


@pytest.mark.parametrize("d", [64, 100, 768, 4096])
def test_many_rows(d):
    Problem(4099, d, "bf16", "f32", seed=d).check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_rows_and_large_means(io):
    Problem(20, 97, io, "f32", seed=1, strided=True).check("strided")
    Problem(20, 96, io, None, seed=2, strided=True).check("strided")
    Problem(20, 768, io, None, seed=3, mean=1000.0).check("large mean")
    Problem(20, 768, io, None, seed=4, mean=0.0, std=1e-4).check("below eps")
    Problem(4, 768, io, None, seed=5, mean=2.0, std=0.0).check("constant rows")


@pytest.mark.parametrize("given", [(False, True), (True, False), (False, False)])
def test_absent_gradients(given):
    Problem(40, 200, "bf16", "f32", seed=6, given=given).check()


def test_nan_stays_in_its_row():
    p = Problem(40, 100, "f32", "f32", seed=7)
    f0, b0 = p.check()
    n0, dx0 = f0.n.clone(), b0.dx.clone()
    p.x[11, 5], p.x[20, 99] = float("nan"), float("inf")
    f, b = PreparedLayerNorm(*p.args(), eps=EPS), PreparedLayerNormGrad(*p.args(), p.dsum, p.dn, EPS)
    f()
    b()
    rest = [r for r in range(40) if r not in (11, 20)]
    assert torch.equal(f.n[rest], n0[rest]) and torch.equal(b.dx[rest], dx0[rest])
    assert torch.isnan(f.n[[11, 20]]).all() and torch.isnan(b.dx[[11, 20]]).all() and torch.isnan(b.dweight).all()


def test_in_place_sum_and_gradient_of_it():
    p = Problem(30, 256, "bf16", "f32", seed=8)
    want = p.check()[0]
    keep = want.sum.clone()
    call = PreparedLayerNorm(*p.args(), eps=EPS, out_sum=p.residual)
    call()
    assert torch.equal(p.residual, keep) and torch.equal(call.n, want.n)


def test_rows_outside_are_left_as_they_were():
    p = Problem(9, 77, "bf16", "f32", seed=9)
    room = torch.full((9 * 77 + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
    call = PreparedLayerNorm(*p.args(), eps=EPS, out_n=room[32:32 + 9 * 77].view(9, 77))
    call()
    assert (room[:32] == 3).all() and (room[32 + 9 * 77:] == 3).all()
    want = reference(*(f64(t) for t in p.args()), None, None)
    check(call.n, want["n"], True)


def test_same_bits_and_graph():
    p = Problem(5000, 200, "bf16", "f32", seed=10)
    f, b = p.check()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        f2, b2 = PreparedLayerNorm(*p.args(), eps=EPS), PreparedLayerNormGrad(*p.args(), p.dsum, p.dn, EPS)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            f2()
            b2()
    for _ in range(3):
        p.x.copy_(torch.randn_like(p.x))
        f()
        b()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in ((f.n, f2.n), (f.sum, f2.sum), (b.dx, b2.dx), (b.dresidual, b2.dresidual), (b.dweight, b2.dweight),
                     (b.dbias, b2.dbias)):
            assert torch.equal(u, v)


def test_empty():
    x = torch.empty(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    s, n = binding.layer_norm(x, None, w, w)
    assert s is None and n.shape == (0, 64)
    g = PreparedLayerNormGrad(x, None, w, w, dn=x)
    g.dweight.fill_(3.0)
    g()
    assert (g.dweight == 0).all() and (g.dbias == 0).all()


def test_autograd():
    p = Problem(50, 96, "f32", "f32", seed=11)
    leaves = [t.clone().requires_grad_() for t in p.args()]
    s, n = autograd.layer_norm(*leaves)
    ((n * p.dn).sum() + (s * p.dsum).sum()).backward()
    want = reference(*(f64(t) for t in p.args()), f64(p.dsum), f64(p.dn))
    for t, k in zip(leaves, ("dx", "dresidual", "dweight", "dbias")):
        check(t.grad, want[k], False, k)
    # without a residual: the norm alone
    x = p.x.clone().requires_grad_()
    _, n = autograd.layer_norm(x)
    n.backward(p.dn)
    check(x.grad, reference(f64(p.x), None, None, None, None, f64(p.dn))["dx"])
    with pytest.raises(RuntimeError):
        _, n = autograd.layer_norm(x)
        g, = torch.autograd.grad(n.sum(), x, create_graph=True)
        g.sum().backward()


def test_against_differences():
    """fp32 gradients against central differences. The norm's third derivative along a direction of unit size per element
    is below 60 |g| for a row of unit variance; eps = 2^-6, and the loss's rounding over it."""
    p = Problem(6, 48, "f32", "f32", seed=12)
    grad = PreparedLayerNormGrad(*p.args(), p.dsum, p.dn, EPS)
    grad()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)

    def loss():
        s, n = binding.layer_norm(*p.args(), eps=EPS)
        return ((n.double() * p.dn.double()).sum() + (s.double() * p.dsum.double()).sum()).item()

    s, n = binding.layer_norm(*p.args(), eps=EPS)
    size = (n.double() * p.dn.double()).abs().sum().item() + (s.double() * p.dsum.double()).abs().sum().item()
    eps = 2.0 ** -6
    for t, g in ((p.x, grad.dx), (p.residual, grad.dresidual), (p.weight, grad.dweight), (p.bias, grad.dbias)):
        d = torch.randn(t.shape, generator=gen, device=DEV)
        keep = t.clone()
        t.copy_(keep + eps * d)
        up = loss()
        t.copy_(keep - eps * d)
        down = loss()
        t.copy_(keep)
        assert abs((up - down) / (2 * eps) - (g.double() * d.double()).sum().item()) <= size * (2.0 ** -22 / eps + 10 * eps ** 2)


def test_refusals():
    x = torch.randn(4, 32, device=DEV)
    w = torch.ones(32, device=DEV)
    for bad in (dict(weight=w[:16]), dict(weight=w.double()), dict(bias=w.cpu()), dict(residual=x[:2]), dict(residual=x.half()),
                dict(with_sum=False, out_sum=x), dict(out_n=x[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            PreparedLayerNorm(x, **bad)
    with pytest.raises(ValueError):
        PreparedLayerNorm(x[:, ::2])
    with pytest.raises(TypeError):
        PreparedLayerNorm(x.half())
    with pytest.raises(ValueError):
        PreparedLayerNorm(x.cpu())
    for bad, status in ((dict(eps=0.0), -13), (dict(out_n=x), -6)):
        with pytest.raises(binding.VimscanError) as e:
            PreparedLayerNorm(x, **bad)()
        assert e.value.status == status
    with pytest.raises(binding.VimscanError) as e:
        PreparedLayerNorm(torch.zeros(1, 32769, device=DEV))()
    assert e.value.status == -2
    with pytest.raises(ValueError):
        PreparedLayerNormGrad(x, dn=x[:2])
