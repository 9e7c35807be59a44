"""The block norm on the GPU (forward and backward) against its 64-bit form, element by element
within the error that 32-bit arithmetic may leave (block_reference)."""
import itertools

import numpy as np
import pytest
import torch

import block_reference as ref
from bidirectional_selective_scan_amd import binding
from bidirectional_selective_scan_amd.binding import PreparedBlockNorm, PreparedBlockNormGrad

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
WEIGHTS = ("w_post", "gamma", "w_pre")


def tensor(a, dtype=torch.float32):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV).to(dtype)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Problem:
    def __init__(self, rows, d, io="f32", res="f32", z=True, after=False, post=True, gamma=True, pre=True, seed=0,
                 fused=False):
        rng = np.random.default_rng(seed)
        dt = torch.bfloat16 if io == "bf16" else torch.float32
        rdt = {"f32": torch.float32, "io": dt, None: None}[res]

        def rnd(*shape, std=1.0, mean=0.0, dtype=dt):
            return tensor(rng.standard_normal(shape) * std + mean, dtype)

        if fused:
            buf = rnd(rows, 2 * d + 3)
            self.x, zz = buf[:, 1:d + 1], buf[:, d + 3:]
        else:
            self.x, zz = rnd(rows, d), rnd(rows, d)
        self.z = zz if z else None
        self.w_post = rnd(d, std=0.2, mean=1.0, dtype=torch.float32) if post else None
        self.residual = rnd(rows, d, std=2.0, dtype=rdt) if rdt else None
        self.gamma = rnd(d, std=0.2, mean=0.4, dtype=torch.float32) if gamma else None
        self.w_pre = rnd(d, std=0.2, mean=1.0, dtype=torch.float32) if pre else None
        self.dsum = rnd(rows, d, dtype=rdt or dt)
        self.dn = rnd(rows, d) if pre else None
        self.after, self.io, self.rbf = after, io == "bf16", (rdt or dt) == torch.bfloat16

    def args(self):
        return self.x, self.z, self.w_post, self.residual, self.gamma, self.w_pre

    def reference(self, grads=True):
        return ref.norm(*(f64(t) for t in self.args()), EPS, self.after, f64(self.dsum), f64(self.dn), grads)

    def run(self, **kw):
        fwd = PreparedBlockNorm(*self.args(), EPS, self.after)
        fwd()
        bwd = PreparedBlockNormGrad(*self.args(), self.dsum, self.dn, EPS, self.after, **kw)
        bwd()
        torch.cuda.synchronize()
        return fwd, bwd

    def check(self, what=""):
        want = self.reference()
        fwd, bwd = self.run()
        got = dict(sum=fwd.sum, n=fwd.n, dx=bwd.dx, dz=bwd.dz, dresidual=bwd.dresidual, dw_post=bwd.dw_post,
                   dgamma=bwd.dgamma, dw_pre=bwd.dw_pre)
        assert {k for k, v in got.items() if v is not None} == set(want)
        for k in want:
            bf = self.rbf if k in ("sum", "dresidual") else self.io and not k.startswith(("dw", "dg"))
            ref.check(got[k], want[k], bf, f"{what} {k}")
        return fwd, bwd


@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "f32"), ("bf16", "io")])
def test_every_combination_of_stages(io, res):
    for k, (z, post, has_res, gamma, pre) in enumerate(itertools.product((True, False), repeat=5)):
        for after in (False, True) if z and post else (False,):
            Problem(5, 72, io, res if has_res else None, z, after, post, gamma, pre, seed=k).check(
                f"z={z} post={post} res={has_res} gamma={gamma} pre={pre} after={after}")


@pytest.mark.parametrize("d", [1, 2, 3, 4, 7, 8, 63, 64, 65, 100, 191, 192, 255, 256, 257, 384, 511, 512, 516, 768,
                               1000, 1023, 1024, 1025, 1028, 1531, 1536, 2047, 2048, 2052])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_widths(d, io):
    Problem(9, d, io, seed=d, after=d % 2 == 1).check(f"D={d}")


@pytest.mark.parametrize("d", [4095, 4096, 4100, 8191, 8192, 8196, 16383, 16384, 16388, 32767, 32768])
def test_wide_rows(d):
    Problem(3, d, "bf16", seed=d).check(f"D={d}")
    Problem(2, d, "f32", seed=d, after=True).check(f"D={d}")


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 64, 255, 256, 257, 511, 513, 1024, 2051])
@pytest.mark.parametrize("d", [96, 50])
def test_rows(rows, d):
    Problem(rows, d, "bf16", seed=rows).check(f"rows={rows}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 61])
def test_strided_inputs(io, d):
    Problem(17, d, io, seed=3, fused=True).check()


def test_leading_dimensions_and_in_place_sum():
    p = Problem(24, 80, "bf16", "f32", seed=4)
    want = p.reference(False)
    res = p.residual.view(4, 6, 80).clone()
    s, n = PreparedBlockNorm(p.x.view(4, 6, 80), p.z.view(4, 6, 80), p.w_post, res, p.gamma, p.w_pre, EPS, out_sum=res)()
    assert s.data_ptr() == res.data_ptr() and n.shape == (4, 6, 80)
    ref.check(s, want["sum"])
    ref.check(n, want["n"], True)


def test_norm_alone_without_the_sum():
    p = Problem(7, 200, "f32", None, False, False, False, False, True, seed=5)
    s, n = binding.block_norm(p.x, w_pre=p.w_pre, eps=EPS, with_sum=False)
    assert s is None
    ref.check(n, p.reference(False)["n"])


def test_zero_rows_of_zeros_and_large_values():
    """A row of zeros gives zeros and finite gradients; values of 1e15 (squares of 1e30) stay exact to
    the bound."""
    p = Problem(6, 128, "f32", seed=6, gamma=False)
    p.x[2] = 0
    p.residual[2] = 0
    p.x[4] *= 1e15
    p.check()


def test_a_row_with_nan_leaves_the_others():
    p = Problem(9, 300, "bf16", seed=7)
    f0, b0 = p.run()
    p.x[3, 17] = float("nan")
    p.residual[5, 2] = float("inf")
    f1, b1 = p.run()
    keep = [0, 1, 2, 4, 6, 7, 8]
    for a, b in ((f0.sum, f1.sum), (f0.n, f1.n), (b0.dx, b1.dx), (b0.dz, b1.dz), (b0.dresidual, b1.dresidual)):
        assert torch.equal(a[keep], b[keep])
    assert bool(f1.n[3].isnan().all())


def test_missing_gradients_are_zero():
    for which in ("dsum", "dn"):
        p = Problem(8, 90, "f32", seed=8)
        setattr(p, which, None)
        want = p.reference()
        bwd = PreparedBlockNormGrad(*p.args(), p.dsum, p.dn, EPS)
        bwd()
        for k in ("dx", "dz", "dresidual", "dw_post", "dgamma", "dw_pre"):
            ref.check(getattr(bwd, k), want[k], False, f"no {which}: {k}")
    bwd = PreparedBlockNormGrad(*p.args(), p.dsum, p.dn, EPS, weights=False)
    bwd()
    assert bwd.dw_post is None
    ref.check(bwd.dx, want["dx"])


@pytest.mark.parametrize("after", [False, True])
def test_gradient_against_differences(after):
    """Directional derivatives of the 64-bit loss sum(s ds) + sum(n dn) by central differences; with
    step 1e-5 their own error stays under 1e-8 of the loss's terms."""
    p = Problem(6, 33, "f32", seed=9, after=after)
    _, bwd = p.run()
    want = p.reference()
    names = ("x", "z", "w_post", "residual", "gamma", "w_pre")
    base = [f64(t) for t in p.args()]
    ds, dn = f64(p.dsum), f64(p.dn)

    def loss(v):
        o = ref.norm(*v, EPS, after)
        return (o["sum"][0] * ds).sum() + (o["n"][0] * dn).sum()

    rng = np.random.default_rng(10)
    for k, name in enumerate(names):
        v = rng.standard_normal(base[k].shape)
        up, dn_ = list(base), list(base)
        up[k], dn_[k] = base[k] + 1e-5 * v, base[k] - 1e-5 * v
        slope = (loss(up) - loss(dn_)) / 2e-5
        mine = (f64(getattr(bwd, "d" + name)) * v).sum()
        tol = (want["d" + name][1] * np.abs(v)).sum() + 1e-8 * (np.abs(ds).sum() + np.abs(dn).sum())
        assert abs(mine - slope) <= tol, (name, mine, slope, tol)


def test_same_bits_every_run_and_in_a_graph():
    p = Problem(1500, 260, "bf16", seed=11)
    f0, b0 = p.run()

    def outs(f, b):
        return f.sum, f.n, b.dx, b.dz, b.dresidual, b.dw_post, b.dgamma, b.dw_pre

    keep = [t.clone() for t in outs(f0, b0)]
    for _ in range(3):
        for a, b in zip(keep, outs(*p.run())):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream().cuda_stream
        f = PreparedBlockNorm(*p.args(), EPS, stream=s)
        f()
        b = PreparedBlockNormGrad(*p.args(), p.dsum, p.dn, EPS, stream=s)
        b()
    for _ in range(3):
        for t in outs(f, b):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(keep, outs(f, b)):
            assert torch.equal(a, c)
        f0()
        b0()


def test_rows_past_32_bit_offsets():
    """2.2e9 channels of bf16: the last rows against 64 bits."""
    rows, d = 540000, 4096
    assert rows * d > 2 ** 31
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    pick = [0, 262143, 524288, rows - 1]
    x[pick] = torch.randn((4, d), generator=g, device=DEV).bfloat16()
    w = torch.rand(d, generator=g, device=DEV) + 0.5
    _, n = binding.block_norm(x, w_pre=w, eps=EPS, with_sum=False)
    ref.check(n[pick], ref.norm(f64(x[pick]), w_pre=f64(w), eps=EPS)["n"], True)
    b = PreparedBlockNormGrad(x, w_pre=w, dn=x, eps=EPS)
    b()
    want = ref.norm(f64(x[pick]), w_pre=f64(w), eps=EPS, dn=f64(x[pick]), want_grads=True)
    ref.check(b.dx[pick], want["dx"], True)
    ref.check(b.dw_pre, want["dw_pre"])


def test_no_rows():
    x = torch.empty((0, 40), device=DEV)
    w = torch.ones(40, device=DEV)
    s, n = binding.block_norm(x, w_pre=w)
    assert s.shape == (0, 40) and n.shape == (0, 40)
    b = PreparedBlockNormGrad(x, w_pre=w, dn=x)
    b()
    assert bool((b.dw_pre == 0).all())


def test_refusals():
    p = Problem(4, 32, "f32", seed=12)
    with pytest.raises(ValueError):
        binding.block_norm(p.x, p.z[:3])
    with pytest.raises(ValueError):
        binding.block_norm(p.x, p.z.bfloat16())
    with pytest.raises(ValueError):
        binding.block_norm(p.x, w_post=torch.ones(31, device=DEV))
    with pytest.raises(ValueError):
        binding.block_norm(p.x, w_post=p.w_post.double())
    with pytest.raises(ValueError):
        binding.block_norm(p.x, gate_after=True, w_post=p.w_post)
    with pytest.raises(ValueError):
        binding.block_norm(p.x, with_sum=False)
    with pytest.raises(ValueError):
        binding.block_norm(p.x.t().contiguous().t())
    with pytest.raises(ValueError):
        PreparedBlockNormGrad(p.x, dn=p.x)
    with pytest.raises(TypeError):
        binding.block_norm(p.x.half())
    with pytest.raises(binding.VimscanError) as e:
        binding.block_norm(p.x.bfloat16(), residual=None, res_dtype=torch.bfloat16, eps=0.0)
    assert e.value.status == -13
    with pytest.raises(binding.VimscanError) as e:
        PreparedBlockNorm(p.x, out_sum=p.x)()
    assert e.value.status == -6
    wide = torch.zeros((1, 32772), device=DEV)
    with pytest.raises(binding.VimscanError) as e:
        binding.block_norm(wide)
    assert e.value.status == -2
