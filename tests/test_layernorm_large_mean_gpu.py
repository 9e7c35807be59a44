"""The layer norm of rows whose mean is large beside their spread: the rounding of the mean does not reach the output."""
import pytest
import torch

from bidirectional_selective_scan_amd import block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ULP = 2.0 ** -23


def exact(x, eps):
    w = x.double()
    w = w - w.mean(-1, keepdim=True)
    return w / torch.sqrt((w * w).mean(-1, keepdim=True) + eps)


@pytest.mark.parametrize("d", [64, 100, 768, 1531, 4096, 8190])
@pytest.mark.parametrize("value", [0.1, 3.0, -1e4])
def test_constant_rows_are_zero(d, value):
    """After a second look at the mean an element is off by half an ulp of what the first left, itself some (d / 64 + 10) half ulps of the
    value: about 1e-10 of it at most, over sqrt(eps)."""
    x = torch.full((3, d), value, device=DEV)
    eps = 1e-12
    left = abs(value) * (d / 64 + 10) * ULP * (d / 64 + 10) * ULP
    assert block.layer_norm(x, eps=eps)[1].abs().max().item() <= left * eps ** -0.5


@pytest.mark.parametrize("d", [64, 768, 1531, 8192])
@pytest.mark.parametrize("mean", [0.0, 10.0, 1000.0, 1e5])
@pytest.mark.parametrize("residual", [False, True])
def test_a_large_mean_costs_no_digits(d, mean, residual):
    """Inputs are taken as they are in fp32, so nothing is lost in s - mean but the rounding of the mean, which the second look
    takes off. What is left: (d / 64 + 24) ulps of the magnitudes, as for a mean of 0; with a residual the sum's own rounding, half
    an ulp of its value, which is in the spread as well."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(d)
    x = torch.randn(64, d, generator=gen, device=DEV) + mean
    r = torch.randn(64, d, generator=gen, device=DEV) if residual else None
    n = block.layer_norm(x, r)[1]
    want = exact(x.double() + r.double() if residual else x, 1e-5)
    bound = (d / 64 + 24) * ULP * want.abs().clamp(min=1.0) + (ULP * (mean + 8) if residual else 0.0)
    assert ((n - want).abs() <= bound).all(), ((n - want).abs() / bound).max().item()


@pytest.mark.parametrize("d", [64, 1531])
def test_gradients_at_a_large_mean(d):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(d)
    x = torch.randn(200, d, generator=gen, device=DEV) + 1000.0
    w, dn = torch.randn(d, generator=gen, device=DEV), torch.randn(200, d, generator=gen, device=DEV)
    g = block.PreparedLayerNormGrad(x, weight=w, bias=w, dn=dn)
    g()
    xh = exact(x, 1e-5)
    rho = 1.0 / torch.sqrt(x.double().var(-1, unbiased=False, keepdim=True) + 1e-5)
    gw = dn.double() * w.double()
    dx = rho * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
    big = rho * (gw.abs().amax(-1, keepdim=True) * (1 + xh.abs()) + xh.abs() * (gw * xh).abs().mean(-1, keepdim=True))
    assert ((g.dx - dx).abs() <= (d / 64 + 48) * ULP * big).all()
    dw = (dn.double() * xh).sum(0)
    assert ((g.dweight - dw).abs() <= (d / 64 + 24 + 200) * ULP * (dn.double() * xh).abs().clamp(min=1e-3).sum(0)
            + (d / 64 + 24) * ULP * dn.double().abs().sum(0)).all()
