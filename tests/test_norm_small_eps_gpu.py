"""The norms with an eps below the normal fp32 numbers, where a row's variance (or mean square) is 0: the root's inverse is
large but finite, so such rows give 0 and their gradients are those of the formula."""
import pytest
import torch

from bidirectional_selective_scan_amd import block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ULP = 2.0 ** -23


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 768, 1531, 4096])
@pytest.mark.parametrize("eps", [1e-39, 1e-42, 1e-30])
def test_rows_without_spread(io, d, eps):
    x = torch.zeros(3, d, dtype=io, device=DEV)
    bias = torch.arange(d, device=DEV, dtype=torch.float32)
    assert torch.equal(block.layer_norm(x, bias=bias, eps=eps)[1], bias.to(io).expand(3, d))
    ones = torch.ones(d, device=DEV)
    total, n = block.block_norm(x, w_pre=ones, eps=eps)
    assert (total == 0).all() and (n == 0).all()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    dn = torch.randn(3, d, generator=gen, device=DEV).to(io)
    rho = float(torch.tensor(eps, dtype=torch.float32).double() ** -0.5)
    half = 2.0 ** -8 if io == torch.bfloat16 else 0.0
    # with every xh = 0: ds = rho (dn - mean dn), of the block norm rho dn. The inverse of the root has two ulps, the mean d / 64 + 8
    # additions and its product an ulp each, the difference and its product one.
    for call, want in ((block.PreparedLayerNormGrad(x, dn=dn, eps=eps), dn.double() - dn.double().mean(-1, keepdim=True)),
                       (block.PreparedBlockNormGrad(x, w_pre=ones, dn=dn, eps=eps), dn.double())):
        call()
        bound = rho * ULP * (d / 64 + 16) * dn.double().abs().amax(-1, keepdim=True) + half * rho * want.abs()
        assert ((call.dx.double() - rho * want).abs() <= bound).all()
