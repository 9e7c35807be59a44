"""What a caller gives as workspace of the recurrent block's operators is checked."""
import pytest
import torch

from bidirectional_selective_scan_amd.binding import PreparedBlockNormGrad, PreparedGated, PreparedGatedGrad
from test_gated_gpu import DEV, Problem

pytestmark = pytest.mark.gpu


def test_a_workspace_that_a_kernel_cannot_use_is_refused():
    """Memory of the host, or a strided view: refused when the call is prepared."""
    p = Problem(1, 1000, 64, "f32", seed=70)
    x = torch.randn(40, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    fwd = PreparedGated(p.inputs(), None, None, None, save_states=True)
    for ws in (torch.empty(1 << 22, dtype=torch.uint8), torch.empty(1 << 23, dtype=torch.uint8, device=DEV)[::2]):
        for call in (lambda: PreparedGated(p.inputs(), None, None, None, workspace=ws),
                     lambda: PreparedGatedGrad(fwd, p.dy, p.dh_last, workspace=ws),
                     lambda: PreparedBlockNormGrad(x, w_pre=w, dn=x, workspace=ws)):
            with pytest.raises(ValueError):
                call()
