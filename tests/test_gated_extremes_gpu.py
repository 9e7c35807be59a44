"""The gated recurrence's gradients where a gate is all but closed, closed or NaN: every pair of gate and
decay rate, both io types, one and two channels a lane, against the 64-bit form (block_reference)."""
import numpy as np
import pytest
import torch

import block_reference as ref
from test_gated_gpu import DEV, Problem, f64, rates

pytestmark = pytest.mark.gpu

NAMES = ("y", "h_last", "dx", "dr", "di", "dlam", "dh0")
INF = float("inf")
GATES = [-INF, -1e4, -200.0, -110.0, -104.0, -100.0, -96.0, -92.0, -90.0, -88.0, -87.5, -87.0, -86.0, -84.0, -80.0, -75.0,
         -60.0, -40.0, -20.0, 20.0, 60.0, 88.0, 200.0, 1e4, INF]
# decay rates from none to very fast, and those of slowest decays 0.9 to 0.999
RATES = [-100.0, -90.0, -88.0, -87.0, -86.0, -80.0, -60.0, -30.0, -10.0, -5.0, 0.0, 5.0, 30.0] + rates(
    np.random.default_rng(3), 5).tolist()


def outputs(fwd, bwd):
    return dict(zip(NAMES, (fwd.y, fwd.h_last, bwd.dx, bwd.dr, bwd.di, bwd.dlam, bwd.dh0)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("extra", [0, 1])
@pytest.mark.parametrize("which", ["r", "i", "both"])
def test_every_gate_with_every_rate(io, extra, which):
    """Every second token has one of the gates in all channels, every channel one of the rates; in odd widths a
    lane has one channel, in even ones two."""
    d = len(RATES) + extra
    p = Problem(2, 2 * len(GATES) + 16, d, io, seed=41)
    p.lam[:len(RATES)] = torch.tensor(RATES, device=DEV)
    gates = torch.tensor(GATES, device=DEV).to(p.x.dtype)
    span = slice(1, 2 * len(GATES), 2)
    if which != "i":
        p.r[:, span] = gates[None, :, None]
    if which != "r":
        p.i[:, span] = gates.flip(0)[None, :, None]
    finite = Problem(2, 2 * len(GATES) + 16, d, io, seed=41)
    for name in ("x", "dy", "h0", "dh_last", "lam"):
        setattr(finite, name, getattr(p, name))
    finite.r, finite.i = p.r.clamp(-1e4, 1e4), p.i.clamp(-1e4, 1e4)
    with np.errstate(all="ignore"):
        want = finite.reference()
    # A gate below 2^-126 is held there or flushed to 0, as is 1 - a^2: m = sqrt(-2 u) is then off by up to
    # sqrt(2 c softplus(30) 2^-126) = 2.4e-18. One token's terms carry that times x (below 5) and the gradient of
    # its state (below 5 (tokens + 1), without decay); dlam and the states add them up over the tokens.
    tokens = 2 * (2 * len(GATES) + 16)
    slack = 2.4e-18 * 5 * 5 * (tokens + 1) * tokens
    fwd, bwd = p.run()
    for name, t in outputs(fwd, bwd).items():
        assert bool(t.isfinite().all()), name
        ref.check(t, (want[name][0], want[name][1] + slack), io == "bf16" and name in ("y", "dx", "dr", "di"), name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [33, 64])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gate", ["r", "i"])
def test_a_nan_gate_reaches_what_depends_on_it(io, d, reverse, gate):
    """A NaN in r or i, in a sequence inside one tile and in one of many tiles: exactly the outputs that depend on
    it by the definition are NaN, at the token, before it, behind it, in dh0 and in dlam."""
    lens = [20, 0, 700, 33, 5]
    offsets = np.concatenate([[0], np.cumsum(lens)]).tolist()
    p = Problem(1, offsets[-1], d, io, offsets=offsets, reverse=reverse, seed=42)
    for token, channel in ((11, 3), (offsets[2] + 350, 5), (offsets[3] + 32, 7), (offsets[4], 9), (offsets[4] - 33, 9)):
        getattr(p, gate)[0, token, channel] = float("nan")
    with np.errstate(all="ignore"):
        want = p.reference()
    fwd, bwd = p.run()
    for name, t in outputs(fwd, bwd).items():
        got, lost = np.isnan(f64(t)).reshape(want[name][0].shape), np.isnan(want[name][0])
        assert lost.any() or (gate == "i" and name == "dh0"), name
        assert (got == lost).all(), (name, np.argwhere(got != lost)[:5])
