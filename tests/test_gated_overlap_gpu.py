"""Gated recurrences that hand states on: several at the same time on several streams, and workgroups that go on
alone because a state does not come."""
import numpy as np
import pytest
import torch

from bidirectional_selective_scan_amd import binding
from test_gated_gpu import Problem

pytestmark = pytest.mark.gpu


def outputs(f, b):
    return (f.y, f.h_last, f.states, b.dx, b.dr, b.di, b.dlam, b.dh0)


def calls(p, stream):
    """A prepared forward and backward pass with buffers of their own on a stream, and their outputs."""
    f = binding.PreparedGated(p.inputs(), None, None, None, save_states=True, stream=stream.cuda_stream)
    b = binding.PreparedGatedGrad(f, p.dy, p.dh_last, stream=stream.cuda_stream)
    return f, b, outputs(f, b)


@pytest.mark.parametrize("shapes", [((1, 40000, 512), (1, 40000, 512)), ((1, 60000, 256), (6, 1025, 768), (40, 197, 384)),
                                    ((2, 65, 32), (1, 30000, 1024), (2, 65, 32))], ids=["long", "mixed", "small"])
def test_overlapping_calls(shapes):
    """Calls of several streams at once, each stream with its own inputs and workspaces: the same bits as one call
    after the other."""
    work = []
    for k, shape in enumerate(shapes):
        p = Problem(*shape, "bf16", seed=50 + k, reverse=k % 2 == 1)
        p.run()
        s = torch.cuda.Stream()
        work.append((p, s) + calls(p, s))
    torch.cuda.synchronize()
    want = []
    for p, s, f, b, outs in work:
        f()
        b()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(6):
        for _, _, f, b, _ in work:
            f()
            b()
    torch.cuda.synchronize()
    for w, (_, _, _, _, outs) in zip(want, work):
        for a, t in zip(w, outs):
            assert torch.equal(a, t)


@pytest.fixture
def no_waiting():
    """Every workgroup whose state is not there at its first look goes on alone."""
    binding.gated_wait_reads(0)
    yield
    binding.gated_wait_reads()


PACKED = [[700, 1, 0, 1900, 64, 64, 0, 3, 2400], [5000], [1] * 900 + [2500] + [0] * 40 + [1600]]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [66, 37])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("seqlen,seg,lens", [(2200, 0, None), (3000, 600, None)] + [(0, 0, v) for v in PACKED],
                         ids=["rows", "folded", "packed", "one", "short"])
def test_alone_gives_the_same_bits(io, d, reverse, seqlen, seg, lens, request):
    """More than two groups of tiles in either direction, so that the states of whole groups are walked again; one
    and two channels a lane, long and short tiles. Rows around y are not touched."""
    offsets = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).tolist()
    p = Problem(1 if lens else 2, offsets[-1] if lens else seqlen, d, io, offsets=offsets, seg_len=seg, reverse=reverse, seed=60)
    if lens is None:
        p.x[0, 5, 1] = float("nan")
        p.dy[1, 900, 2] = float("inf")
    f0, b0 = p.run()
    want = [t.clone() for t in outputs(f0, b0)]
    before = binding.gated_alone()
    request.getfixturevalue("no_waiting")
    ybuf = torch.full((p.x.numel() // d + 8, d), 7.0, dtype=p.x.dtype, device=p.x.device)
    f = binding.PreparedGated(p.inputs(), None, None, None, save_states=True, out=ybuf[4:-4].view_as(p.x))
    f()
    b = binding.PreparedGatedGrad(f, p.dy, p.dh_last)
    b()
    for name, a, t in zip(("y", "h_last", "states", "dx", "dr", "di", "dlam", "dh0"), want, outputs(f, b)):
        t = t.contiguous()
        same = (a == t) | (a.isnan() & t.isnan())
        assert bool(same.all()), (name, same.logical_not().nonzero()[:4].tolist())
    assert bool((ybuf[:4] == 7).all()) and bool((ybuf[-4:] == 7).all())
    assert binding.gated_alone() > before
