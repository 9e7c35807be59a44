"""Linear attention on the paths that small calls do not take, against a 64-bit form with tight bounds (linattn_bounds): folds of
more than eight segments, the search among more than 64 packed sequences, inputs past the memory-side cache, gradients without
the decays', offsets that break the rules with guards around every output and the workspace."""
import numpy as np
import pytest
import torch

import linattn_bounds
from bidirectional_selective_scan_amd.binding import PreparedLinAttn, PreparedLinAttnGrad
from test_linattn_decay_grad_gpu import DEV, Call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dk,dv,decay", [(64, 64, "token"), (24, 128, "head")])
def test_a_long_sequence_of_many_segments(io, reverse, dk, dv, decay):
    p = Call((1, 2503), 1, 1, dk, dv, io, decay, reverse, seed=1, strength=0.02)
    p.check()
    assert p.plan["kernels"] == 3 and p.plan["chunks"] > 16


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
def test_many_packed_sequences_cut(io, reverse):
    rng = np.random.default_rng(2)
    lens = [int(v) for v in rng.integers(0, 260, 150)]
    lens[70], lens[3], lens[149] = 900, 0, 1
    p = Call(lens, 1, 1, 32, 16, io, reverse=reverse, seed=2, strength=0.05)
    p.check()
    assert p.plan["kernels"] == 3 and p.plan["sequences"] == 150


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape,H,split", [((16, 2000), 24, True), ((600, 150), 12, False)])
def test_inputs_past_the_memory_side_cache(io, shape, H, split):
    """Two heads of the first and the last sequence stand for all."""
    d = 64 if io == "bf16" else 32     # (heads whose rows are lines of their own and that one wave reads)
    p = Call(shape, H, H, d, d, io, state=False, seed=3, strength=0.05)
    assert p.n * H * 4 * d * p.q.element_size() > 256 << 20
    got = p.run()
    assert (p.plan["kernels"] == 3) == split
    few = Call((2, shape[1]), 2, 2, d, d, io, state=False)
    pick = [0, shape[0] - 1]
    for name in ("q", "k", "v", "dy", "g"):
        setattr(few, name, getattr(p, name)[pick][:, :, [1, H - 1]].contiguous())
    want = few.want()
    for name in ("y", "dq", "dk", "dv", "dg"):
        part = got[name].reshape(*shape, H, -1)[pick][:, :, [1, H - 1]]
        check(part, want[name], p.bf16 and name != "dg", name)
    check(got["h_last"][pick][:, [1, H - 1]], want["h_last"], False, "h_last")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(4, 4), (4, 2), (3, 1)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (16, 24), (128, 64), (40, 56)])
@pytest.mark.parametrize("reverse", [False, True])
def test_gradients_without_the_decays(io, H, G, dk, dv, reverse):
    p = Call((2, 170), H, G, dk, dv, io, reverse=reverse, seed=H + dk)
    p.check(decays=False)
    p = Call([70, 0, 33, 129], H, G, dk, dv, io, "head", reverse, seed=G + dv)
    p.check(decays=False)


def test_bf16_outputs_have_their_own_rounding_alone():
    """In the 2-norm an output is no further from the 64-bit form than that form's own rounding to bf16, but for a tenth of
    it: two parts of 2^-17 each, in quadrature to a rounding of 2^-9 and more, are far less; one part would be as large as it."""
    p = Call((4, 300), 4, 4, 64, 64, "bf16", seed=30)
    want = p.want()
    for decays in (True, False):
        got = p.run(decays)
        for name in ("y", "dq", "dk", "dv"):
            val = want[name][0]
            own = np.linalg.norm(torch.from_numpy(val).to(torch.bfloat16).double().numpy() - val)
            assert np.linalg.norm(got[name].reshape(val.shape) - val) <= 1.1 * own, (name, decays)


@pytest.mark.parametrize("bad", [[0, 50, 20, 73], [5, 60, 10 ** 6, 10 ** 9], [-7, -3, 2 ** 31 - 1, 0], [73, 73, 73, 0]])
@pytest.mark.parametrize("length", [73, 1000])
@pytest.mark.parametrize("G", [1, 2])
def test_offsets_that_break_the_rules_touch_no_other_memory(bad, length, G):
    """Guards around every output and the workspace of the forward and the backward pass."""
    p = Call([length // 2, 0, length - length // 2], 2, G, 16, 16, "bf16", seed=19)
    p.offsets = torch.tensor(bad, dtype=torch.int32, device=DEV)
    rooms = []

    def room(shape, dtype):
        n = int(np.prod(shape))
        whole = torch.full((n + 2048,), 3, dtype=dtype, device=DEV)
        rooms.append((whole, n))
        return whole[1024:1024 + n].view(shape)

    def untouched():
        torch.cuda.synchronize()
        for whole, n in rooms:
            assert (whole[:1024] == 3).all() and (whole[1024 + n:] == 3).all()

    args = (p.q, p.k, p.v, p.g, None, p.h0, 0, p.offsets, p.reverse)
    need = PreparedLinAttn(*args).plan["workspace_bytes"]
    call = PreparedLinAttn(*args, out=room(tuple(p.v.shape), torch.bfloat16), h_last=room(tuple(p.h0.shape), torch.float32),
                           workspace=room((need,), torch.uint8))
    call()
    untouched()
    need = PreparedLinAttnGrad(call, p.dy, p.dh).plan["workspace_bytes"]
    grad = PreparedLinAttnGrad(call, p.dy, p.dh, workspace=room((need,), torch.uint8))
    struct = grad._keep[1]
    for field, like in (("dq", p.q), ("dk", p.k), ("dv", p.v), ("dlog_decay", p.g), ("dh0", p.h0)):
        setattr(struct, field, room(tuple(like.shape), like.dtype).data_ptr())
    grad()
    untouched()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
def test_one_long_sequence_packed_with_many_short_ones(io, reverse):
    """Sequences that a plan would leave whole by their mean, one of them cut; two heads stand for all."""
    lens = [150] * 12 + [0, 1] + [150] * 8 + [4300] + [150] * 9
    p = Call(lens, 48, 48, 16, 16, io, reverse=reverse, seed=6, strength=0.05)
    got = p.run()
    assert p.plan["kernels"] == 3 and p.plan["chunk_len"] == 2048
    heads = [3, 47]
    few = Call(lens, 2, 2, 16, 16, io, reverse=reverse)
    for name in ("q", "k", "v", "dy", "g"):
        setattr(few, name, getattr(p, name)[:, :, heads].contiguous())
    few.h0, few.dh = p.h0[:, heads].contiguous(), p.dh[:, heads].contiguous()
    want = few.want()
    for name in ("y", "dq", "dk", "dv", "dg"):
        check(got[name].reshape(p.n, 48, -1)[:, heads], want[name], p.bf16 and name != "dg", name)
    for name in ("h_last", "dh0"):
        check(got[name][:, heads], want[name], False, name)


def test_gradients_of_cut_sequences_against_differences():
    """Gradients against central differences of the forward pass in fp32, several segments and windows. A difference over 2 eps of a
    loss of value W carries rounding of about 2^-22 |W| / eps and, the loss being bilinear in all but the decays, no truncation there; of
    the decays eps^2 |W|."""
    p = Call((1, 700), 2, 1, 12, 20, "f32", seed=10)
    call = PreparedLinAttn(p.q, p.k, p.v, p.g, None, p.h0)
    grad = PreparedLinAttnGrad(call, p.dy, p.dh)
    call()
    grad()
    assert call.plan["kernels"] == 3

    def loss():
        call()
        return ((call.y.double() * p.dy.double()).sum() + (call.h_last.double() * p.dh.double()).sum()).item()

    size = (call.y.double() * p.dy.double()).abs().sum().item() + (call.h_last.double() * p.dh.double()).abs().sum().item()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    for t, g in ((p.q, grad.dq), (p.k, grad.dk), (p.v, grad.dv), (p.g, grad.dlog_decay), (p.h0, grad.dh0)):
        d = torch.randn(t.shape, generator=gen, device=DEV)
        keep, eps = t.clone(), 2.0 ** -7
        t.copy_(keep + eps * d)
        up = loss()
        t.copy_(keep - eps * d)
        down = loss()
        t.copy_(keep)
        assert abs((up - down) / (2 * eps) - (g.double() * d.double()).sum().item()) <= size * (2.0 ** -22 / eps + 8 * eps ** 2)


@pytest.mark.parametrize("reverse", [False, True])
def test_folded_sequences_cut_are_those_of_a_batch(reverse):
    p = Call((2, 700), 2, 2, 32, 64, "bf16", reverse=reverse, seed=11)
    want = p.run()
    assert p.plan["kernels"] == 3
    q, k, v, g, dy = (t.reshape(1, 1400, *t.shape[2:]) for t in (p.q, p.k, p.v, p.g, p.dy))
    call = PreparedLinAttn(q, k, v, g, None, p.h0, 700, None, reverse)
    call()
    grad = PreparedLinAttnGrad(call, dy, p.dh)
    grad()
    for name, t in dict(y=call.y, h_last=call.h_last, dq=grad.dq, dk=grad.dk, dv=grad.dv, dg=grad.dlog_decay, dh0=grad.dh0).items():
        assert (t.double().cpu().numpy().reshape(want[name].shape) == want[name]).all(), name


def test_captured_and_replayed_over_windows():
    """A graph of a forward and a backward pass with borders of windows, replayed between eager calls on other inputs."""
    p = Call((300, 300), 3, 3, 32, 32, "bf16", state=False, seed=12)
    call = PreparedLinAttn(p.q, p.k, p.v, p.g)
    grad = PreparedLinAttnGrad(call, p.dy)
    call()
    grad()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c2 = PreparedLinAttn(p.q, p.k, p.v, p.g)
        g2 = PreparedLinAttnGrad(c2, p.dy)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            c2()
            g2()
    for _ in range(3):
        p.v.copy_(torch.randn_like(p.v))
        p.g.copy_(-torch.rand_like(p.g))
        call()
        grad()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((call.y, c2.y), (grad.dq, g2.dq), (grad.dk, g2.dk), (grad.dv, g2.dv), (grad.dlog_decay, g2.dlog_decay)):
            assert torch.equal(a, b)
