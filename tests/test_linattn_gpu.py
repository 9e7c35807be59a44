"""Linear attention with a decay for each head on the GPU against a plain form in float64, with bounds derived from
the number formats (linattn_reference)."""
import numpy as np
import pytest
import torch

import block_reference
import linattn_reference as ref
from bidirectional_selective_scan_amd import binding
from bidirectional_selective_scan_amd.binding import PreparedLinAttn, PreparedLinAttnGrad

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


class Problem:
    """Inputs of a call and its plain form. lens: the sequences' lengths (packed) or (sequences, length)."""

    def __init__(self, lens, H, G, dk, dv, io, decay="token", state=True, reverse=False, seed=0, scale=None, seg_len=0,
                 strength=1.0):
        rng = np.random.default_rng(seed)
        self.packed = isinstance(lens, list)
        if self.packed:
            off = np.concatenate([[0], np.cumsum(lens)]).astype(int)
            self.bounds, shape = list(zip(off[:-1], off[1:])), (1, int(off[-1]))
            self.offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        else:
            nseq, length = lens
            T = seg_len or length
            self.bounds = [(i * T, (i + 1) * T) for i in range(nseq * length // T if T else nseq)]
            shape, self.offsets = (nseq, length), None
        self.shape, self.H, self.G, self.dk, self.dv = shape, H, G, dk, dv
        self.bf16, self.reverse, self.scale, self.seg_len = io == "bf16", reverse, scale, seg_len
        n = shape[0] * shape[1]
        self.n = n

        def rows(h, d):
            return torch.from_numpy(rng.standard_normal((*shape, h, d)).astype(np.float32)).to(DEV).to(DT[io])

        self.q, self.k, self.v, self.dy = rows(G, dk), rows(G, dk), rows(H, dv), rows(H, dv)
        lead = (*shape, H) if decay == "token" else (H,)
        self.g = torch.from_numpy((-strength * np.abs(rng.standard_normal(lead)) ** 3 * 0.3).astype(np.float32)).to(DEV)
        st = (len(self.bounds), H, dk, dv)
        self.h0 = torch.from_numpy(rng.standard_normal(st).astype(np.float32)).to(DEV) if state else None
        self.dh_last = torch.from_numpy(rng.standard_normal(st).astype(np.float32)).to(DEV) if state else None

    def forward(self, **kw):
        return PreparedLinAttn(self.q, self.k, self.v, self.g, self.scale, self.h0, self.seg_len, self.offsets,
                               self.reverse, **kw)

    def want_without_decays(self):
        return self.want(True, False)

    def want(self, grads, decays=True):
        g = f64(self.g)
        g = g if g.ndim == 1 else g.reshape(self.n, self.H)
        flat = [f64(t).reshape(self.n, *t.shape[2:]) for t in (self.q, self.k, self.v, self.dy)]
        return ref.linattn(flat[0], flat[1], flat[2], g, float(np.float32(self.dk ** -0.5 if self.scale is None else self.scale)),
                           self.bounds, None if self.h0 is None else f64(self.h0), self.reverse, flat[3] if grads else None,
                           f64(self.dh_last) if grads and self.dh_last is not None else None, self.bf16, decays)

    def check(self, what=""):
        want = self.want(True)
        call = self.forward()
        call()
        grad = PreparedLinAttnGrad(call, self.dy, self.dh_last)
        grad()
        got = dict(y=call.y, h_last=call.h_last, dq=grad.dq, dk=grad.dk, dv=grad.dv, dg=grad.dlog_decay)
        if self.h0 is not None:
            got["dh0"] = grad.dh0
        for name, t in got.items():
            block_reference.check(t, want[name], self.bf16 and name in ("y", "dq", "dk", "dv"), f"{what} {name}")
        return call, grad


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (16, 16), (128, 64), (32, 128), (128, 128)])
def test_lengths(io, dk, dv):
    for length in (1, 2, 31, 32, 33, 64, 70, 130):
        Problem((2, length), 2, 2, dk, dv, io, seed=length).check(f"length {length}")


def test_bf16_outputs_are_near_their_own_rounding():
    """In the 2-norm: a rounding of values spread over a binade has a relative error of at most 2^-8 / sqrt(3); an output
    in bf16 has its own and, term by term at random, that of its scores or of the state."""
    p = Problem((4, 300), 4, 4, 64, 64, "bf16", seed=30)
    want = p.want(True)
    call = p.forward()
    call()
    for decays in (True, False):
        g = PreparedLinAttnGrad(call, p.dy, p.dh_last, decays=decays)
        g()
        for name, t in (("y", call.y), ("dq", g.dq), ("dk", g.dk), ("dv", g.dv)):
            ref_v = want[name][0]
            err = np.linalg.norm(f64(t).reshape(ref_v.shape) - ref_v) / np.linalg.norm(ref_v)
            assert err <= 2.0 ** -8 / 3 ** 0.5 * 2 ** 0.5, (name, err)
        for name, t in (("h_last", call.h_last), ("dh0", g.dh0)) + ((("dg", g.dlog_decay),) if decays else ()):
            ref_v = want[name][0]
            err = np.linalg.norm(f64(t).reshape(ref_v.shape) - ref_v) / np.linalg.norm(ref_v)
            assert err <= 1e-5, (name, err)
        block_reference.check(g.dq, p.want_without_decays()["dq"] if not decays else want["dq"], True, "dq")
        block_reference.check(g.dk, p.want_without_decays()["dk"] if not decays else want["dk"], True, "dk")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(40, 56), (1, 1), (7, 33), (33, 7), (65, 127), (127, 65), (20, 96), (80, 24), (128, 3)])
def test_head_sizes(io, dk, dv):
    Problem((3, 75), 3, 3, dk, dv, io, seed=dk).check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(4, 1), (6, 3), (6, 2), (5, 5)])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_shared_heads_and_decays(io, H, G, decay):
    Problem((2, 75), H, G, 24, 40, io, decay, seed=H + G).check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("state", [False, True])
def test_packed(io, reverse, decay, state):
    p = Problem([30, 0, 64, 1, 0, 129, 33, 0], 2, 1, 32, 48, io, decay, state, reverse, seed=5)
    call, grad = p.check()
    if state:
        for j, (lo, hi) in enumerate(p.bounds):
            if lo == hi:
                assert torch.equal(call.h_last[j], p.h0[j]) and torch.equal(grad.dh0[j], p.dh_last[j])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
def test_sequences_cut_into_segments(io, reverse):
    p = Problem((2, 333), 2, 2, 64, 32, io, reverse=reverse, seed=6)
    assert p.forward().plan["chunks"] > 3
    p.check("uniform")
    p = Problem([200, 0, 333, 1, 64, 65], 1, 1, 32, 64, io, reverse=reverse, seed=7)
    call, _ = p.check("packed")
    assert call.plan["kernels"] == 3
    p = Problem((1, 300), 2, 2, 16, 32, io, "head", reverse=reverse, seg_len=150, seed=8)
    p.check("folded")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_many_sequences_whole(io):
    p = Problem((40, 70), 32, 4, 16, 16, io, seed=9)
    assert p.forward().plan["kernels"] == 1
    p.check()


def test_against_differences():
    """Gradients against central differences of the forward pass (fp32, long segments and shared heads). A
    difference over 2 eps of a loss of value W carries rounding of about 2^-22 |W| / eps and, the loss being bilinear in
    all but the decays, no truncation there; of the decays eps^2 |W|."""
    p = Problem((1, 150), 2, 1, 12, 20, "f32", seed=10)
    call = p.forward()
    grad = PreparedLinAttnGrad(call, p.dy, p.dh_last)
    call()
    grad()

    def loss():
        call()
        return ((call.y.double() * p.dy.double()).sum() + (call.h_last.double() * p.dh_last.double()).sum()).item()

    size = (call.y.double() * p.dy.double()).abs().sum().item() + (call.h_last.double() * p.dh_last.double()).abs().sum().item()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    for t, g in ((p.q, grad.dq), (p.k, grad.dk), (p.v, grad.dv), (p.g, grad.dlog_decay), (p.h0, grad.dh0)):
        d = torch.randn(t.shape, generator=gen, device=DEV)
        keep = t.clone()
        eps = 2.0 ** -7
        t.copy_(keep + eps * d)
        up = loss()
        t.copy_(keep - eps * d)
        down = loss()
        t.copy_(keep)
        want = (g.double() * d.double()).sum().item()
        assert abs((up - down) / (2 * eps) - want) <= size * (2.0 ** -22 / eps + 8 * eps ** 2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strides(io):
    """Slices of one projection, an interleaved layout, one sequence in [heads][tokens][d] order, odd offsets."""
    p = Problem((2, 70), 3, 3, 16, 24, io, seed=11)
    base, _ = p.check()
    for build in ("sliced", "heads-first", "interleaved", "odd"):
        r = Problem((2, 70), 3, 3, 16, 24, io, seed=11)
        if build == "sliced":
            wide = torch.zeros(2, 70, 3 * (16 + 16 + 24) + 6, dtype=DT[io], device=DEV)
            parts = wide[..., 2:2 + 48], wide[..., 50:98], wide[..., 100:172]
            news = [s.unflatten(-1, (3, -1)) for s in parts]
        elif build == "odd":
            wide = torch.zeros(2, 70, 3 * (16 + 16 + 24) + 5, dtype=DT[io], device=DEV)
            parts = wide[..., 1:49], wide[..., 49:97], wide[..., 98:170]
            news = [s.unflatten(-1, (3, -1)) for s in parts]
        elif build == "interleaved":
            wide = torch.zeros(2, 70, 3, 16 + 16 + 24, dtype=DT[io], device=DEV)
            news = [wide[..., :16], wide[..., 16:32], wide[..., 32:]]
        else:
            news = [torch.zeros(3, 140, d, dtype=DT[io], device=DEV).transpose(0, 1).view(2, 70, 3, d) for d in (16, 16, 24)]
        for new, old in zip(news, (r.q, r.k, r.v)):
            new.copy_(old)
        r.q, r.k, r.v = news
        wide_g = torch.zeros(2, 70, 5, device=DEV)
        wide_g[..., 1:4] = r.g
        r.g = wide_g[..., 1:4]
        call, _ = r.check(build)
        assert torch.equal(call.y, base.y) and torch.equal(call.h_last, base.h_last)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_extreme_decays(io):
    """Minus infinity (a reset), the type's lowest value, zero and very strong decays, next to ordinary ones."""
    p = Problem((2, 140), 2, 2, 16, 16, io, seed=12, strength=1.0)
    g = p.g
    g[0, 40, 0] = float("-inf")
    g[0, 41, 0] = float("-inf")
    g[0, 70, 1] = torch.finfo(torch.float32).min
    g[1, :, 0] = 0.0
    g[1, 30:60, 1] = -150.0
    g[1, 139] = float("-inf")
    p.check()
    p = Problem((2, 90), 2, 2, 16, 16, io, "head", seed=13)
    p.g.copy_(torch.tensor([float("-inf"), 0.0]))
    p.check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("which", ["q", "k", "v", "g", "h0"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_infinity_stay_where_they_belong(io, split, which, bad):
    """A token's NaN or infinity reaches neither the tokens before it nor other heads or sequences: those have the same bits."""
    H = 3
    shape = (2, 200) if split else (400, 70)

    def build():
        return Problem(shape, H, H, 16, 24, io, seed=14)

    p = build()
    clean = p.forward()
    assert (clean.plan["kernels"] == 3) == split
    clean()
    at = 45
    if which == "g":
        p.g[1, at, 1] = float("nan")
    elif which == "h0":
        p.h0[1, 1, 3, 5] = bad
    else:
        getattr(p, which)[1, at, 1, 5] = bad
    call = p.forward()
    call()
    y, y0 = call.y, clean.y
    for b in (0, 1, -1):
        for h in range(H):
            same = (b != 1 and b % shape[0] != 1) or h != 1
            upto = shape[1] if same else (0 if which == "h0" else at)
            assert torch.equal(y[b, :upto, h], y0[b, :upto, h]), (b, h)
    assert torch.equal(call.h_last[0], clean.h_last[0]) and torch.equal(call.h_last[1, [0, 2]], clean.h_last[1, [0, 2]])
    # and it is not lost
    hit = y[1, (0 if which == "h0" else at):, 1].float()
    assert not torch.isfinite(hit[0]).all()
    if which == "q":
        assert torch.equal(y[1, at + 1:, 1], y0[1, at + 1:, 1])
    elif which != "v" and which != "h0":
        assert not torch.isfinite(hit).all(-1).any()
    else:
        assert not torch.isfinite(hit[:, 5]).any() and torch.equal(hit[:, :5], y0[1, (0 if which == "h0" else at):, 1, :5].float())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_only_one_gradient_given(io):
    p = Problem((2, 100), 2, 2, 16, 16, io, seed=15)
    call = p.forward()
    call()
    keep = p.dh_last
    p.dh_last = None
    want = p.want(True)
    g = PreparedLinAttnGrad(call, p.dy)
    g()
    for name, t in (("dq", g.dq), ("dk", g.dk), ("dv", g.dv), ("dg", g.dlog_decay), ("dh0", g.dh0)):
        block_reference.check(t, want[name], p.bf16 and name in ("dq", "dk", "dv"), name)
    p.dh_last, p.dy = keep, torch.zeros_like(p.dy)
    want = p.want(True)
    g = PreparedLinAttnGrad(call, None, p.dh_last)
    g()
    for name, t in (("dq", g.dq), ("dk", g.dk), ("dv", g.dv), ("dg", g.dlog_decay), ("dh0", g.dh0)):
        block_reference.check(t, want[name], p.bf16 and name in ("dq", "dk", "dv"), name)
    none = PreparedLinAttnGrad(call, p.dy, p.dh_last, decays=False)
    none()
    assert none.dlog_decay is None


def test_empty_calls():
    for shape in ((2, 0), (0, 5)):
        p = Problem(shape, 2, 2, 16, 16, "bf16", "head", seed=16)
        call = p.forward()
        call()
        g = PreparedLinAttnGrad(call, p.dy, p.dh_last)
        g.dlog_decay.fill_(7.0)
        g()
        assert torch.equal(call.h_last, p.h0) and torch.equal(g.dh0, p.dh_last)
        assert torch.equal(g.dlog_decay, torch.zeros(2, device=DEV))


def test_same_bits_every_time():
    for io in ("bf16", "f32"):
        p = Problem([200, 0, 333, 64], 4, 2, 64, 64, io, "head", seed=17)
        call = p.forward()
        grad = PreparedLinAttnGrad(call, p.dy, p.dh_last)
        outs = []
        for _ in range(3):
            call()
            grad()
            outs.append([t.clone() for t in (call.y, call.h_last, grad.dq, grad.dk, grad.dv, grad.dlog_decay, grad.dh0)])
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_rows_outside_are_left_as_they_were():
    """Outputs given inside larger arrays, and tokens behind the last packed sequence: untouched."""
    p = Problem([40, 33], 2, 2, 16, 16, "bf16", seed=18)
    room = torch.full((p.n + 64, 2, 16), 3.0, dtype=torch.bfloat16, device=DEV)
    call = p.forward(out=room[32:32 + p.n].view(1, p.n, 2, 16))
    call()
    assert (room[:32] == 3).all() and (room[32 + p.n:] == 3).all()
    block_reference.check(call.y, p.want(False)["y"], True)
    # offsets that end before the array does
    short = torch.tensor([0, 40, 60], dtype=torch.int32, device=DEV)
    out = torch.full((1, p.n, 2, 16), 5.0, dtype=torch.bfloat16, device=DEV)
    q = PreparedLinAttn(p.q, p.k, p.v, p.g, p.scale, p.h0, 0, short, out=out)
    q()
    assert torch.equal(q.y[:, :60], call.y[:, :60]) and (q.y[:, 60:] == 5).all()


@pytest.mark.parametrize("bad", [[0, 50, 20, 73], [5, 60, 10 ** 6, 10 ** 9], [-7, -3, 2 ** 31 - 1, 0], [73, 73, 73, 0]])
@pytest.mark.parametrize("length", [73, 1000])
def test_offsets_that_break_the_rules_stay_inside(bad, length):
    p = Problem([length // 2, 0, length - length // 2], 2, 2, 16, 16, "bf16", seed=19)
    guard = torch.full((p.n + 64, 2, 16), 3.0, dtype=torch.bfloat16, device=DEV)
    p.offsets = torch.tensor(bad, dtype=torch.int32, device=DEV)
    call = p.forward(out=guard[32:32 + p.n].view(1, p.n, 2, 16))
    call()
    grad = PreparedLinAttnGrad(call, p.dy, p.dh_last)
    grad()
    torch.cuda.synchronize()
    assert (guard[:32] == 3).all() and (guard[32 + p.n:] == 3).all()


# ------------------------------------------------------------------------------------------
# Single tokens


def step_reference(q, k, v, g, state, scale):
    rep = v.shape[1] // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    a = np.exp(np.maximum(np.broadcast_to(g, v.shape[:2]), -200.0))[..., None, None]
    kv = k[..., None] * v[..., None, :]
    s = a * state + kv
    mag = np.abs(a * state) + np.abs(kv)
    se = block_reference.ULP * (np.abs(np.log(np.maximum(a, 1e-80))) + 6) * mag
    y = scale * (q[..., None] * s).sum(-2)
    dk = q.shape[-1]
    ye = abs(scale) * (np.abs(q)[..., None] * (se + block_reference.ULP * (dk + 6) * mag)).sum(-2)
    return (y, ye + block_reference.TINY), (s, se + block_reference.TINY)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,dk,dv", [(2, 2, 64, 64), (3, 1, 16, 16), (4, 2, 128, 128), (2, 2, 40, 56), (1, 1, 1, 1), (2, 1, 7, 33),
                                       (2, 2, 33, 100), (2, 2, 5, 32), (1, 1, 128, 127)])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_step(io, H, G, dk, dv, decay):
    rng = np.random.default_rng(dk)
    B, slots = 5, 9

    def rows(h, d):
        return torch.from_numpy(rng.standard_normal((B, h, d)).astype(np.float32)).to(DEV).to(DT[io])

    q, k, v = rows(G, dk), rows(G, dk), rows(H, dv)
    g = torch.from_numpy(-np.abs(rng.standard_normal((B, H) if decay == "token" else H)).astype(np.float32)).to(DEV)
    pool = torch.from_numpy(rng.standard_normal((slots, H, dk, dv)).astype(np.float32)).to(DEV)
    before = pool.clone()
    src = torch.tensor([3, 0, 7, 1, 12], dtype=torch.int32, device=DEV)
    dst = torch.tensor([3, 5, 2, -1, 4], dtype=torch.int32, device=DEV)
    y = binding.linattn_step(q, k, v, g, pool, 0.3, src, dst)
    gg = f64(g) if decay == "head" else f64(g)[:3]
    want_y, want_s = step_reference(f64(q)[:3], f64(k)[:3], f64(v)[:3], gg, f64(before)[[3, 0, 7]], float(np.float32(0.3)))
    block_reference.check(y[:3], want_y, io == "bf16", "y")
    block_reference.check(pool[[3, 5, 2]], want_s, False, "state")
    assert (y[3:] == 0).all()
    rest = [s for s in range(slots) if s not in (3, 5, 2)]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_steps_continue_a_sequence(io):
    """A prompt's final state, then token by token: each within its own bound of the whole sequence's float64 form."""
    p = Problem((3, 50), 4, 2, 32, 48, io, seed=20)
    want = p.want(False)
    cut = [t[:, :30].contiguous() for t in (p.q, p.k, p.v, p.g)]
    y, state = binding.linattn_fwd(*cut, h0=p.h0)
    ys = [y]
    for t in range(30, 50):
        ys.append(binding.linattn_step(p.q[:, t], p.k[:, t], p.v[:, t], p.g[:, t].contiguous(), state)[:, None])
    block_reference.check(torch.cat(ys, 1), want["y"], io == "bf16", "y")
    block_reference.check(state, want["h_last"], False, "state")


def test_step_skips_nan_of_skipped_rows():
    q = torch.full((1, 1, 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    pool = torch.ones(2, 1, 16, 16, device=DEV)
    y = binding.linattn_step(q, q, q, torch.zeros(1, device=DEV), pool, slots_in=torch.tensor([2], dtype=torch.int32, device=DEV))
    assert (y == 0).all() and (pool == 1).all()


# ------------------------------------------------------------------------------------------
# Graphs, streams, refusals


def test_captured_and_replayed():
    p = Problem([200, 0, 133, 64], 2, 2, 32, 32, "bf16", seed=21)
    call = p.forward()
    grad = PreparedLinAttnGrad(call, p.dy, p.dh_last)
    call()
    grad()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c2 = p.forward()
        g2 = PreparedLinAttnGrad(c2, p.dy, p.dh_last)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            c2()
            g2()
    for k in range(3):
        new = torch.randn_like(p.v)
        p.v.copy_(new)
        call()
        grad()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((call.y, c2.y), (call.h_last, c2.h_last), (grad.dq, g2.dq), (grad.dk, g2.dk), (grad.dv, g2.dv),
                     (grad.dlog_decay, g2.dlog_decay), (grad.dh0, g2.dh0)):
            assert torch.equal(a, b)


def test_two_streams():
    a, b = (Problem((2, 333), 2, 2, 64, 64, "bf16", seed=s) for s in (22, 23))
    want = []
    for p in (a, b):
        c = p.forward()
        c()
        want.append((c.y.clone(), c.h_last.clone()))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    calls = [p.forward(stream=s.cuda_stream) for p, s in ((a, s1), (b, s2))]
    torch.cuda.synchronize()
    for _ in range(4):
        for c in calls:
            c()
    torch.cuda.synchronize()
    for c, (y, h) in zip(calls, want):
        assert torch.equal(c.y, y) and torch.equal(c.h_last, h)


def test_refusals():
    p = Problem((2, 20), 2, 2, 16, 16, "bf16", seed=24)
    args = [p.q, p.k, p.v, p.g]

    def bad(k, t, exc=ValueError):
        a = list(args)
        a[k] = t
        with pytest.raises(exc):
            PreparedLinAttn(*a)

    bad(0, p.q.float())
    bad(1, p.k[:, :10])
    bad(2, p.v[..., ::2])
    bad(3, p.g.double())
    bad(3, p.g[:1])
    bad(0, p.q.half(), TypeError)
    bad(0, p.q.cpu())
    bad(2, p.v[:, :, :1].expand(2, 20, 3, 16))
    with pytest.raises(ValueError):
        PreparedLinAttn(*args, h0=torch.zeros(2, 2, 16, 15, device=DEV))
    with pytest.raises(ValueError):
        PreparedLinAttn(*args, seg_len=10, offsets=torch.tensor([0, 40], dtype=torch.int32, device=DEV))
    with pytest.raises(binding.VimscanError):
        PreparedLinAttn(*args, seg_len=7)
    with pytest.raises(binding.VimscanError):
        wide = torch.zeros(1, 4, 1, 129, dtype=torch.bfloat16, device=DEV)
        PreparedLinAttn(wide, wide, wide, torch.zeros(1, device=DEV))
    with pytest.raises(binding.VimscanError) as e:
        PreparedLinAttn(*args, out=p.v)()
    assert e.value.status == -6
    with pytest.raises(binding.VimscanError) as e:
        PreparedLinAttn(*args, scale=float("nan"))()
    assert e.value.status == -13
    with pytest.raises(ValueError):
        PreparedLinAttnGrad(p.forward(), p.dy[:, :5])
    with pytest.raises(ValueError):
        binding.linattn_step(p.q[:, 0], p.k[:, 0], p.v[:, 0], p.g[:, 0].contiguous(), torch.zeros(2, 2, 16, 8, device=DEV))
