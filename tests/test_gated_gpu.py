"""The gated linear recurrence on the GPU (forward, backward, single tokens) against its 64-bit form,
element by element within the error that 32-bit arithmetic may leave (block_reference)."""
import numpy as np
import pytest
import torch

import block_reference as ref
from bidirectional_selective_scan_amd import binding
from bidirectional_selective_scan_amd.binding import (GatedInputs, PreparedGated, PreparedGatedGrad, PreparedGatedStep)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
C = 8.0


def rates(rng, d):
    a = rng.uniform(0.9, 0.999, d)
    return np.log(np.expm1(-np.log(a) / C))


def tensor(a, io="f32"):
    t = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV)
    return t.to(torch.bfloat16) if io == "bf16" else t


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Problem:
    """Random inputs of a shape: tokens as (batch, seqlen, d) or packed by offsets."""

    def __init__(self, batch, seqlen, d, io="f32", offsets=None, seg_len=0, state=True, reverse=False, seed=0,
                 fused=False):
        rng = np.random.default_rng(seed)
        self.io, self.d, self.reverse, self.seg_len = io, d, reverse, seg_len
        n = batch * seqlen
        if fused:   # x, r and i as column slices of one array
            buf = tensor(rng.standard_normal((batch, seqlen, 3 * d + 5)), io)
            self.x, self.r, self.i = buf[..., :d], buf[..., d:2 * d], buf[..., 2 * d + 5:]
        else:
            self.x, self.r, self.i = (tensor(rng.standard_normal((batch, seqlen, d)), io) for _ in range(3))
        self.dy = tensor(rng.standard_normal((batch, seqlen, d)), io)
        self.lam = tensor(rates(rng, d))
        self.bounds = ref.bounds_of(n // seg_len if seg_len else batch, seg_len or seqlen, offsets)
        nseq = len(self.bounds)
        self.h0 = tensor(rng.standard_normal((nseq, d))) if state else None
        self.dh_last = tensor(rng.standard_normal((nseq, d))) if state else None
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)

    def inputs(self):
        return GatedInputs(self.x, self.r, self.i, self.lam, C, self.h0, self.seg_len, self.offsets, self.reverse)

    def reference(self, grads=True):
        rows = [f64(t).reshape(-1, self.d) for t in (self.x, self.r, self.i, self.dy)]
        return ref.gated(*rows[:3], f64(self.lam), C, self.bounds, f64(self.h0), self.reverse, rows[3],
                         f64(self.dh_last), grads)

    def run(self, **kw):
        fwd = PreparedGated(self.inputs(), None, None, None, save_states=True)
        fwd()
        bwd = PreparedGatedGrad(fwd, self.dy, self.dh_last, **kw)
        bwd()
        torch.cuda.synchronize()
        return fwd, bwd

    def check(self, what=""):
        want = self.reference()
        fwd, bwd = self.run()
        bf = self.io == "bf16"
        for name, t, b in (("y", fwd.y, bf), ("h_last", fwd.h_last, False), ("dx", bwd.dx, bf), ("dr", bwd.dr, bf),
                           ("di", bwd.di, bf), ("dlam", bwd.dlam, False)):
            ref.check(t, want[name], b, f"{what} {name}")
        if self.h0 is not None:
            ref.check(bwd.dh0, want["dh0"], False, f"{what} dh0")
        return fwd, bwd


@pytest.mark.parametrize("seqlen", [1, 2, 7, 63, 64, 65, 127, 128, 129, 197, 300, 1025])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_lengths(seqlen, io):
    Problem(3, seqlen, 68, io, seed=seqlen).check(f"L={seqlen}")


@pytest.mark.parametrize("d", [1, 2, 3, 4, 6, 31, 32, 33, 63, 64, 65, 66, 100, 130, 192, 257])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_widths(d, io):
    Problem(2, 150, d, io, seed=d, reverse=d % 2 == 0).check(f"D={d}")


@pytest.mark.parametrize("io,reverse", [("f32", False), ("f32", True), ("bf16", True)])
def test_folded_segments(io, reverse):
    Problem(3, 51 * 9, 70, io, seg_len=51, reverse=reverse, seed=4).check()


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens", [[5], [0, 5, 0], [1, 1, 1, 1], [0, 0, 130, 0, 0, 1, 64, 64, 63, 65, 0],
                                  [128, 128, 1, 127, 256, 0, 300, 2], [700, 1, 0, 900], [3] * 90, [0] * 70 + [200] + [0] * 70],
                         ids=lambda v: "x".join(map(str, v[:6])))
def test_packed_sequences(lens, reverse):
    offsets = np.concatenate([[0], np.cumsum(lens)]).tolist()
    for io, d in (("f32", 33), ("bf16", 64)):
        Problem(1, offsets[-1], d, io, offsets=offsets, reverse=reverse, seed=len(lens)).check(f"{io}")


def test_no_initial_state_and_no_gradient_of_the_last():
    p = Problem(2, 133, 40, "f32", state=False, seed=8)
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [48, 45])
def test_strided_inputs_and_gradients(io, d):
    """x, r, i as slices of one array (rows that no wide load is aligned to, too), gradients into
    slices of another, which is untouched between them."""
    p = Problem(2, 140, d, io, seed=9, fused=True)
    want = p.reference()
    buf = torch.full((2, 140, 3 * d + 7), 7.0, dtype=p.x.dtype, device=DEV)
    grads = (buf[..., 1:d + 1], buf[..., d + 2:2 * d + 2], buf[..., 2 * d + 5:3 * d + 5])
    fwd, bwd = p.run(grads=grads)
    for k, t in (("dx", grads[0]), ("dr", grads[1]), ("di", grads[2])):
        ref.check(t, want[k], io == "bf16", k)
    ref.check(fwd.y, want["y"], io == "bf16", "y")
    for col in (0, d + 1, 2 * d + 2, 2 * d + 4, 3 * d + 5, 3 * d + 6):
        assert bool((buf[..., col] == 7.0).all())


def test_a_long_sequence_many_workgroups():
    Problem(1, 9000, 66, "f32", seed=10).check()


def test_split_in_two_calls_carries_the_state():
    p = Problem(2, 400, 96, "f32", seed=11)
    whole, h = binding.gated_fwd(p.x, p.r, p.i, p.lam, C, p.h0)
    cut = 170
    a, ha = binding.gated_fwd(*(t[:, :cut].contiguous() for t in (p.x, p.r, p.i)), p.lam, C, p.h0)
    b, hb = binding.gated_fwd(*(t[:, cut:].contiguous() for t in (p.x, p.r, p.i)), p.lam, C, ha)
    want = p.reference(False)
    ref.check(torch.cat([a, b], 1), want["y"])
    ref.check(hb, want["h_last"])
    ref.check(h, want["h_last"])
    ref.check(whole, want["y"])


@pytest.mark.parametrize("reverse", [False, True])
def test_nothing_crosses_a_sequence_boundary(reverse):
    """NaN and infinities in one sequence (inputs and initial state) leave the others' outputs and
    gradients as they are without them."""
    lens = [40, 130, 0, 64, 200, 1, 90]
    offsets = np.concatenate([[0], np.cumsum(lens)]).tolist()
    clean = Problem(1, offsets[-1], 36, "f32", offsets=offsets, reverse=reverse, seed=12)
    fwd0, bwd0 = clean.run()
    bad = Problem(1, offsets[-1], 36, "f32", offsets=offsets, reverse=reverse, seed=12)
    hit = (1, 4)
    for q in hit:
        lo, hi = offsets[q], offsets[q + 1]
        bad.x[0, lo + 3] = float("nan")
        bad.r[0, hi - 1] = float("nan")
        bad.dy[0, lo] = float("inf")
        bad.i[0, lo + 7] = float("nan")
        bad.h0[q] = float("inf")
        bad.dh_last[q] = float("nan")
    fwd1, bwd1 = bad.run()
    keep = torch.ones(offsets[-1], dtype=torch.bool)
    for q in hit:
        keep[offsets[q]:offsets[q + 1]] = False
    keep = keep.to(DEV)
    for a, b in ((fwd0.y, fwd1.y), (bwd0.dx, bwd1.dx), (bwd0.dr, bwd1.dr), (bwd0.di, bwd1.di)):
        assert torch.equal(a[0][keep], b[0][keep])
    others = [q for q in range(len(lens)) if q not in hit]
    assert torch.equal(fwd0.h_last[others], fwd1.h_last[others]) and torch.equal(bwd0.dh0[others], bwd1.dh0[others])
    assert bool(fwd1.y[0, offsets[2] - 1 if not reverse else offsets[1]].isnan().all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [33, 64])
@pytest.mark.parametrize("reverse", [False, True])
def test_non_finite_values_stay_in_their_sequence(io, d, reverse):
    """A NaN input makes every later output NaN, a NaN gradient every earlier one, an infinite initial state every
    output: also where the product of the decays between them is far below the smallest number."""
    offsets = [0, 50, 50 + 3000, 50 + 3000 + 70]
    p = Problem(1, offsets[-1], d, io, offsets=offsets, reverse=reverse, seed=21)
    p.lam[:] = 1.0   # decays of about e^-5 a token
    order = range(offsets[2] - 1, offsets[1] - 1, -1) if reverse else range(offsets[1], offsets[2])
    tokens = torch.tensor(list(order), device=DEV)
    p.x[0, tokens[700], 3] = float("nan")
    p.dy[0, tokens[2200], 5] = float("nan")
    p.h0[1, 7] = float("inf")
    fwd, bwd = p.run()
    y, dx = fwd.y[0], bwd.dx[0]
    lost = torch.zeros_like(y, dtype=torch.bool)
    lost[tokens[700:], 3] = True
    lost[tokens, 7] = True
    assert torch.equal(~y.isfinite(), lost)
    assert torch.equal(~fwd.h_last.isfinite().cpu(), torch.tensor([[q == 1 and c in (3, 7) for c in range(d)] for q in range(3)]))
    lost[:] = False
    lost[tokens[:2201], 5] = True
    lost[tokens[700], 3] = False   # dx does not depend on x
    assert torch.equal(dx.isnan(), lost)
    assert bool(bwd.dh0[1, 5].isnan()) and bool(bwd.dh0[[0, 2]].isfinite().all())


def test_extreme_gates_and_rates():
    """Gates at both ends, infinite among them, and decay rates from 0 (lam -> -inf) to very fast."""
    p = Problem(2, 90, 24, "f32", seed=13)
    vals = torch.tensor([-float("inf"), -200.0, -60.0, -20.0, 20.0, 60.0, 200.0, float("inf")], device=DEV)
    idx = torch.arange(2 * 90 * 24, device=DEV).view(2, 90, 24)
    p.r[:] = torch.where(idx % 5 == 0, vals[idx // 5 % 8], p.r)
    p.i[:] = torch.where(idx % 7 == 0, vals[idx // 7 % 8], p.i)
    p.lam[:] = torch.tensor([-90.0, -60.0, -30.0, -10.0, -5.0, 0.0, 5.0, 30.0], device=DEV).repeat(3)
    finite = Problem(2, 90, 24, "f32", seed=13)
    for name in ("x", "dy", "h0", "dh_last", "lam"):
        setattr(finite, name, getattr(p, name))
    finite.r, finite.i = p.r.clamp(-1e4, 1e4), p.i.clamp(-1e4, 1e4)
    with np.errstate(all="ignore"):
        want = finite.reference()
    # gates and rates below 2^-126 are held there or flushed to 0: m = sqrt(-2 u) is then off by up to
    # sqrt(2 c 2^-126) = 4e-19, times inputs and gradients of a few units
    fwd, bwd = p.run()
    for name, t in (("y", fwd.y), ("h_last", fwd.h_last), ("dx", bwd.dx), ("dr", bwd.dr), ("di", bwd.di),
                    ("dlam", bwd.dlam), ("dh0", bwd.dh0)):
        assert bool(t.isfinite().all()), name
        ref.check(t, (want[name][0], want[name][1] + 1e-16), False, name)


def test_gradient_against_differences():
    """The kernels' gradients in random directions against central differences of the 64-bit loss
    sum(y dy) + sum(h_last dh_last). With step 1e-5 the difference's own error (third derivatives of
    order 1e2, rounding 1e-16 / 1e-5) stays under 1e-7 of the loss's terms."""
    p = Problem(2, 70, 9, "f32", seed=14)
    _, bwd = p.run()
    rng = np.random.default_rng(15)
    base = {k: f64(getattr(p, k)) for k in ("x", "r", "i", "lam", "h0")}
    base = {k: v.reshape(-1, 9) if k in "xri" else v for k, v in base.items()}
    dy, dh = f64(p.dy).reshape(-1, 9), f64(p.dh_last)

    def loss(v):
        o = ref.gated(v["x"], v["r"], v["i"], v["lam"], C, p.bounds, v["h0"])
        return (o["y"][0] * dy).sum() + (o["h_last"][0] * dh).sum()

    bound = p.reference()
    for name, got in (("x", bwd.dx), ("r", bwd.dr), ("i", bwd.di), ("lam", bwd.dlam), ("h0", bwd.dh0)):
        v = rng.standard_normal(base[name].shape)
        h = 1e-5
        up, dn = dict(base), dict(base)
        up[name], dn[name] = base[name] + h * v, base[name] - h * v
        slope = (loss(up) - loss(dn)) / (2 * h)
        mine = (f64(got).reshape(v.shape) * v).sum()
        tol = (bound["d" + name][1] * np.abs(v)).sum() + 1e-7 * np.abs(dy).sum()
        assert abs(mine - slope) <= tol, (name, mine, slope, tol)


def test_same_bits_every_run():
    p = Problem(4, 777, 132, "bf16", seed=16)
    f0, b0 = p.run()
    first = [t.clone() for t in (f0.y, f0.h_last, b0.dx, b0.dr, b0.di, b0.dlam, b0.dh0)]
    for _ in range(4):
        f, b = p.run()
        for t, u in zip(first, (f.y, f.h_last, b.dx, b.dr, b.di, b.dlam, b.dh0)):
            assert torch.equal(t, u)


def test_optional_outputs():
    """No dy, a gradient of h_last only: only the given gradients are formed."""
    p = Problem(2, 65, 20, "f32", seed=17)
    fwd = PreparedGated(p.inputs(), None, None, None, save_states=True)
    fwd()
    only_last = PreparedGatedGrad(fwd, None, p.dh_last)
    only_last()
    rows = [f64(t).reshape(-1, 20) for t in (p.x, p.r, p.i)]
    want = ref.gated(*rows, f64(p.lam), C, p.bounds, f64(p.h0), False, np.zeros_like(rows[0]), f64(p.dh_last), True)
    for k in ("dx", "dr", "di", "dlam", "dh0"):
        ref.check(getattr(only_last, k), want[k], False, k)


def test_offsets_past_32_bits():
    """2.2e9 channels of bf16 (rows past 2^32 bytes): a sample of the channels against 64 bits."""
    d, length, nseq = 1536, 512, 2800
    assert d * length * nseq > 2 ** 31
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x, r, i = (torch.randn((nseq, length, d), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    lam = tensor(rates(np.random.default_rng(1), d))
    fwd = PreparedGated(x, r, i, lam, C, save_states=True)
    fwd()
    bwd = PreparedGatedGrad(fwd, x)
    bwd()
    for q in (0, 1399, nseq - 1):
        for c in (0, 700, d - 1):
            rows = [f64(t[q, :, c:c + 1]) for t in (x, r, i)]
            want = ref.gated(*rows, f64(lam[c:c + 1]), C, [(0, length)], None, False, rows[0], None, True)
            for name, t in (("y", fwd.y), ("dx", bwd.dx), ("dr", bwd.dr), ("di", bwd.di)):
                ref.check(t[q, :, c:c + 1], want[name], True, f"{name} {q} {c}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,d", [(1, 1), (1, 768), (3, 77), (70, 64), (5, 130), (9, 36)])
def test_step(batch, d, io):
    rng = np.random.default_rng(batch + d)
    x, r, i = (tensor(rng.standard_normal((batch, d)), io) for _ in range(3))
    lam = tensor(rates(rng, d))
    pool = tensor(rng.standard_normal((2 * batch + 1, d)))
    before = pool.clone()
    perm = rng.permutation(2 * batch + 1).astype(np.int32)
    src, dst = (torch.from_numpy(v.copy()).to(DEV) for v in (perm[:batch], perm[batch:2 * batch]))
    y = binding.gated_step(x, r, i, lam, pool, C, src, dst)
    bounds = [(k, k + 1) for k in range(batch)]
    want = ref.gated(f64(x), f64(r), f64(i), f64(lam), C, bounds, f64(before[src.long()]))
    ref.check(y, want["y"], io == "bf16", "y")
    ref.check(pool[dst.long()], want["h_last"], False, "state")
    rest = torch.ones(2 * batch + 1, dtype=torch.bool, device=DEV)
    rest[dst.long()] = False
    assert torch.equal(pool[rest], before[rest])


def test_step_skips_rows_outside_the_pool():
    rng = np.random.default_rng(2)
    x, r, i = (tensor(rng.standard_normal((6, 40))) for _ in range(3))
    lam = tensor(rates(rng, 40))
    pool = tensor(rng.standard_normal((4, 40)))
    before = pool.clone()
    src = torch.tensor([0, -1, 4, 1, 2, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    dst = torch.tensor([0, 1, 2, 7, 3, 0], dtype=torch.int32, device=DEV)
    y = binding.gated_step(x, r, i, lam, pool, C, src, dst)
    want = ref.gated(f64(x), f64(r), f64(i), f64(lam), C, [(k, k + 1) for k in range(6)],
                     f64(before[torch.tensor([0, 0, 0, 0, 2, 0])]))
    for row in (0, 4):
        ref.check(y[row], (want["y"][0][row], want["y"][1][row]))
    assert bool((y[[1, 2, 3, 5]] == 0).all())
    assert torch.equal(pool[[1, 2]], before[[1, 2]])
    ref.check(pool[0], (want["h_last"][0][0], want["h_last"][1][0]))
    ref.check(pool[3], (want["h_last"][0][4], want["h_last"][1][4]))


def test_steps_continue_a_prefill():
    """A prompt through the whole-sequence form, then token by token in place: the same outputs as
    one long sequence."""
    p = Problem(3, 150, 52, "f32", seed=21)
    cut = 101
    _, state = binding.gated_fwd(*(t[:, :cut].contiguous() for t in (p.x, p.r, p.i)), p.lam, C, p.h0)
    ys = []
    for t in range(cut, 150):   # strided rows: token t of every stream
        ys.append(binding.gated_step(p.x[:, t], p.r[:, t], p.i[:, t], p.lam, state, C))
    want = p.reference(False)
    y = want["y"][0].reshape(3, 150, 52)[:, cut:]
    e = want["y"][1].reshape(3, 150, 52)[:, cut:]
    ref.check(torch.stack(ys, 1), (y, e))
    ref.check(state, want["h_last"])


def test_no_tokens():
    x = torch.empty((3, 0, 16), device=DEV)
    lam = torch.zeros(16, device=DEV)
    h0 = torch.randn(3, 16, device=DEV)
    y, h = binding.gated_fwd(x, x, x, lam, C, h0)
    assert y.shape == (3, 0, 16) and torch.equal(h, h0)
    fwd = PreparedGated(x, x, x, lam, C, h0, save_states=True)
    fwd()
    bwd = PreparedGatedGrad(fwd, x, h0)
    bwd()
    assert torch.equal(bwd.dh0, h0) and bool((bwd.dlam == 0).all())
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    x = torch.empty((1, 0, 16), device=DEV)
    y, h = binding.gated_fwd(x, x, x, lam, C, offsets=off)
    assert h.shape == (4, 16) and bool((h == 0).all())


def test_in_a_graph_and_on_another_stream():
    p = Problem(2, 513, 70, "bf16", seed=22)
    f0, b0 = p.run()
    keep = [t.clone() for t in (f0.y, f0.h_last, b0.dx, b0.dr, b0.di, b0.dlam, b0.dh0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f1, b1 = p.run()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(keep, (f1.y, f1.h_last, b1.dx, b1.dr, b1.di, b1.dlam, b1.dh0)):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream().cuda_stream
        f2 = PreparedGated(p.inputs(), None, None, None, save_states=True, stream=s)
        f2()
        b2 = PreparedGatedGrad(f2, p.dy, p.dh_last, stream=s)
        b2()
    outs = (f2.y, f2.h_last, b2.dx, b2.dr, b2.di, b2.dlam, b2.dh0)
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(keep, outs):
            assert torch.equal(a, b)
        f0()
        b0()
    assert binding.wait_timeouts() == 0


def test_refusals():
    p = Problem(2, 32, 16, "f32", seed=23)
    x, r, i, lam = p.x, p.r, p.i, p.lam
    with pytest.raises(ValueError):
        PreparedGated(x[0], r, i, lam)
    with pytest.raises(ValueError):
        PreparedGated(x, r[:, :31], i, lam)
    with pytest.raises(ValueError):
        PreparedGated(x, r.bfloat16(), i, lam)
    with pytest.raises(ValueError):
        PreparedGated(x.transpose(1, 2).contiguous().transpose(1, 2), r, i, lam)
    with pytest.raises(ValueError):
        PreparedGated(x[:, :1].expand(2, 32, 16), r, i, lam)
    with pytest.raises(ValueError):
        PreparedGated(x, r, i, lam.double())
    with pytest.raises(ValueError):
        PreparedGated(x, r, i, lam, h0=torch.zeros(3, 16, device=DEV))
    with pytest.raises(ValueError):
        PreparedGated(x, r, i, lam, seg_len=8, offsets=torch.tensor([0, 64], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        PreparedGated(x, r, i, lam, offsets=torch.tensor([0, 64], device=DEV))
    with pytest.raises(TypeError):
        PreparedGated(x.half(), r.half(), i.half(), lam)
    with pytest.raises(binding.VimscanError) as e:
        PreparedGated(x, r, i, lam, seg_len=5)
    assert e.value.status == -3
    for c in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(binding.VimscanError) as e:
            binding.gated_fwd(x, r, i, lam, c=c)
        assert e.value.status == -13
    with pytest.raises(binding.VimscanError) as e:
        binding.gated_fwd(x, r, i, lam, out=x)
    assert e.value.status == -6
    fwd = PreparedGated(x, r, i, lam)
    fwd()
    with pytest.raises(ValueError):
        PreparedGatedGrad(fwd, p.dy)
    with pytest.raises(ValueError):
        PreparedGatedStep(x[:, 0], r[:, 0], i[:, 0], lam, torch.zeros(2, 17, device=DEV))
    with pytest.raises(binding.VimscanError) as e:
        state = torch.zeros(2, 16, device=DEV)
        PreparedGatedStep(x[:, 0], r[:, 0], i[:, 0], lam, state, out=state)()
    assert e.value.status == -6


@pytest.mark.parametrize("seqlen,seg", [(2, 0), (3, 0), (7, 0), (1, 0), (130, 13), (66, 1), (66, 2)])
@pytest.mark.parametrize("d", [68, 5])
def test_nothing_is_written_past_the_last_sequence(seqlen, seg, d):
    """Streams that end inside a thread's positions: rows around y and h_last stay as they are."""
    p = Problem(3, seqlen, d, "f32", seg_len=seg, seed=seqlen)
    nseq = len(p.bounds)
    hbuf = torch.full((nseq + 8, d), 7.0, device=DEV)
    ybuf = torch.full((3 * seqlen + 200, d), 7.0, device=DEV)
    y, h = ybuf[100:100 + 3 * seqlen].view(3, seqlen, d), hbuf[4:4 + nseq]
    PreparedGated(p.inputs(), None, None, None, out=y, h_last=h)()
    want = p.reference(False)
    ref.check(y, want["y"])
    ref.check(h, want["h_last"])
    assert bool((hbuf[:4] == 7).all()) and bool((hbuf[4 + nseq:] == 7).all())
    assert bool((ybuf[:100] == 7).all()) and bool((ybuf[100 + 3 * seqlen:] == 7).all())


def test_graph_replays_see_new_inputs():
    """A captured forward and backward pass over a sequence of many workgroups, replayed on inputs that
    change between the replays: the states handed over are this replay's, not the last one's."""
    p = Problem(1, 20000, 64, "f32", seed=31)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream().cuda_stream
        f = PreparedGated(p.inputs(), None, None, None, save_states=True, stream=s)
        f()
        b = PreparedGatedGrad(f, p.dy, p.dh_last, stream=s)
        b()
    for k in range(4):
        for t in (p.x, p.r, p.i, p.dy, p.h0):
            t.copy_(torch.randn_like(t))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        f1, b1 = p.run()
        for a, c in zip((f.y, f.h_last, b.dx, b.dr, b.di, b.dlam, b.dh0),
                        (f1.y, f1.h_last, b1.dx, b1.dr, b1.di, b1.dlam, b1.dh0)):
            assert torch.equal(a, c), k
    assert binding.wait_timeouts() == 0


def test_a_workspace_of_arbitrary_contents():
    """The hand-over needs no cleared workspace: zeros, ones, equal words and another call's leftovers."""
    p = Problem(1, 3000, 66, "f32", seed=32)
    f0, b0 = p.run()
    need = max(f0.plan["workspace_bytes"], b0.plan["workspace_bytes"])
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    other = Problem(1, 3000, 66, "f32", seed=33)
    for fill in (0, 255, 63, "other"):
        if fill == "other":
            PreparedGated(other.inputs(), None, None, None, workspace=ws)()
        else:
            ws.fill_(fill)
        f = PreparedGated(p.inputs(), None, None, None, save_states=True, workspace=ws)
        f()
        assert torch.equal(f.y, f0.y) and torch.equal(f.h_last, f0.h_last)
        if fill != "other":
            ws.fill_(fill)
        b = PreparedGatedGrad(f, p.dy, p.dh_last, workspace=ws)
        b()
        for a, c in ((b.dx, b0.dx), (b.dr, b0.dr), (b.di, b0.di), (b.dlam, b0.dlam), (b.dh0, b0.dh0)):
            assert torch.equal(a, c)
