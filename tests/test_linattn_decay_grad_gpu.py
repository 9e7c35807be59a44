"""The decays' gradient of linear attention keeps to its definition, dg_t = exp(g_t) <S_{t-1}, D_t>: what a token does not
depend on reaches it over at most 127 tokens and not past a reset. Against a 64-bit form with bounds (linattn_bounds)."""
import numpy as np
import pytest
import torch

import block_reference
import linattn_bounds
from bidirectional_selective_scan_amd import binding
from bidirectional_selective_scan_amd.binding import PreparedLinAttn, PreparedLinAttnGrad

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("dq", "dk", "dv", "dg", "dh0")


class Call:
    """A call's tensors: shape (sequences, tokens), or lengths of packed sequences."""

    def __init__(self, shape, H, G, dk, dv, io, decay="token", reverse=False, state=True, seed=0, strength=1.0):
        rng = np.random.default_rng(seed)
        self.offsets = None
        if isinstance(shape, list):
            off = np.concatenate([[0], np.cumsum(shape)]).astype(int)
            self.bounds = list(zip(off[:-1], off[1:]))
            self.offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
            shape = (1, int(off[-1]))
        else:
            self.bounds = [(i * shape[1], (i + 1) * shape[1]) for i in range(shape[0])]
        self.n, self.H, self.bf16, self.reverse = shape[0] * shape[1], H, io == "bf16", reverse

        def rows(h, d):
            return torch.from_numpy(rng.standard_normal((*shape, h, d)).astype(np.float32)).to(DEV).to(DT[io])

        self.q, self.k, self.v, self.dy = rows(G, dk), rows(G, dk), rows(H, dv), rows(H, dv)
        lead = (*shape, H) if decay == "token" else (H,)
        self.g = torch.from_numpy(-strength * np.abs(rng.standard_normal(lead)).astype(np.float32)).to(DEV)
        st = (len(self.bounds), H, dk, dv)
        self.h0, self.dh = (torch.from_numpy(rng.standard_normal(st).astype(np.float32)).to(DEV) if state else None for _ in range(2))

    def run(self, decays=True):
        call = PreparedLinAttn(self.q, self.k, self.v, self.g, None, self.h0, 0, self.offsets, self.reverse)
        call()
        grad = PreparedLinAttnGrad(call, self.dy, self.dh, decays=decays)
        grad()
        self.plan = call.plan
        out = dict(y=call.y, h_last=call.h_last, dq=grad.dq, dk=grad.dk, dv=grad.dv)
        if decays:
            out["dg"] = grad.dlog_decay
        if self.h0 is not None:
            out["dh0"] = grad.dh0
        return {k: t.double().cpu().numpy() for k, t in out.items()}

    def want(self):
        def f(t):
            return None if t is None else t.double().cpu().numpy()

        def flat(t):
            return f(t).reshape(self.n, *t.shape[2:])

        g = f(self.g) if self.g.dim() == 1 else flat(self.g)
        return linattn_bounds.linattn(flat(self.q), flat(self.k), flat(self.v), g, float(np.float32(self.q.shape[-1] ** -0.5)),
                                      self.bounds, f(self.h0), self.reverse, flat(self.dy), f(self.dh), self.bf16)

    def check(self, names=None, decays=True):
        got, want = self.run(decays), self.want()
        for name in names or got:
            check(got[name], want[name], self.bf16 and name in ("y", "dq", "dk", "dv"), name)


def check(got, want, bf16, name, where=None):
    val, err = want
    got = got.reshape(val.shape)
    bound = err + (block_reference.BF16_HALF * np.abs(val) if bf16 else 0.0)
    bad = ~(np.abs(got - val) <= bound)
    if where is not None:
        bad &= where
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(got - val)[bad])), np.argwhere(bad)[:3].tolist())


def copies(p, n, H, G, dk, dv):
    """A call of n sequences, all but the second copies of the first, and the call of those two alone."""
    for t in (p.q, p.k, p.v, p.dy, p.g):
        t[2:] = t[0]
    two = Call((2, p.q.shape[1]), H, G, dk, dv, "bf16" if p.bf16 else "f32", reverse=p.reverse, state=False)
    two.q, two.k, two.v, two.dy, two.g = (t[:2] for t in (p.q, p.k, p.v, p.dy, p.g))
    return two


def check_copies(p, two, n):
    got = p.run()
    assert p.plan["kernels"] == 1      # (whole sequences)
    want = two.want()
    for name in ("y", "dq", "dk", "dv", "dg"):
        full = got[name].reshape(n, -1)
        check(full[:2], want[name], p.bf16 and name != "dg", name)
        assert (full[2:] == full[0]).all()
    return got


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("factor", [10.0, 30.0])
@pytest.mark.parametrize("what", [float("-inf"), torch.finfo(torch.float32).min, -110.0])
def test_larger_tokens_behind_a_reset(io, reverse, factor, what):
    """197 tokens, a reset at 100, everything from it on larger: nothing of that is left in the tokens before it."""
    p = Call((400, 197), 2, 2, 64, 64, io, reverse=reverse, state=False, seed=1)
    at = 196 - 100 if reverse else 100
    behind = slice(0, at + 1) if reverse else slice(at, 197)
    for t in (p.q, p.k, p.v, p.dy):
        t[:, behind] *= factor
    p.g[:, at] = what
    got = check_copies(p, copies(p, 400, 2, 2, 64, 64), 400)
    assert (got["dg"].reshape(400, 197, 2)[:, at] == 0).all()


def ramp(p):
    """Sizes that grow 4-fold every 40 tokens, four times over."""
    size = torch.exp2(torch.arange(p.n, device=DEV) // 40 % 5 * 2.0).view(*p.q.shape[:2], 1, 1)
    for t in (p.q, p.k, p.v, p.dy):
        t *= size.to(t.dtype)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("shape", [(2, 197), [60, 0, 333, 1, 100, 33]])
def test_larger_tokens_without_a_reset(io, reverse, shape):
    """Decays that are strong but not 0: the error keeps to a window of 128 tokens."""
    p = Call(shape, 2, 1, 24, 40, io, reverse=reverse, seed=2, strength=6.0)
    ramp(p)
    p.check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("length", [300, 128, 129, 256, 512])
def test_whole_sequences_of_several_windows(io, reverse, length):
    p = Call((400, length), 2, 1, 24, 40, io, reverse=reverse, state=False, seed=5, strength=6.0)
    ramp(p)
    check_copies(p, copies(p, 400, 2, 1, 24, 40), 400)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("seqs", [2, 400])
@pytest.mark.parametrize("which", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_how_far_nan_and_infinity_reach(io, reverse, seqs, which, bad):
    """Of the tokens of its sequence and head that a gradient does not depend on, a NaN or infinity may reach 31, the decays'
    gradient of 127."""
    length, H, u = 400, 3, 200        # u: walking position
    p = Call((seqs, length), H, H, 16, 24, io, reverse=reverse, seed=3, strength=0.1)
    clean = p.run()
    assert (p.plan["kernels"] == 3) == (seqs == 2)
    at = length - 1 - u if reverse else u
    getattr(p, which)[1, at, 1, 5] = bad
    got = p.run()
    walk = np.arange(length)[::-1] if reverse else np.arange(length)
    # the walking positions whose gradient depends on the token: [from, to)
    depends = {"q": dict(dq=(u, u + 1), dk=(0, u + 1), dv=(0, u + 1), dg=(0, u + 1)),
               "k": dict(dq=(u, length), dk=(u, u + 1), dv=(u, u + 1), dg=(u + 1, length)),
               "v": dict(dq=(u, length), dk=(u, u + 1), dv=(u, u + 1), dg=(u + 1, length)),
               "dy": dict(dq=(u, u + 1), dk=(0, u + 1), dv=(0, u + 1), dg=(0, u + 1))}[which]
    for name, (lo, hi) in depends.items():
        a, b = (t[name].reshape(seqs, length, H, -1) for t in (got, clean))
        reach = 127 if name == "dg" else 31
        free = np.ones((seqs, length, H, 1), dtype=bool)
        free[1, (walk >= lo - reach) & (walk < hi + reach), 1] = False
        assert free[1, :, 1].any()
        same = (a == b) | ~free
        assert same.all(), (name, int((~same).sum()))
        if name == "dg":     # and it is not lost
            assert not np.isfinite(a[1, (walk >= lo) & (walk < hi), 1]).any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("dk,dv,G", [(64, 64, 2), (16, 16, 1), (128, 64, 1), (40, 56, 2), (1, 3, 2), (128, 128, 2)])
def test_every_shape_of_the_state(io, decay, dk, dv, G):
    Call((3, 100), 2, G, dk, dv, io, decay, seed=dk).check()
    Call([33, 0, 400, 64, 1, 32], 2, G, dk, dv, io, decay, True, seed=dv).check()


def test_its_sums_alone_need_the_room_at_the_borders():
    """A backward pass without the decays' gradient is content with a smaller workspace."""
    p = Call((400, 200), 2, 2, 64, 64, "bf16", seed=4)
    call = PreparedLinAttn(p.q, p.k, p.v, p.g)
    full, none = PreparedLinAttnGrad(call, p.dy), PreparedLinAttnGrad(call, p.dy, decays=False)
    assert none.plan["workspace_bytes"] < full.plan["workspace_bytes"]
    full()
    none()
    assert torch.isfinite(none.dq.float()).all()
    with pytest.raises(binding.VimscanError) as e:
        small = torch.empty(none.plan["workspace_bytes"], dtype=torch.uint8, device=DEV)
        bad = PreparedLinAttnGrad(call, p.dy, workspace=torch.empty(full.plan["workspace_bytes"], dtype=torch.uint8, device=DEV))
        bad._launch.workspace, bad._launch.workspace_bytes = small.data_ptr(), small.numel()
        bad()
    assert e.value.status == -7
