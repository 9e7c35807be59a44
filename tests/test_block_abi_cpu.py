"""The C ABI of the gated recurrence and the block norm without a GPU: every bad argument is refused
with the documented status before any HIP call (each call here fails validation or is empty)."""
import ctypes
import os

import pytest

from bidirectional_selective_scan_amd import binding, block

NULL, SHAPE, SEGLEN, DTYPE, ALIGN, ALIAS, WORKSPACE, CHUNK, FLAGS, PARAM = (-1, -2, -3, -4, -5, -6, -7, -9, -10, -13)
BASE = 1 << 40   # addresses that no call here dereferences
GAP = 1 << 32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return binding.load_library()


def launch(batch=2, seqlen=100, d=48, d_state=1, io=1, flags=0, chunk=0, ws=None, ws_bytes=0):
    l = binding.make_launch(batch, seqlen, d, d_state, io, chunk)
    l.flags, l.workspace, l.workspace_bytes = flags, ws, ws_bytes
    return l


def addr(k):
    return BASE + k * GAP


def gated(d=48, **kw):
    f = dict(x=addr(0), r=addr(1), i=addr(2), ld_x=d, ld_r=d, ld_i=d, lam=addr(3), h0=addr(4), offsets=None, nseq=0, c=8.0)
    f.update(kw)
    return block._Gated(**f)


def fwd(lib, g, l, y=addr(5), h=addr(6), st=addr(7), seg=0):
    return lib.vimscan_gated_fwd(ctypes.byref(g) if g else None, seg, y, h, st, ctypes.byref(l) if l else None)


def grad(d=48, **kw):
    f = dict(dy=addr(8), dh_last=addr(9), states=addr(10), dx=addr(11), dr=addr(12), di=addr(13), ld_dy=d, ld_dx=d,
             ld_dr=d, ld_di=d, dlam=addr(14), dh0=addr(15))
    f.update(kw)
    return block._GatedGrad(**f)


def bwd(lib, g, gr, l, seg=0):
    return lib.vimscan_gated_bwd(ctypes.byref(g), seg, ctypes.byref(gr) if gr else None, ctypes.byref(l))


def test_status_text_of_the_new_code(lib):
    assert "bad parameter" in binding.status_string(PARAM)
    assert binding.status_string(-14) == "unknown status"


def test_gated_forward_refusals(lib):
    assert fwd(lib, None, launch()) == NULL and fwd(lib, gated(), None) == NULL
    for l in (launch(batch=-1), launch(seqlen=-1), launch(d=-1), launch(d_state=16), launch(d=1 << 22),
              launch(batch=1 << 16, seqlen=1 << 15), launch(batch=1 << 40)):
        assert fwd(lib, gated(d=1 << 23), l) == SHAPE
    assert fwd(lib, gated(), launch(io=2)) == DTYPE
    assert fwd(lib, gated(), launch(chunk=16)) == CHUNK
    for flag in (1, 2, 4, 16, 32):
        assert fwd(lib, gated(), launch(flags=flag)) == FLAGS
    assert fwd(lib, gated(), launch(), seg=-1) == SEGLEN and fwd(lib, gated(), launch(), seg=33) == SEGLEN
    assert fwd(lib, gated(offsets=addr(9), nseq=3), launch(), seg=50) == PARAM
    assert fwd(lib, gated(offsets=addr(9), nseq=-1), launch()) == SHAPE
    assert fwd(lib, gated(offsets=addr(9), nseq=0), launch()) == SHAPE
    for c in (0.0, -1.0, float("inf"), float("nan")):
        assert fwd(lib, gated(c=c), launch()) == PARAM
    for kw in (dict(ld_x=47), dict(ld_r=0), dict(ld_i=-48), dict(ld_x=1 << 24)):
        assert fwd(lib, gated(**kw), launch()) == PARAM
    for kw in (dict(x=None), dict(r=None), dict(i=None), dict(lam=None)):
        assert fwd(lib, gated(**kw), launch()) == NULL
    assert fwd(lib, gated(), launch(), y=None) == NULL
    for kw in (dict(x=addr(0) + 1), dict(lam=addr(3) + 2), dict(h0=addr(4) + 1), dict(offsets=addr(9) + 2, nseq=1)):
        assert fwd(lib, gated(**kw), launch()) == ALIGN
    assert fwd(lib, gated(), launch(io=0), y=addr(5) + 2) == ALIGN
    assert fwd(lib, gated(), launch(), h=addr(6) + 2) == ALIGN
    n = 200 * 48 * 2
    for y in (addr(0), addr(1) + n - 2, addr(2) - n + 2, addr(3), addr(4)):
        assert fwd(lib, gated(), launch(), y=y) == ALIAS
    assert fwd(lib, gated(), launch(), h=addr(5)) == ALIAS and fwd(lib, gated(), launch(), st=addr(6)) == ALIAS
    # the extent of strided rows counts, to the last row's end
    assert fwd(lib, gated(ld_x=100), launch(), y=addr(0) + (199 * 100 + 47) * 2) == ALIAS


def test_gated_backward_refusals(lib):
    big = dict(ws=addr(20), ws_bytes=1 << 30)
    assert bwd(lib, gated(), None, launch(**big)) == NULL
    assert bwd(lib, gated(), grad(dx=None), launch(**big)) == NULL
    assert bwd(lib, gated(), grad(states=None), launch(**big)) == NULL
    for kw in (dict(ld_dx=47), dict(ld_dy=1), dict(ld_dr=-1), dict(ld_di=1 << 24)):
        assert bwd(lib, gated(), grad(**kw), launch(**big)) == PARAM
    for kw in (dict(dx=addr(11) + 1), dict(dlam=addr(14) + 2), dict(dh0=addr(15) + 2), dict(states=addr(10) + 2)):
        assert bwd(lib, gated(), grad(**kw), launch(**big)) == ALIGN
    for kw in (dict(dx=addr(0)), dict(dr=addr(8)), dict(di=addr(10)), dict(dlam=addr(3)), dict(dh0=addr(4)),
               dict(dh0=addr(14)), dict(dr=addr(11)), dict(dlam=addr(13))):
        assert bwd(lib, gated(), grad(**kw), launch(**big)) == ALIAS
    need = binding.gated_info(2, 100, 48, backward=True)["workspace_bytes"]
    assert need > 0
    assert bwd(lib, gated(), grad(), launch()) == WORKSPACE
    assert bwd(lib, gated(), grad(), launch(ws=addr(20), ws_bytes=need - 1)) == WORKSPACE
    assert bwd(lib, gated(), grad(), launch(ws=addr(20) + 8, ws_bytes=need)) == ALIGN
    for k in (0, 8, 11, 14):
        assert bwd(lib, gated(), grad(), launch(ws=addr(k), ws_bytes=need)) == ALIAS


def test_gated_step_refusals(lib):
    def step(g, l, state=addr(5), slots=10, si=addr(6), so=addr(7), y=addr(8)):
        return lib.vimscan_gated_step(ctypes.byref(g) if g else None, state, slots, si, so, y,
                                      ctypes.byref(l) if l else None)
    one = dict(seqlen=1)
    assert step(None, launch(**one)) == NULL and step(gated(), None) == NULL
    assert step(gated(), launch(seqlen=2)) == SHAPE and step(gated(), launch(**one), slots=-1) == SHAPE
    assert step(gated(), launch(flags=8, **one)) == FLAGS
    assert step(gated(c=0.0), launch(**one)) == PARAM and step(gated(ld_r=3), launch(**one)) == PARAM
    assert step(gated(x=None), launch(**one)) == NULL and step(gated(), launch(**one), y=None) == NULL
    assert step(gated(), launch(**one), state=None) == NULL
    assert step(gated(), launch(**one), state=addr(5) + 2) == ALIGN and step(gated(), launch(**one), si=addr(6) + 2) == ALIGN
    assert step(gated(), launch(**one), y=addr(0)) == ALIAS and step(gated(), launch(**one), y=addr(5)) == ALIAS
    assert step(gated(), launch(**one), state=addr(6)) == ALIAS
    assert step(gated(), launch(batch=0, **one)) == 0


def norm(d=48, **kw):
    f = dict(x=addr(0), z=addr(1), ld_x=d, ld_z=d, w_post=addr(2), residual=addr(3), gamma=addr(4), w_pre=addr(5),
             eps=1e-5, res_dtype=0)
    f.update(kw)
    return block._Norm(**f)


def norm_fwd(lib, n, l, s=addr(6), o=addr(7)):
    return lib.vimscan_norm_fwd(ctypes.byref(n) if n else None, s, o, ctypes.byref(l) if l else None)


def test_norm_forward_refusals(lib):
    ok = dict(d_state=0)
    assert norm_fwd(lib, None, launch(**ok)) == NULL and norm_fwd(lib, norm(), None) == NULL
    assert norm_fwd(lib, norm(), launch()) == SHAPE
    assert norm_fwd(lib, norm(d=32769), launch(d=32769, **ok)) == SHAPE
    assert norm_fwd(lib, norm(), launch(chunk=1, **ok)) == CHUNK
    assert norm_fwd(lib, norm(), launch(flags=8, **ok)) == FLAGS
    assert norm_fwd(lib, norm(res_dtype=2), launch(**ok)) == DTYPE
    assert norm_fwd(lib, norm(res_dtype=1), launch(io=0, **ok)) == DTYPE
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert norm_fwd(lib, norm(eps=eps), launch(**ok)) == PARAM
    assert norm_fwd(lib, norm(ld_x=47), launch(**ok)) == PARAM and norm_fwd(lib, norm(ld_z=1), launch(**ok)) == PARAM
    assert norm_fwd(lib, norm(x=None), launch(**ok)) == NULL
    for kw in (dict(z=None), dict(w_post=None)):
        assert norm_fwd(lib, norm(**kw), launch(flags=16, **ok)) == PARAM
    assert norm_fwd(lib, norm(w_pre=None), launch(**ok)) == PARAM and norm_fwd(lib, norm(), launch(**ok), o=None) == PARAM
    assert norm_fwd(lib, norm(w_pre=None), launch(**ok), s=None, o=None) == NULL
    for kw in (dict(x=addr(0) + 1), dict(residual=addr(3) + 2), dict(gamma=addr(4) + 1)):
        assert norm_fwd(lib, norm(**kw), launch(**ok)) == ALIGN
    for k in (0, 1, 2, 4, 5):
        assert norm_fwd(lib, norm(), launch(**ok), s=addr(k)) == ALIAS
    assert norm_fwd(lib, norm(), launch(**ok), s=addr(3) + 4) == ALIAS     # only the residual itself may be the sum
    assert norm_fwd(lib, norm(), launch(**ok), o=addr(3)) == ALIAS and norm_fwd(lib, norm(), launch(**ok), o=addr(6)) == ALIAS
    assert norm_fwd(lib, norm(x=None), launch(batch=0, **ok)) == 0


def test_norm_backward_refusals(lib):
    def run(n, ws=addr(20), nbytes=1 << 30, flags=0, batch=2, **kw):
        f = dict(dsum=addr(8), dn=addr(9), dx=addr(10), dz=addr(11), ld_dx=48, ld_dz=48, dresidual=addr(12),
                 dw_post=addr(13), dgamma=addr(14), dw_pre=addr(15))
        f.update(kw)
        g = block._NormGrad(**f)
        l = launch(batch=batch, d_state=0, ws=ws, ws_bytes=nbytes, flags=flags)
        return lib.vimscan_norm_bwd(ctypes.byref(n), ctypes.byref(g), ctypes.byref(l))
    assert run(norm(w_pre=None)) == PARAM and run(norm(w_pre=None), dn=None) == PARAM
    assert run(norm(z=None)) == PARAM and run(norm(residual=None)) == PARAM
    assert run(norm(gamma=None)) == PARAM and run(norm(w_post=None)) == PARAM
    assert run(norm(), ld_dx=47) == PARAM and run(norm(), ld_dz=0) == PARAM
    assert run(norm(), dx=addr(10) + 1) == ALIGN and run(norm(), dw_pre=addr(15) + 2) == ALIGN
    for kw in (dict(dx=addr(0)), dict(dz=addr(10)), dict(dresidual=addr(3)), dict(dresidual=addr(8) + 4),
               dict(dw_post=addr(2)), dict(dgamma=addr(13)), dict(dx=addr(8)), dict(dw_pre=addr(12))):
        assert run(norm(), **kw) == ALIAS
    need = binding.norm_info(200, 48, backward=True)["workspace_bytes"]
    assert run(norm(), ws=None) == WORKSPACE and run(norm(), nbytes=need - 1) == WORKSPACE
    assert run(norm(), ws=addr(20) + 4) == ALIGN and run(norm(), ws=addr(3)) == ALIAS


def test_plans(lib):
    for backward in (False, True):
        p = binding.gated_info(8, 1025, 768, backward=backward)
        assert (p["sequences"], p["seq_tokens"]) == (8, 1025) and p["workgroups"] > 0
        assert binding.gated_info(1, 13056, 1536, seg_len=51, backward=backward)["sequences"] == 256
        assert binding.gated_info(1, 500, 64, nseq=7, backward=backward)["sequences"] == 7
        assert binding.gated_info(2, 100, 0, backward=backward)["workgroups"] == 0
        assert binding.norm_info(0, 64, backward=backward)["workgroups"] == 0
        assert binding.norm_info(100, 768, backward=backward)["sequences"] == 100
    with pytest.raises(binding.VimscanError):
        binding.gated_info(1 << 30, 1, 1 << 21)
    with pytest.raises(binding.VimscanError):
        binding.norm_info(10, 40000)
    plan = binding._Plan()
    assert lib.vimscan_norm_plan(None, 0, ctypes.byref(plan)) == NULL
    assert lib.vimscan_gated_plan(ctypes.byref(launch()), 0, 0, 0, 0, None) == NULL
