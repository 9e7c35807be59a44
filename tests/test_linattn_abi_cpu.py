"""The C ABI of linear attention and the layer norm without a GPU: every bad argument is refused with the documented
status before any HIP call (each call here fails validation or is empty), and the plans keep their promises."""
import ctypes
import os

import pytest

from bidirectional_selective_scan_amd import attention, binding, block

NULL, SHAPE, SEGLEN, DTYPE, ALIGN, ALIAS, WORKSPACE, CHUNK, FLAGS, PARAM = (-1, -2, -3, -4, -5, -6, -7, -9, -10, -13)
BASE, GAP = 1 << 40, 1 << 32     # addresses that no call here dereferences


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return binding.load_library()


def addr(k):
    return BASE + k * GAP


def launch(batch=2, seqlen=100, d=96, d_state=16, io=1, flags=0, chunk=0, ws=None, ws_bytes=0):
    l = binding.make_launch(batch, seqlen, d, d_state, io, chunk)
    l.flags, l.workspace, l.workspace_bytes = flags, ws, ws_bytes
    return l


BIG = dict(ws=addr(40), ws_bytes=1 << 31)


def lin(**kw):
    f = dict(q=addr(0), k=addr(1), v=addr(2), ld_q=64, ld_k=64, ld_v=96, hs_q=16, hs_k=16, hs_v=24, log_decay=addr(3), ld_decay=4,
             h0=addr(4), offsets=None, nseq=0, heads=4, groups=4, scale=0.25)
    f.update(kw)
    return attention._LinAttn(**f)


def fwd(lib, p, l, y=addr(5), h=addr(6), seg=0):
    return lib.vimscan_linattn_fwd(ctypes.byref(p) if p else None, seg, y, h, ctypes.byref(l) if l else None)


def grad(**kw):
    f = dict(dy=addr(8), ld_dy=96, hs_dy=24, dh_last=addr(9), dq=addr(10), dk=addr(11), dv=addr(12), dlog_decay=addr(13),
             dh0=addr(14))
    f.update(kw)
    return attention._LinAttnGrad(**f)


def bwd(lib, p, g, l, seg=0):
    return lib.vimscan_linattn_bwd(ctypes.byref(p), seg, ctypes.byref(g) if g else None, ctypes.byref(l))


def test_forward_refusals(lib):
    assert fwd(lib, None, launch()) == NULL and fwd(lib, lin(), None) == NULL
    for l in (launch(batch=-1), launch(seqlen=-1), launch(d=-1), launch(d=0), launch(d=1 << 22), launch(d_state=0), launch(d_state=129),
              launch(d=4 * 129), launch(d=97), launch(batch=1 << 16, seqlen=1 << 15), launch(batch=1 << 40)):
        assert fwd(lib, lin(), l) == SHAPE
    for kw in (dict(heads=0), dict(heads=-4), dict(groups=0), dict(groups=3), dict(heads=3), dict(groups=8)):
        assert fwd(lib, lin(**kw), launch()) == SHAPE
    # heads * dk of 2^22
    assert fwd(lib, lin(heads=1 << 15, groups=1), launch(d=1 << 15, d_state=128)) == SHAPE
    assert fwd(lib, lin(), launch(io=2)) == DTYPE
    assert fwd(lib, lin(), launch(chunk=16)) == CHUNK
    for flag in (1, 2, 4, 16, 32):
        assert fwd(lib, lin(), launch(flags=flag)) == FLAGS
    assert fwd(lib, lin(), launch(), seg=-1) == SEGLEN and fwd(lib, lin(), launch(), seg=33) == SEGLEN
    assert fwd(lib, lin(offsets=addr(9), nseq=3), launch(), seg=50) == PARAM
    assert fwd(lib, lin(offsets=addr(9), nseq=-1), launch()) == SHAPE
    assert fwd(lib, lin(offsets=addr(9), nseq=0), launch()) == SHAPE
    for s in (float("inf"), float("nan")):
        assert fwd(lib, lin(scale=s), launch(**BIG)) == PARAM
    for kw in (dict(ld_q=15), dict(ld_k=0), dict(ld_v=-96), dict(ld_q=1 << 22), dict(hs_q=-1), dict(hs_k=1 << 38), dict(hs_v=-24),
               dict(ld_decay=3), dict(ld_decay=-4), dict(ld_decay=1 << 22)):
        assert fwd(lib, lin(**kw), launch(**BIG)) == PARAM
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(log_decay=None)):
        assert fwd(lib, lin(**kw), launch(**BIG)) == NULL
    assert fwd(lib, lin(), launch(**BIG), y=None) == NULL
    for kw in (dict(q=addr(0) + 1), dict(log_decay=addr(3) + 2), dict(h0=addr(4) + 1), dict(offsets=addr(9) + 2, nseq=1)):
        assert fwd(lib, lin(**kw), launch(**BIG)) == ALIGN
    assert fwd(lib, lin(), launch(io=0, **BIG), y=addr(5) + 2) == ALIGN
    assert fwd(lib, lin(), launch(**BIG), h=addr(6) + 2) == ALIGN
    n = 200 * 96 * 2
    for y in (addr(0), addr(2) + n - 2, addr(2) - n + 2, addr(3), addr(4)):
        assert fwd(lib, lin(), launch(**BIG), y=y) == ALIAS
    assert fwd(lib, lin(), launch(**BIG), h=addr(5)) == ALIAS
    # the extent of strided rows and heads counts, to the last one's end
    assert fwd(lib, lin(ld_q=100, hs_q=1000), launch(**BIG), y=addr(0) + (199 * 100 + 3 * 1000 + 15) * 2) == ALIAS
    need = binding.linattn_info(2, 100, 4, 16, 24)["workspace_bytes"]
    long_need = binding.linattn_info(2, 2000, 4, 16, 24)["workspace_bytes"]
    assert long_need > need >= 0
    assert fwd(lib, lin(), launch(seqlen=2000)) == WORKSPACE
    assert fwd(lib, lin(), launch(seqlen=2000, ws=addr(40), ws_bytes=long_need - 1)) == WORKSPACE
    assert fwd(lib, lin(), launch(seqlen=2000, ws=addr(40) + 8, ws_bytes=long_need)) == ALIGN
    for k in (0, 3, 5, 6):
        assert fwd(lib, lin(), launch(seqlen=2000, ws=addr(k), ws_bytes=long_need)) == ALIAS


def test_backward_refusals(lib):
    assert bwd(lib, lin(), None, launch(**BIG)) == NULL
    for kw in (dict(dq=None), dict(dk=None), dict(dv=None)):
        assert bwd(lib, lin(), grad(**kw), launch(**BIG)) == NULL
    for kw in (dict(ld_dy=23), dict(hs_dy=-1), dict(ld_dy=1 << 22)):
        assert bwd(lib, lin(), grad(**kw), launch(**BIG)) == PARAM
    for kw in (dict(dq=addr(10) + 1), dict(dlog_decay=addr(13) + 2), dict(dh0=addr(14) + 2), dict(dy=addr(8) + 1)):
        assert bwd(lib, lin(), grad(**kw), launch(**BIG)) == ALIGN
    for kw in (dict(dq=addr(0)), dict(dk=addr(8)), dict(dv=addr(12), dk=addr(12)), dict(dlog_decay=addr(3)), dict(dh0=addr(9)),
               dict(dh0=addr(13))):
        assert bwd(lib, lin(), grad(**kw), launch(**BIG)) == ALIAS
    need = binding.linattn_info(2, 100, 4, 16, 24, backward=True)["workspace_bytes"]
    assert need > 0
    assert bwd(lib, lin(), grad(), launch()) == WORKSPACE
    assert bwd(lib, lin(), grad(), launch(ws=addr(40), ws_bytes=need - 1)) == WORKSPACE
    for k in (0, 8, 10, 13):
        assert bwd(lib, lin(), grad(), launch(ws=addr(k), ws_bytes=need)) == ALIAS


def test_step_refusals(lib):
    def step(p, l, state=addr(5), slots=10, si=addr(6), so=addr(7), y=addr(8)):
        return lib.vimscan_linattn_step(ctypes.byref(p) if p else None, state, slots, si, so, y, ctypes.byref(l) if l else None)
    one = dict(seqlen=1)
    assert step(None, launch(**one)) == NULL and step(lin(), None) == NULL
    assert step(lin(), launch(seqlen=2)) == SHAPE and step(lin(), launch(**one), slots=-1) == SHAPE
    assert step(lin(), launch(batch=1 << 23, **one)) == SHAPE
    assert step(lin(), launch(flags=8, **one)) == FLAGS
    assert step(lin(scale=float("nan")), launch(**one)) == PARAM and step(lin(ld_k=3), launch(**one)) == PARAM
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(log_decay=None)):
        assert step(lin(**kw), launch(**one)) == NULL
    assert step(lin(), launch(**one), state=None) == NULL and step(lin(), launch(**one), y=None) == NULL
    assert step(lin(), launch(**one), state=addr(5) + 2) == ALIGN and step(lin(), launch(**one), si=addr(6) + 1) == ALIGN
    for kw in (dict(y=addr(0)), dict(y=addr(5)), dict(state=addr(3)), dict(si=addr(5))):
        assert step(lin(), launch(**one), **kw) == ALIAS
    assert step(lin(), launch(batch=0, **one)) == 0


def test_empty_calls_need_no_pointers(lib):
    none = dict(q=None, k=None, v=None, log_decay=None, h0=None)
    assert fwd(lib, lin(**none), launch(batch=0), y=None, h=None) == 0
    assert fwd(lib, lin(**none), launch(seqlen=0), y=None, h=None) == 0
    # rows of no tokens, cut every 50: no sequences, so nothing to write
    assert fwd(lib, lin(), launch(seqlen=0), seg=50) == 0
    p = binding.linattn_info(2, 0, 4, 16, 24, seg_len=50)
    assert (p["sequences"], p["workgroups"], p["kernels"]) == (0, 0, 0)
    assert bwd(lib, lin(**none), grad(dy=None, dh_last=None, dq=None, dk=None, dv=None, dlog_decay=None, dh0=None), launch(seqlen=0)) == 0


def test_plans(lib):
    info = binding.linattn_info
    p = info(128, 197, 12, 64, 64)
    assert (p["sequences"], p["chunks"], p["kernels"], p["workspace_bytes"]) == (128, 1, 1, 0)
    p = info(1, 65537, 24, 64, 64)
    assert p["kernels"] == 3 and p["chunk_len"] % 32 == 0 and p["chunks"] * p["chunk_len"] >= 65537
    assert p["workspace_bytes"] >= p["chunks"] * 24 * 64 * 64 * 4
    assert info(1, 0, 2, 16, 16)["kernels"] == 1 and info(0, 5, 2, 16, 16)["workgroups"] == 0
    p = info(1, 10000, 2, 64, 64, nseq=7)
    assert p["chunks"] == 10000 // p["chunk_len"] + 7 and p["seq_tokens"] == 0
    for args in ((1, 10, 3, 200, 16), (1, 10, 3, 16, 200)):
        with pytest.raises(binding.VimscanError):
            info(*args)
    with pytest.raises(binding.VimscanError):
        info(1, 10, 4, 16, 16, groups=3)


# ------------------------------------------------------------------------------------------
# Layer norm


def ln(**kw):
    f = dict(x=addr(0), ld_x=96, residual=addr(1), weight=addr(2), bias=addr(3), eps=1e-5, res_dtype=0)
    f.update(kw)
    return block._LayerNorm(**f)


def lfwd(lib, p, l, s=addr(5), n=addr(6)):
    return lib.vimscan_layernorm_fwd(ctypes.byref(p) if p else None, s, n, ctypes.byref(l) if l else None)


def lgrad(**kw):
    f = dict(dsum=addr(8), dn=addr(9), dx=addr(10), ld_dx=96, dresidual=addr(11), dweight=addr(12), dbias=addr(13))
    f.update(kw)
    return block._LayerNormGrad(**f)


def lbwd(lib, p, g, l):
    return lib.vimscan_layernorm_bwd(ctypes.byref(p), ctypes.byref(g) if g else None, ctypes.byref(l))


def test_layernorm_refusals(lib):
    ok = dict(d_state=0)
    assert lfwd(lib, None, launch(**ok)) == NULL and lfwd(lib, ln(), None) == NULL
    assert lfwd(lib, ln(), launch()) == SHAPE and lfwd(lib, ln(), launch(d=32769, **ok)) == SHAPE
    assert lfwd(lib, ln(), launch(flags=16, **ok)) == FLAGS and lfwd(lib, ln(), launch(io=3, **ok)) == DTYPE
    assert lfwd(lib, ln(res_dtype=1), launch(io=0, **ok)) == DTYPE
    for e in (0.0, -1.0, float("nan"), float("inf")):
        assert lfwd(lib, ln(eps=e), launch(**ok)) == PARAM
    assert lfwd(lib, ln(ld_x=95), launch(**ok)) == PARAM
    assert lfwd(lib, ln(x=None), launch(**ok)) == NULL and lfwd(lib, ln(), launch(**ok), n=None) == NULL
    assert lfwd(lib, ln(weight=addr(2) + 2), launch(**ok)) == ALIGN and lfwd(lib, ln(), launch(**ok), s=addr(5) + 2) == ALIGN
    for kw in (dict(s=addr(0)), dict(n=addr(1)), dict(n=addr(5)), dict(s=addr(1) + 4), dict(n=addr(3))):
        assert lfwd(lib, ln(), launch(**ok), **kw) == ALIAS
    big = dict(BIG, **ok)
    assert lbwd(lib, ln(), None, launch(**big)) == NULL
    for p, g in ((ln(weight=None), lgrad()), (ln(bias=None), lgrad()), (ln(residual=None), lgrad()), (ln(), lgrad(ld_dx=3))):
        assert lbwd(lib, p, g, launch(**big)) == PARAM
    for kw in (dict(dx=addr(0)), dict(dresidual=addr(8) + 4), dict(dresidual=addr(1)), dict(dweight=addr(13)), dict(dx=addr(11)),
               dict(dresidual=addr(9))):
        assert lbwd(lib, ln(), lgrad(**kw), launch(**big)) == ALIAS
    need = binding.layernorm_info(200, 96, backward=True)["workspace_bytes"]
    assert need > 0 and lbwd(lib, ln(), lgrad(), launch(**ok)) == WORKSPACE
    assert lbwd(lib, ln(), lgrad(), launch(ws=addr(40), ws_bytes=need - 1, **ok)) == WORKSPACE
    for k in (0, 1, 8, 9, 10, 11):
        assert lbwd(lib, ln(), lgrad(), launch(ws=addr(k), ws_bytes=need, **ok)) == ALIAS
    assert lfwd(lib, ln(x=None), launch(batch=0, **ok), s=None, n=None) == 0
