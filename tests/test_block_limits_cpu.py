"""Limits of the gated recurrence's and the block norm's launches, and what their plans say, without a GPU."""
import ctypes

import pytest

from bidirectional_selective_scan_amd import binding
from test_block_abi_cpu import addr, gated, launch, lib  # noqa: F401

MOST = 2 ** 24 - 1     # workgroups of 256 threads: a grid holds fewer than 2^32 threads


@pytest.mark.parametrize("tokens,tile,backward", [(2 ** 30, 64, True), (2 ** 31, 128, False)])
def test_a_plan_fits_a_grid(tokens, tile, backward):
    """The largest plan that is given is one that can be launched, and positions past its last tile's end still fit
    in 32 bits; one token more is refused."""
    most = tokens - tile
    info = binding.gated_info(1, most, 64, backward=backward)
    assert info["chunk_len"] == tile and info["workgroups"] == MOST and info["workgroups"] * 256 < 2 ** 32
    assert info["chunks"] * tile < 2 ** 31
    for more in (most + 1, tokens - 1):
        with pytest.raises(binding.VimscanError) as e:
            binding.gated_info(1, more, 64, backward=backward)
        assert e.value.status == -2
    # two channel blocks: half the tokens
    assert binding.gated_info(1, (most - tile) // 2, 128, backward=backward)["workgroups"] == MOST - 1
    with pytest.raises(binding.VimscanError):
        binding.gated_info(1, tokens // 2, 128, backward=backward)


def test_single_tokens_are_taken_up_to_their_limit(lib):  # noqa: F811
    def step(batch):
        l, g = launch(batch=batch, seqlen=1, d=64), gated(d=64, x=addr(0) - (1 << 36), r=addr(100), i=addr(200))
        return lib.vimscan_gated_step(ctypes.byref(g), addr(300), 10, addr(400), addr(500), addr(300), ctypes.byref(l))
    assert step(1 << 24) == -6 and step((1 << 24) + 1) == -2      # past the limit only the size is refused


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("backward", [False, True])
def test_a_norm_plan_is_what_is_launched(io, backward):
    """Workgroups, the rows of the first one and the workspace follow from the rows that the width's spread works
    on at once."""
    from test_block_index_replay import SPREADS_SINGLE, SPREADS_VECTOR_BWD, SPREADS_VECTOR_FWD
    for d in (1, 32, 63, 64, 65, 128, 129, 256, 257, 260, 512, 768, 1000, 1024, 1025, 1028, 1531, 2048, 2050, 4096, 8192, 20000, 32768):
        singles = io == "f32" and d % 4 != 0
        spreads, v = (SPREADS_SINGLE, 1) if singles else (SPREADS_VECTOR_BWD if backward else SPREADS_VECTOR_FWD, 4)
        nv, lanes, waves = next(s for s in spreads if s[0] * s[1] * s[2] * v >= d)
        at_once = (256 if waves <= 4 else 64 * waves) // (lanes * waves)
        for rows in (1, 3, 16, 17, 100, 511, 2048, 2049, 4097, 30000, 25216):
            turns = -(-rows // at_once)
            wgs = min(turns, 2048 if d <= 256 else 512)
            info = binding.norm_info(rows, d, io, backward)
            assert info["workgroups"] == wgs
            # the first workgroup takes turns 0, wgs, 2 wgs, ..
            assert info["chunk_len"] == -(-turns // wgs) * at_once
            need = wgs * 3 * d * 4 if backward else 0
            assert need <= info["workspace_bytes"] < need + 256


def test_gradient_rows_that_share_elements_are_refused(lib):  # noqa: F811
    """dx, dr and di (dx and dz) as slices of one array: side by side they are taken (the call then stops at its
    missing workspace), shifted into each other they are refused."""
    from bidirectional_selective_scan_amd import block
    from test_block_abi_cpu import bwd, grad, norm
    big = addr(11)

    def gated_status(*offsets, ld=(200, 200, 200), io=1):
        e = 2 if io else 4
        at = [None if o is None else big + o * e for o in offsets]
        return bwd(lib, gated(), grad(dx=at[0], dr=at[1], di=at[2], ld_dx=ld[0], ld_dr=ld[1], ld_di=ld[2]), launch(io=io))

    def norm_status(x, z, ld=100):
        g = block._NormGrad(dsum=addr(8), dn=addr(9), dx=big + 2 * x, dz=big + 2 * z, ld_dx=ld, ld_dz=ld, dresidual=addr(12),
                            dw_post=addr(13), dgamma=addr(14), dw_pre=addr(15))
        return lib.vimscan_norm_bwd(ctypes.byref(norm()), ctypes.byref(g), ctypes.byref(launch(d_state=0)))

    for io in (0, 1):
        assert gated_status(0, 48, 96, io=io) == -7 and gated_status(152, 0, 104, io=io) == -7
        assert gated_status(0, 48 + 200 * 7, 96, io=io) == -7                     # other rows of the array
        assert gated_status(0, 200 * 200, 2 * 200 * 200, io=io) == -7             # arrays behind each other
        assert gated_status(0, None, None, io=io) == -7
        for shift in (1, 47, 153, 199, 200, 201, 200 * 199 + 47):
            assert gated_status(0, shift, None, io=io) == -6 and gated_status(shift, 0, None, io=io) == -6
            assert gated_status(0, None, shift, io=io) == -6
            assert gated_status(3 * 10 ** 6, 0, shift, io=io) == -6
    assert gated_status(0, 48, 96, ld=(96, 192, 192)) == -7 and gated_status(0, 47, 96, ld=(96, 192, 192)) == -6
    assert norm_status(0, 48) == -7 and norm_status(52, 0) == -7
    for shift in (0, 1, 47, 53, 100, 100 * 150 + 20):
        assert norm_status(0, shift) == -6 and norm_status(shift, 0) == -6
