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
