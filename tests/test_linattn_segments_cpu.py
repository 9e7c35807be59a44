"""How linear attention's plans cut sequences into segments (linattn_info, host only)."""
import pytest

from bidirectional_selective_scan_amd import binding


def segments(*a, **kw):
    p = binding.linattn_info(*a, **kw)
    return (p["chunk_len"], p["chunks"]) if p["kernels"] > 1 else None


@pytest.mark.parametrize("length", [4096, 4097, 6000, 65537])
@pytest.mark.parametrize("batch", [43, 64, 256])
def test_sequences_that_fill_the_chip_stay_whole(batch, length):
    assert segments(batch, length, 24, 64, 64) is None


@pytest.mark.parametrize("batch,length", [(16, 8200), (1, 4097), (8, 32769), (4, 65537), (1, 65537), (3, 10000), (8, 1025)])
def test_segments_are_of_nearly_equal_length(batch, length):
    seg, count = segments(batch, length, 24, 64, 64)
    chunks = -(-length // 32)
    assert seg == -(-chunks // count) * 32 and (count - 1) * seg < length <= count * seg
