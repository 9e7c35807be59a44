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


@pytest.mark.parametrize("heads,io,d", [(1, "bf16", 64), (2, "bf16", 64), (1, "f32", 16), (1, "f32", 128)])
@pytest.mark.parametrize("length", [2048, 16385, 65537, 1 << 20, (1 << 31) - 1])
def test_few_heads_do_not_wait_for_the_fold(heads, io, d, length):
    """The fold's rounds of eight segments, each some 0.4 of a chunk in two passes, are not many more than the segment's chunks."""
    seg, count = segments(1, length, heads, d, d, io_dtype=io)
    assert 0.4 * count / 8 <= 1.6 * seg / 32 + 1


@pytest.mark.parametrize("tokens,nseq", [(65600, 64), (65569, 33), (40000, 201), (8448, 257), (1 << 20, 4096), (1 << 20, 40), (33000, 1000)])
@pytest.mark.parametrize("heads,io", [(24, "bf16"), (1, "bf16"), (24, "f32")])
@pytest.mark.parametrize("backward", [False, True])
def test_one_long_packed_sequence_is_never_walked_whole(tokens, nseq, heads, io, backward):
    """Only the mean length is known: where all tokens could be one sequence's, it is cut at 2048 tokens or twice the mean."""
    p = binding.linattn_info(1, tokens, heads, 64, 64, io_dtype=io, nseq=nseq, backward=backward)
    assert 0 < p["chunk_len"] <= max(2048, 2 * -(-tokens // nseq) + 31)
    assert p["chunks"] == tokens // p["chunk_len"] + nseq


def test_few_packed_tokens_take_one_kernel():
    assert binding.linattn_info(1, 8192, 12, 64, 64, nseq=128)["kernels"] == 1
