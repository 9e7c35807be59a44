"""Host replay of the memory indices that the gated recurrence's and the block norm's kernels form,
against the sizes of what they address, without a GPU.

The index formulas restate the kernel code (gated.hip: TileRows, seq_at, seq_at_wave, WaveSeqs,
chain_gather, chain_leave, pass_empty, the kernels; blocknorm.hip: Spread, ld_row, k_norm_bwd's partial
gradients; block_device.h: column_sum). Offsets that break their rules (not sorted, negative, past
the end) must not lead outside the arrays either."""
import numpy as np
import pytest

from bidirectional_selective_scan_amd import binding

BLOCK, FWD, FWD_SMALL, BWD, GROUP, STRIDE = 64, 128, 64, 64, 16, 64
OUTSIDE = 0x80000000


class Call:
    """The sequences of a call, in walking order."""

    def __init__(self, n, rev, lp=0, offsets=None, nseq=None):
        self.n, self.rev, self.lp, self.off = n, rev, lp, offsets
        self.nseq = len(offsets) - 1 if offsets is not None else (n // lp if nseq is None else nseq)

    def bound(self, q):
        if self.off is None:
            return q * self.lp
        k = self.nseq - q if self.rev else q
        assert 0 <= k <= self.nseq          # the index read
        o = min(max(int(self.off[k]), 0), self.n)
        return self.n - o if self.rev else o

    def at(self, p, lo, hi):
        if self.off is None:
            return p // self.lp
        while lo < hi:
            mid = lo + (hi - lo + 1) // 2
            if self.bound(mid) <= p:
                lo = mid
            else:
                hi = mid - 1
        return lo

    def at_wave(self, p):
        if self.off is None:
            return p // self.lp
        lo, n, rounds = 0, self.nseq, 0
        while n > 1:
            step = (n + 63) // 64
            k = sum(1 for lane in range(64) if (lane + 1) * step < n and self.bound(lo + (lane + 1) * step) <= p) * step
            lo, n = lo + k, min(n - k, step)
            rounds += 1
            assert rounds < 8 and n >= 1
        return lo

    def wave_seqs(self, pw, size, lo):
        """(starts, ends, rows) of positions pw .. pw + size - 1."""
        starts, ends, rows = set(), set(), {}
        pe = min(pw + size, self.n)
        if pw >= self.n or (self.bound(lo) != pw and self.bound(lo + 1) > pe):
            return starts, ends, rows
        hi = self.at_wave(pe - 1) if self.off is not None else 0
        for lane in range(size):
            p = pw + lane
            q = self.at(p, lo, hi) if p < pe else lo
            rows[lane] = self.nseq - 1 - q if self.rev else q
            if p < pe and self.bound(q) == p:
                starts.add(lane)
            if p < pe and (self.bound(q + 1) == p + 1 or p + 1 == self.n):
                ends.add(lane)
        return starts, ends, rows


def truth(n, rev, bounds):
    """Per walking position: the caller's sequence, first of it, last of it."""
    out = [None] * n
    for s, (lo, hi) in enumerate(bounds):
        for t in range(lo, hi):
            p = n - 1 - t if rev else t
            out[p] = (s, t == (hi - 1 if rev else lo), t == (lo if rev else hi - 1))
    return out


def replay_sequences(call, tile, size, good):
    """Every wave of every tile: rows inside the sequences, flags as the offsets say (when they are good),
    and the tiles a tile waits for are ones before it in its group."""
    n = call.n
    tiles = -(-n // tile)
    for j in range(tiles):
        p0 = j * tile
        q0 = call.at_wave(p0)
        assert 0 <= q0 < call.nseq
        for w in range(4):
            pw = p0 + w * size
            starts, ends, rows = call.wave_seqs(pw, size, q0)
            for lane, r in rows.items():
                assert 0 <= lane < size and 0 <= r < call.nseq
            assert (starts | ends) <= set(rows)
            if pw < n <= pw + size:
                assert n - 1 - pw in ends      # the stream's last position, whatever the offsets hold
            if good is None:
                continue
            for lane in range(size):
                p = pw + lane
                want = good[p] if p < n else (None, False, False)
                assert (lane in starts) == want[1] and (lane in ends) == want[2], (p, want)
                if want[1] or want[2]:
                    assert rows[lane] == want[0]
        # forward: waits for tiles first .. j - 1
        start = call.bound(q0)
        first = j if start >= p0 else start // tile
        assert 0 <= first <= j
        if good is not None and first < j:
            assert not good[p0][1]
            assert all(not good[t * tile][1] for t in range(first + 1, j + 1))
        replay_gather(j, first, tiles)
        # backward: the chain runs from the last tile, jb its index
        jb, nxt = tiles - 1 - j, p0 + tile
        first = jb
        if nxt < n:
            q = call.at_wave(nxt)
            if call.bound(q) != nxt:
                first = tiles - 1 - (call.bound(q + 1) - 1) // tile
        first = min(max(first, 0), jb)
        if good is not None and nxt < n:
            assert (first == jb) == good[nxt][1]
            if first < jb:   # the sequence that goes on behind this tile ends in tile tiles - 1 - first
                last = next(p for p in range(nxt, n) if good[p][2])
                assert tiles - 1 - first == last // tile
        replay_gather(jb, first, tiles)


def replay_gather(j, first, tiles):
    each, g0 = GROUP // 4, j // GROUP * GROUP
    lo0 = g0 if first < g0 else first
    seen = []
    for w in range(4):
        lo = lo0 + w * each
        for k in range(max(0, min(j - lo, each))):
            seen.append(lo + k)
    assert seen == list(range(lo0, j))        # each awaited tile once, in order, all before j
    if first < g0:
        assert g0 > 0 and g0 // GROUP - 1 < -(-tiles // GROUP)


def positions_per_wave(vec, tile):
    lanes = BLOCK // vec
    return tile // (256 // lanes) * 64 // lanes


@pytest.mark.parametrize("tile,vec", [(FWD, 2), (FWD, 1), (FWD_SMALL, 2), (FWD_SMALL, 1), (BWD, 2), (BWD, 1)])
@pytest.mark.parametrize("rev", [False, True])
def test_sequences_of_a_tile(tile, vec, rev):
    size = positions_per_wave(vec, tile)
    assert 4 * size == tile and size <= 64
    for n, lp in ((1, 1), (7, 1), (64, 64), (130, 65), (130, 13), (394, 197), (255, 51), (512, 128), (1025, 1025), (2050, 1025)):
        replay_sequences(Call(n, rev, lp), tile, size, truth(n, rev, [(k * lp, k * lp + lp) for k in range(n // lp)]))
    rng = np.random.default_rng(tile + vec)
    for k in range(14):
        lens = rng.integers(0, [3, 30, 300][k % 3], size=[200, 70, 12][k % 3])
        if k % 4 == 0:
            lens[rng.integers(0, len(lens), size=len(lens) // 2)] = 0
        off = np.concatenate([[0], np.cumsum(lens)])
        if off[-1] == 0:
            continue
        replay_sequences(Call(int(off[-1]), rev, offsets=off), tile, size,
                         truth(int(off[-1]), rev, list(zip(off[:-1].tolist(), off[1:].tolist()))))


@pytest.mark.parametrize("rev", [False, True])
def test_offsets_that_break_the_rules_stay_inside(rev):
    rng = np.random.default_rng(5)
    for k in range(30):
        n = int(rng.integers(1, 500))
        off = rng.integers(-2 ** 31, 2 ** 31 - 1, size=int(rng.integers(2, 90)))
        if k % 2:
            off = rng.integers(-5, n + 5, size=len(off))
        for tile, vec in ((FWD, 2), (BWD, 1)):
            replay_sequences(Call(n, rev, offsets=off), tile, positions_per_wave(vec, tile), None)


@pytest.mark.parametrize("vec", [1, 2])
@pytest.mark.parametrize("tile", [FWD, FWD_SMALL, BWD])
@pytest.mark.parametrize("rev", [False, True])
def test_rows_of_a_tile(vec, tile, rev):
    """The byte offset of every element a thread touches is that of the position's token and channel;
    what lies outside the stream or the row gets an offset that the resource does not hold."""
    lanes = BLOCK // vec
    groups = 256 // lanes
    per = tile // groups
    tid = np.arange(256)
    cl, tg = tid % lanes, tid // lanes
    for e in (2, 4):
        for n, d, ld in ((1, vec, vec), (tile, 64, 64), (tile + 5, 70 * vec, 211 * vec), (3 * tile - 1, 96, 2 ** 22 - 2)):
            row_bytes = ld * e
            for j in range(-(-n // tile)):
                p0 = j * tile
                first = n - p0 - tile if rev else p0
                full = p0 + tile <= n
                for cb in range(-(-d // BLOCK)):
                    c0 = cb * BLOCK + cl * vec
                    row = (tile // per - 1 - tg if rev else tg) * per
                    vo = np.where(c0 < d, row * row_bytes + c0 * e, OUTSIDE)
                    assert (vo[c0 < d] < 2 ** 31).all()
                    for k in range(per):
                        so = ((per - 1) * row_bytes if rev else 0) + k * (-row_bytes if rev else row_bytes)
                        assert 0 <= so < 2 ** 31
                        p = p0 + tg * per + k
                        inside = (c0 < d) & (full | (p < n))
                        at = first * row_bytes + vo + so
                        token = n - 1 - p if rev else p
                        assert (at[inside] == (token * row_bytes + c0 * e)[inside]).all()
                        assert (token[inside] >= 0).all() and (c0[inside] + vec <= d).all()
                        assert (vo + so)[inside].max(initial=0) + vec * e <= 0x7fffffff
                        dropped = np.where(c0 < d, OUTSIDE, vo)[~inside]
                        assert (dropped + so >= OUTSIDE).all() and (dropped + so < 2 ** 32).all()


def test_division_by_the_length():
    """position / Lp = position * mul >> shift for every position below 2^31."""
    rng = np.random.default_rng(9)
    lengths = [1, 2, 3, 5, 7, 51, 65, 197, 1025, 2 ** 30, 2 ** 31 - 1] + [int(v) for v in rng.integers(1, 2 ** 31 - 1, 200)]
    for lp in lengths:
        s = 0
        while (1 << s) < lp:
            s += 1
        mul = (1 << (31 + s)) // lp + 1
        assert mul < 2 ** 32
        top = (2 ** 31 - 1) // lp * lp
        for p in [0, 1, lp - 1, lp, top, max(top - 1, 0), 2 ** 31 - 1] + [int(v) for v in rng.integers(0, 2 ** 31 - 1, 50)]:
            if p < 2 ** 31:
                assert p * mul >> (31 + s) == p // lp


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 65, 32), (8, 1025, 768), (128, 197, 768), (1, 65537, 1536), (3, 77, 130)])
def test_workspace_of_the_hand_over(shape, backward):
    batch, length, d = shape
    info = binding.gated_info(batch, length, d, backward=backward)
    n, tile = batch * length, info["chunk_len"]
    tiles, ncb = info["chunks"], -(-d // BLOCK)
    assert tile in ((BWD,) if backward else (FWD, FWD_SMALL)) and tiles == -(-n // tile)
    assert info["workgroups"] == tiles * ncb
    width = ncb * BLOCK
    end = 0
    if tiles > 1 and tile % length != 0:
        groups = -(-tiles // GROUP)
        off_inc = -(-tiles * width * 16 // 256) * 256
        # words of tile j: 2 j width + block + lane and width further on
        assert (2 * (tiles - 1) * width + width + (ncb - 1) * BLOCK + 63 + 1) * 8 <= off_inc
        end = off_inc + -(-groups * width * 16 // 256) * 256
        assert off_inc + (2 * (groups - 1) * width + width + (ncb - 1) * BLOCK + 63 + 1) * 8 <= end
    if backward:
        # partial sums: tile * width + block + lane; read by column_sum at k * width + c, c < d
        assert end + tiles * width * 4 <= info["workspace_bytes"]
    else:
        assert info["workspace_bytes"] == end


SPREADS_VECTOR_FWD = [(1, 16, 1), (1, 32, 1), (1, 64, 1), (2, 64, 1), (3, 64, 1), (4, 64, 1), (2, 64, 4), (4, 64, 4), (4, 64, 8),
                      (4, 64, 16), (8, 64, 16)]
SPREADS_VECTOR_BWD = SPREADS_VECTOR_FWD[:6] + [(1, 64, 8), (1, 64, 16), (2, 64, 16), (4, 64, 16), (8, 64, 16)]
SPREADS_SINGLE = [(4, 16, 1), (4, 32, 1), (4, 64, 1), (8, 64, 1), (4, 64, 4), (4, 64, 8), (8, 64, 8), (8, 64, 16), (16, 64, 16),
                  (32, 64, 16)]


@pytest.mark.parametrize("spreads,v", [(SPREADS_VECTOR_FWD, 4), (SPREADS_VECTOR_BWD, 4), (SPREADS_SINGLE, 1)])
def test_every_width_is_covered_once(spreads, v):
    """The first spread that holds a row touches each of its channels exactly once, inside the row, also
    where the last vector is read as the row's last four channels."""
    for d in list(range(1, 300)) + [511, 512, 513, 767, 768, 1000, 1024, 1025, 1531, 2048, 2049, 4096, 4097, 8191, 8192, 8193,
                                    16384, 16385, 32767, 32768]:
        nv, lanes, waves = next(s for s in spreads if s[0] * s[1] * s[2] * v >= d)
        place = np.arange(lanes * waves)
        c = np.concatenate([(k * lanes * waves + place) * v for k in range(nv)])
        c = c[c < d]
        if v == 1 or d % v == 0:
            read = c
        elif d >= v:
            read = np.minimum(c, d - v)
            # what was read, shifted down by c + v - d, starts at channel c
            shift = np.maximum(c + v - d, 0)
            assert (read + shift == c).all() and (shift < v).all()
        else:
            read = c[:0]                       # by elements, only those below d
        assert (read >= 0).all() and (read + v <= d).all()
        touched = np.concatenate([np.minimum(c + k, d) for k in range(v)])
        assert (np.bincount(touched, minlength=d + 1)[:d] == 1).all()
        rows = (256 if waves <= 4 else 64 * waves) // (lanes * waves)
        assert rows >= 1
        # LDS of the partial gradients (several rows) and of the sums
        assert rows == 1 or 3 * 4 * nv * v * lanes * 4 <= 64 * 1024
        assert waves < 16 or nv * v < 8 or nv * lanes * waves * v > 8192 or 3 * nv * 64 * waves * v * 4 <= 128 * 1024


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 768), (25216, 768), (4099, 8192), (30000, 32), (5, 32768)])
def test_workspace_of_the_partial_gradients(rows, d):
    info = binding.norm_info(rows, d, backward=True)
    # workgroup w leaves rows w * 3 * d .. + 3 d; no more workgroups run than the plan says
    assert info["workgroups"] * 3 * d * 4 <= info["workspace_bytes"]
    assert info["workgroups"] * info["chunk_len"] >= rows
