"""What a workgroup of the gated recurrence does whose wait takes too long (gated.hip: Alone), without a GPU: it
composes the maps of the tiles before its own exactly as the hand-over does; and why there must be such a way."""
import random

import pytest

GROUP, EACH = 16, 4


def then(f, g):
    return f + g


def leaves(first_of, group):
    """chain_leave of a group's last tile: its map on what chain_gather brought in. A state is a nested tuple of
    the maps applied to it, a map the tuple of tiles it is composed of, in order."""
    j = group * GROUP + GROUP - 1
    return ("apply", (j,), enters(first_of, j))


def enters(first_of, j):
    """chain_gather and chain_carry."""
    first, g0 = first_of(j), j // GROUP * GROUP
    h = leaves(first_of, j // GROUP - 1) if first < g0 else 0
    lo = g0 if first < g0 else first
    for w in range(4):
        f = ()
        for t in range(lo + w * EACH, min(j, lo + w * EACH + EACH)):
            f = then(f, (t,))
        h = ("apply", f, h)
    return h


def enters_alone(first, j):
    """Alone::gather, then chain_carry."""
    g0 = j // GROUP * GROUP
    parts = []
    inc = 0
    for wave in range(4):
        lo = (g0 if first < g0 else first) + wave * EACH
        h, f, quarters = 0, (), 0
        for t in range(first if wave == 0 and first < g0 else lo, min(j, lo + EACH)):
            last = t < lo and t % GROUP == GROUP - 1
            if not last:
                f = then(f, (t,))
            if t >= lo:
                continue
            if not last and (t - max(first, t // GROUP * GROUP)) % EACH != EACH - 1:
                continue
            while True:
                h, f = ("apply", f, h), ()
                quarters += 1
                if not (quarters < 4 and last):
                    break
            if last:
                h, quarters = ("apply", (t,), h), 0
        parts.append(f)
        if wave == 0:
            inc = h
    for f in parts:
        inc = ("apply", f, inc)
    return inc


@pytest.mark.parametrize("start", [0, 1, 3, 5, 14, 15, 16, 17, 30, 31, 47, 50])
def test_the_same_maps_in_the_same_order(start):
    """One sequence from tile start on. A tile where another one is still going on before it (start itself, when
    the sequence starts inside it) takes nothing from there: its map does not depend on it."""
    def first_of(j):
        return start if j > start else j
    for j in range(start, start + 70):
        assert enters_alone(first_of(j), j) == enters(first_of, j), j


class Gpu:
    """XCDs with a few places for workgroups each. The workgroups of a call go to the XCDs in turn and, on an XCD,
    start in the order of their ids; which call starts one first is up to the caller."""

    def __init__(self, xcds, room, calls, alone):
        self.room, self.alone = [room] * xcds, alone
        self.queue = {(c, x): [w for w in range(n) if w % xcds == x] for c, n in enumerate(calls) for x in range(xcds)}
        self.running, self.done, self.left = [], [set() for _ in calls], sum(calls)

    def start(self, c, x):
        if not self.queue[c, x] or not self.room[x]:
            return False
        self.room[x] -= 1
        self.running.append((c, x, self.queue[c, x].pop(0)))
        return True

    def end(self, r):
        c, x, tile = r
        self.running.remove(r)
        self.done[c].add(tile)
        self.room[x] += 1
        self.left -= 1

    def run(self, order):
        for c, x in order:
            self.start(c, x)
        while True:
            ready = [r for r in self.running if all(t in self.done[r[0]] for t in range(r[2]))]
            if not ready and self.alone:
                ready = list(self.running)      # they have waited for long enough
            for r in ready:
                self.end(r)
            started = [self.start(c, x) for c, x in list(self.queue) for _ in range(self.room[x])]
            if not ready and not any(started):
                return self.left == 0


# two calls of twelve tiles on two XCDs with three places each: the first call fills one XCD, the second the other
CROSSED = [(0, 0)] * 3 + [(1, 1)] * 3


def test_waits_alone_can_block_each_other():
    assert not Gpu(2, 3, (12, 12), alone=False).run(CROSSED)
    assert Gpu(2, 3, (12, 12), alone=True).run(CROSSED)


def test_every_call_ends():
    rng = random.Random(1)
    for _ in range(300):
        xcds, calls = rng.choice((1, 2, 4, 8)), [rng.randint(1, 40) for _ in range(rng.randint(1, 4))]
        order = [(rng.randrange(len(calls)), rng.randrange(xcds)) for _ in range(rng.randint(0, 60))]
        assert Gpu(xcds, rng.randint(1, 5), calls, alone=True).run(order)


def test_the_number_of_reads_is_checked():
    from bidirectional_selective_scan_amd import binding
    with pytest.raises(binding.VimscanError) as e:
        binding.gated_wait_reads(-1)
    assert e.value.status == -13
    binding.gated_wait_reads()
    assert binding.load_library().vimscan_gated_alone(None) == -1
