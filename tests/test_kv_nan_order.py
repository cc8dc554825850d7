"""What the chunk kernels know of NaN in a tile's values is not cleared before both
row tiles have looked, however late one of them is: a model on the CPU.

The converting warps note NaN values by tile in a ring of eight entries and clear the
one four tiles ahead; the softmax warps of the two row tiles look when a tile's
product is done.  The warps are run here as the kernels' waits let them, one row
tile held back before each of its looks until nobody else can go on.  Whether the
products wait for row tile 1 after a piece of two row tiles is read from the
kernel source."""
import itertools
import re

import pytest

import test_kv4_drains as drains

RING, AHEAD, SLOTS = 8, 4, 3


def run(pieces, late, waits):
    """pieces: (row tiles, key tiles) of a CTA's run.  Returns the tiles whose entry was cleared or taken before a look."""
    placed, empty, s_full, p_full, q_full, o_full, looked = (set() for _ in range(7))
    arrived, lost, first = [0], [], [sum(n for _, n in pieces[:i]) for i in range(len(pieces) + 1)]
    two_at = {first[i] + k: two for i, (two, n) in enumerate(pieces) for k in range(n)}

    def look_over(entry, before):   # every tile that the entry has stood for must have been looked at
        lost.extend(t for t, two in two_at.items() if t % RING == entry and t < before and not looked >= {(x, t) for x in range(two)})

    def convert():
        for t in range(first[-1]):
            look_over((t + AHEAD) % RING, t + 1)
            look_over(t % RING, t)
            for i in (2 * t, 2 * t + 1):
                while i >= SLOTS and i - SLOTS not in empty:
                    yield False
                placed.add(i)
                yield True

    def products():
        before, twos = 0, 0
        for i, (two, n) in enumerate(pieces):
            for k in range(n + 1):
                t = first[i] + k
                while k and 2 * t - 1 not in placed:
                    yield False
                if k == 1 and before == 2:
                    twos += 1
                    while waits and arrived[0] < twos:
                        yield False
                for x in range(two):
                    while ((x, t - 1) not in p_full) if k else ((x, i) not in q_full):
                        yield False
                    if k == n:
                        o_full.add((x, i))
                    if k and x == two - 1:
                        empty.add(2 * t - 1)
                    if k < n:
                        while 2 * t not in placed:
                            yield False
                        s_full.add((x, t))
                        if x == two - 1:
                            empty.add(2 * t)
                    yield True
            before = two

    def softmax(x):
        if x < pieces[0][0]:
            q_full.add((x, 0))
        for i, (two, n) in enumerate(pieces):
            more = i + 1 < len(pieces) and x < pieces[i + 1][0]
            if x >= two:
                if more:
                    q_full.add((x, i + 1))
                yield True
                continue
            for k in range(n):
                while (x, first[i] + k) not in s_full:
                    yield False
                if k:
                    yield None      # may be late
                    looked.add((x, first[i] + k - 1))
                p_full.add((x, first[i] + k))
                yield True
            if more:
                q_full.add((x, i + 1))
            while (x, i) not in o_full:
                yield False
            yield None
            looked.add((x, first[i] + n - 1))
            arrived[0] += x
            yield True
    actors = {"convert": convert(), "products": products(), 0: softmax(0), 1: softmax(1)}
    held = None
    while actors:
        went = False
        for name in list(actors):
            if name == held:
                continue
            try:
                got = next(actors[name])
                if got is None and name == late:
                    held = name
                went = went or got is not False
            except StopIteration:
                del actors[name]
                went = True
        if not went:
            assert held is not None, "nobody can go on"
            held = None
    assert looked == {(x, t) for t, two in two_at.items() for x in range(two)}
    return lost


RUNS = [list(zip(twos, tiles)) for twos in itertools.product((1, 2), repeat=4)
        for tiles in ((1, 1, 1, 1), (1, 9, 1, 9), (9, 1, 9, 1), (2, 3, 5, 2), (17, 6, 4, 30))]


def test_without_the_wait_a_late_row_tile_loses_what_was_known():
    assert any(run(r, 1, False) for r in RUNS)
    assert not any(run(r, 0, False) for r in RUNS)


@pytest.mark.parametrize("kernel", ["hs_kv4_prefill.cu", "hs_kv8_prefill.cu"])
@pytest.mark.parametrize("late", [None, 0, 1])
def test_a_late_row_tile_finds_what_is_known_of_nan(kernel, late):
    src = drains._squeeze(kernel)
    assert "const int on = (tiles + 4) % kPfInfo;" in src and f"kPfInfo = {RING};" in src and re.search(rf"kPfSlots = {SLOTS}\b", src)
    waits = ("if (k == 1 && two_before) { wait(&sh.nan_read, nan_phase); nan_phase ^= 1; }" in src and "two_before = two; next_piece();" in src
             and "see_nan(cnt - 1); if (x) { __syncwarp(); if (lane == 0) mbar_arrive(&sh.nan_read); }" in src
             and "mbar_init(&sh.nan_read, 4);" in src)
    for r in RUNS:
        assert not run(r, late, waits), r
