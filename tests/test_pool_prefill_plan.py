"""The host's plan of a ragged pre-fill, read back from the library (duo_debug_prefill_runs,
duo_debug_prefill_deal): visible ring slots, key tiles and dealt shares have the properties
that the kernel relies on, and are what the forms restated in test_pool_prefill.py say."""
import numpy as np
import pytest

import oracle
from head_split_kv_duo_b200 import duo
from test_pool_prefill import deal, ring_view, tiles_of

SOURCES = ("pages", "slots", "chunk")


def runs(retrieval, length, n, r0, npos, S, W):
    st, got, ring = duo.duo_debug_prefill_runs(retrieval, length, n, r0, npos, S, W)
    assert st == duo.DUO_OK and len(got) <= 5 and all(c >= 1 for _, _, c in got)
    return [(SOURCES[s], t) for s, first, c in got for t in range(first, first + c)], ring


def test_ring_slots_are_the_mask():
    """Slots of the library's runs hold exactly the visible positions that are no sinks, each once."""
    for S in (0, 1, 3, 9):
        for W in (1, 2, 5, 8):
            for length in range(0, 30):
                held = oracle.ring_replay(S, W, [length])[0] if length else -np.ones(S + W, dtype=np.int64)
                for i in range(12):
                    _, (lo1, hi1, lo2, hi2) = runs(0, length, 12, i, 1, S, W)
                    assert [(lo1, hi1), (lo2, hi2)] == list(ring_view(length + i, length, S, W))
                    got = sorted(int(held[x]) for lo, hi in ((lo1, hi1), (lo2, hi2)) for x in range(lo, hi))
                    assert got == [p for p in range(S, length) if length + i - p < W], (S, W, length, i)


def test_tiles_are_what_is_visible():
    """A streaming head's tiles: every visible key's, each once; a retrieval head's: the pages of
    the history, then the rows up to its last query."""
    rng = np.random.default_rng(5)
    for _ in range(2000):
        S, W = int(rng.integers(0, 300)), int(rng.integers(1, 600))
        length, n = int(rng.integers(0, 1500)), int(rng.integers(1, 900))
        npos = 128 // int(rng.choice([1, 2, 3, 4, 5, 8, 16]))
        r0 = 2 * npos * int(rng.integers(0, -(-n // (2 * npos))))
        rows = min(r0 + 2 * npos, n)
        got, _ = runs(1, length, n, r0, npos, S, W)
        assert got == [("pages", t) for t in range(-(-length // 128))] + [("chunk", t) for t in range(-(-rows // 128))]
        got, _ = runs(0, length, n, r0, npos, S, W)
        assert len(got) == len(set(got)) and got == tiles_of(r0, rows, length, S, W)
        want = set()
        for i in {length + r0, length + rows - 1}:
            for p in list(range(min(S, i + 1))) + list(range(max(0, i - W + 1), i + 1)):
                want.add(("chunk", (p - length) // 128) if p >= length else
                         ("slots", (p if p < S else S + p % W) // 128))
        assert want <= set(got), (S, W, length, n, r0)


def dealt(items, sms):
    st, *plan = duo.duo_debug_prefill_deal([t for t, _ in items], [c for _, c in items], sms)
    assert st == duo.DUO_OK
    return plan


def test_dealing_covers_every_tile_once():
    """Every tile of every item goes to one CTA; the pieces of a cut item have places of their
    own in the scratch, found in order; whole items in rounds."""
    rng = np.random.default_rng(6)
    for _ in range(400):
        n = int(rng.choice([1, 2, 5, 40, 148, 149, 600]))
        top = int(rng.choice([1, 2, 7, 60, 1000]))
        items = sorted(((int(rng.integers(1, top + 1)), int(rng.choice([4, 5]))) for _ in range(n)), reverse=True)
        sms = int(rng.choice([1, 3, 132, 148, 160]))
        whole, ctas, shares, cuts = dealt(items, sms)
        assert (whole, ctas, shares, [list(c) for c in cuts]) == deal(items, sms)
        assert 1 <= ctas <= min(sms, 148) and whole % ctas == 0 and whole <= n and len(cuts) <= ctas
        pieces = {u: [(0, items[u][0], -1)] for u in range(whole)}
        for first, tile, left, place in shares:  # as the kernel walks them
            u, j = first, tile
            while left > 0:
                nt = min(items[u][0] - j, left)
                pieces.setdefault(u, []).append((j, nt, -1 if nt == items[u][0] else place + (u != first)))
                left, j, u = left - nt, 0, u + 1
        used = [p for v in pieces.values() for _, _, p in v if p >= 0]
        assert len(used) == len(set(used)) and all(p < 2 * 148 for p in used)
        by_item = {c[0]: c for c in cuts}
        for u in range(n):
            at = 0
            for j, nt, _ in pieces[u]:
                assert j == at and nt >= 1
                at += nt
            assert at == items[u][0]
            places = [p for _, _, p in pieces[u]]
            if len(places) > 1:
                _, count, part0, part1 = by_item[u]
                assert places == [part0] + [part1 + 2 * i for i in range(count - 1)]
            else:
                assert places == [-1] and u not in by_item


@pytest.mark.parametrize("call", [
    lambda: duo.duo_debug_prefill_runs(2, 0, 1, 0, 32, 4, 16), lambda: duo.duo_debug_prefill_runs(0, -1, 1, 0, 32, 4, 16),
    lambda: duo.duo_debug_prefill_runs(0, 0, 0, 0, 32, 4, 16), lambda: duo.duo_debug_prefill_runs(0, 0, 5, 5, 32, 4, 16),
    lambda: duo.duo_debug_prefill_runs(0, 0, 5, 0, 0, 4, 16), lambda: duo.duo_debug_prefill_runs(0, 0, 5, 0, 32, -1, 16),
    lambda: duo.duo_debug_prefill_runs(0, 0, 5, 0, 32, 4, 0), lambda: duo.duo_debug_prefill_deal([], [], 148),
    lambda: duo.duo_debug_prefill_deal([0], [4], 148), lambda: duo.duo_debug_prefill_deal([3], [0], 148),
    lambda: duo.duo_debug_prefill_deal([3], [4], 0)])
def test_read_back_refuses(call):
    assert call()[0] == duo.DUO_ERR_INVALID
