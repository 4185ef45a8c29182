"""Ragged pre-fill attention over the pool (duo_pool_prefill): the slot arithmetic of the
kernel restated and checked on the CPU, refusals and bookkeeping with launches skipped, and
on the GPU outputs against the fp64 oracle over each sequence's own tokens, with the cached
rows bit for bit."""
import time

import numpy as np
import pytest
import torch

import oracle
from head_split_kv_duo_b200 import duo, inputs
from head_split_kv_duo_b200.duo import DuoPool, DuoRope
from parity import assert_close, bits
from test_norm_rope import freqs, reference
from test_pool_share import _fail, _fill, _free, _listed, _pool, check_rows

FAKE, POOL = 2 << 40, 1 << 40  # tensors, and the pool's buffer (of test_pool_share)
Q, K, V, OUT, LSE = (FAKE + (i << 36) for i in range(5))
DEV = "cuda"


@pytest.fixture
def dry_run():
    assert duo.duo_debug_launch_controls(1, -1) == duo.DUO_OK
    yield
    assert duo.duo_debug_launch_controls(0, -1) == duo.DUO_OK


# ---------------------------------------------------------------- arithmetic on the CPU

def ring_view(i, length, S, W):
    """The kernel's two runs of visible ring slots (as slots of the sink + ring array)."""
    r = length % W
    a, e = i - length + r + 1, S - length + r + W
    return (S + max(0, max(a, e) - W), S + r), (S + max(r, max(a, e)), S + W)


def test_ring_view_is_the_mask():
    """For every small sink, window, length and query: the slots that the runs name hold
    exactly the visible non-sink positions, each once."""
    for S in (0, 1, 3, 9):
        for W in (1, 2, 5, 8):
            for length in range(0, 30):
                held = oracle.ring_replay(S, W, [length])[0] if length else -np.ones(S + W, dtype=np.int64)
                for i in range(length, length + 12):
                    runs = ring_view(i, length, S, W)
                    got = sorted(int(held[x]) for lo, hi in runs for x in range(lo, hi))
                    want = [p for p in range(S, length) if i - p < W]
                    assert got == want, (S, W, length, i, runs)


def test_slots_are_two_runs():
    """A row's visible slots as the kernel masks them: [0, front) and [lo, hi)."""
    for S in (0, 1, 3, 9):
        for W in (1, 2, 5, 8):
            for length in range(0, 30):
                held = oracle.ring_replay(S, W, [length])[0] if length else -np.ones(S + W, dtype=np.int64)
                for i in range(length, length + 12):
                    (lo1, hi1), (lo, hi) = ring_view(i, length, S, W)
                    front = min(S, length)
                    if lo1 == S:
                        front = max(front, hi1)
                    else:
                        lo, hi = lo1, hi1
                    got = [x for x in range(S + W) if x < front or lo <= x < hi]
                    want = [x for x in range(S + W) if held[x] >= 0 and (held[x] < S or i - held[x] < W)]
                    assert got == want, (S, W, length, i)


def tiles_of(r0, rows, length, S, W):
    """The kernel's key tiles of a streaming CTA whose first query is chunk position r0 and
    whose chunk rows end at `rows`: {(source, tile)}."""
    out, at = [], 0

    def add(src, lo, hi):
        nonlocal at
        if lo >= hi:
            return
        a, b = max(lo // 128, at), -(-hi // 128)
        if a < b:
            out.extend((src, t) for t in range(a, b))
            at = b

    (lo1, hi1), (lo2, hi2) = ring_view(length + r0, length, S, W)
    add("slots", 0, min(S, length))
    add("slots", lo1, hi1)
    add("slots", lo2, hi2)
    at = 0
    add("chunk", 0, min(rows, S - length))
    add("chunk", max(0, r0 - W + 1), rows)
    return out


def test_streaming_tiles_cover_what_is_visible():
    rng = np.random.default_rng(0)
    for _ in range(3000):
        S, W = int(rng.integers(0, 300)), int(rng.integers(1, 600))
        length, n = int(rng.integers(0, 1500)), int(rng.integers(1, 900))
        npos = 2 * (128 // int(rng.choice([1, 2, 3, 4, 5, 8, 16])))
        r0 = npos * int(rng.integers(0, -(-n // npos)))
        rows = min(r0 + npos, n)
        tiles = tiles_of(r0, rows, length, S, W)
        assert len(tiles) == len(set(tiles)) and len(tiles) >= 1
        want = set()
        for i in {length + r0, length + rows - 1}:
            for p in range(max(0, i - W + 1), i + 1):
                want.add(("chunk", (p - length) // 128) if p >= length else
                         ("slots", (p if p < S else S + p % W) // 128))
            for p in range(0, min(S, i + 1)):
                want.add(("chunk", (p - length) // 128) if p >= length else ("slots", p // 128))
        assert want <= set(tiles), (S, W, length, n, r0)


def deal(items, sms):
    """The host's dealing of items [(tiles, cost of one)]: (whole, ctas, shares, cuts), a share
    (item, tile, tiles, part) per CTA, a cut (item, pieces, part0, part1)."""
    piece = 16
    cost = [t * c + piece for t, c in items]
    n, tiles = len(items), sum(t for t, _ in items)
    ctas = min(sms, 148, tiles)
    even = -(-sum(cost) // ctas)
    while True:
        load, u = [0] * ctas, 0
        while u + ctas <= n and all(load[c] + cost[u + c] <= even for c in range(ctas)):
            for c in range(ctas):
                load[c] += cost[u + c]
            u += ctas
        whole, shares, cuts, rank, t0 = u, [(0, 0, 0, 0)] * ctas, [], 0, 0
        for c in range(ctas):
            if u >= n:
                break
            room, first, tile, got = even - load[c], u, t0, 0
            while u < n:
                rest = items[u][0] - t0
                can = int((room - piece) / items[u][1])  # towards zero
                if can < 1:
                    break
                take = min(rest, can)
                if t0 > 0:
                    cuts[-1][1] += 1
                elif take < rest:
                    cuts.append([u, 1, 2 * rank + (first != u), 2 * (rank + 1)])
                got += take
                room -= take * items[u][1] + piece
                t0 += take
                if t0 < items[u][0]:
                    break
                u, t0 = u + 1, 0
            shares[c] = (first, tile, got, 2 * rank)
            rank += got > 0
        if u == n:
            return whole, ctas, shares, cuts
        even += max(1, (sum(cost[u:]) - t0 * items[u][1]) // ctas, even // 128)


def test_dealing_covers_every_tile_once():
    """Every tile of every item goes to one CTA; the pieces of a cut item have places of their
    own, found in order at part0, part1, part1 + 2, ...; few places, whole items in rounds."""
    rng = np.random.default_rng(1)
    for _ in range(400):
        n = int(rng.choice([1, 2, 5, 40, 148, 149, 600]))
        top = int(rng.choice([1, 2, 7, 60, 1000]))
        items = sorted(((int(rng.integers(1, top + 1)), int(rng.choice([4, 5]))) for _ in range(n)), reverse=True)
        sms = int(rng.choice([1, 3, 132, 148, 160]))
        whole, ctas, shares, cuts = deal(items, sms)
        assert 1 <= ctas <= min(sms, 148) and whole % ctas == 0 and whole <= n and len(cuts) <= ctas
        pieces = {u: [(0, items[u][0], -1)] for u in range(whole)}
        for first, tile, left, part in shares:  # as the kernel walks them
            u, j = first, tile
            while left > 0:
                nt = min(items[u][0] - j, left)
                pieces.setdefault(u, []).append((j, nt, -1 if nt == items[u][0] else part + (u != first)))
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
            parts = [p for _, _, p in pieces[u]]
            if len(parts) > 1:
                _, count, part0, part1 = by_item[u]
                assert parts == [part0] + [part1 + 2 * i for i in range(count - 1)]
            else:
                assert parts == [-1] and u not in by_item


# ---------------------------------------------------------------- host side

def _prefill(h, layer, seqs, n, q=Q, k=K, v=V, out=OUT, lse=None):
    return duo.duo_pool_prefill(h, layer, seqs, n, q, k, v, out, lse)


def test_prefill_bookkeeping(dry_run):
    """Lengths advance by each sequence's own count on the one layer; pages are taken when a
    sequence first needs them, on whichever layer, and every page once."""
    h = _pool(num_pages=20, max_len=1500)
    a, b, c = (duo.duo_pool_open(h)[1] for _ in range(3))
    assert _prefill(h, 0, [b, a, c], [130, 1, 256]) == duo.DUO_OK
    assert [duo.duo_pool_len(h, s, 0)[1] for s in (a, b, c)] == [1, 130, 256]
    assert [duo.duo_pool_len(h, s, 1)[1] for s in (a, b, c)] == [0, 0, 0]
    assert _free(h) == 20 - 1 - 2 - 2
    assert _prefill(h, 1, [a, b, c], [1, 130, 256]) == duo.DUO_OK and _free(h) == 15
    assert _prefill(h, 0, [c], [1]) == duo.DUO_OK and _free(h) == 14
    pages = [p for s in (a, b, c) for p in _listed(h, s)]
    assert len(set(pages)) == len(pages) == 6
    # a fork's chunk takes pages of its own
    (d,) = duo.duo_pool_fork(h, b, 1)[1]
    assert _prefill(h, 0, [d, b], [200, 3]) == duo.DUO_OK
    assert not set(_listed(h, d)[1:]) & set(_listed(h, b)[1:]) and _listed(h, d)[0] == _listed(h, b)[0]
    duo.duo_pool_destroy(h)


def test_prefill_refusals_change_nothing(dry_run):
    h = _pool(num_pages=6, max_len=700)
    a, b = duo.duo_pool_open(h)[1], duo.duo_pool_open(h)[1]
    _fill(h, a, [100, 100])
    I, C = duo.DUO_ERR_INVALID, duo.DUO_ERR_CAPACITY
    lib, arr = duo.lib(), (duo.ctypes.c_int * 1)(a)
    one = (duo.ctypes.c_int * 1)(1)
    for st, call in [
            (I, lambda: _prefill(h, 2, [a], [1])), (I, lambda: _prefill(h, -1, [a], [1])),
            (I, lambda: _prefill(h, 0, [], [])), (I, lambda: _prefill(h, 0, [a, a], [1, 1])),
            (I, lambda: _prefill(h, 0, [a, 3], [1, 1])), (I, lambda: _prefill(h, 0, [-1], [1])),
            (I, lambda: _prefill(h, 0, [a], [0])), (I, lambda: _prefill(h, 0, [a, b], [1, -5])),
            (I, lambda: _prefill(h, 0, [a], [300000])), (I, lambda: _prefill(h, 0, list(range(129)), [1] * 129)),
            (I, lambda: _prefill(h, 0, [a], [1], q=None)), (I, lambda: _prefill(h, 0, [a], [1], v=V + 8)),
            (I, lambda: _prefill(h, 0, [a], [1], out=OUT + 4)), (I, lambda: _prefill(h, 0, [a], [1], lse=LSE + 2)),
            (I, lambda: _prefill(None, 0, [a], [1])),
            # results over inputs, one another or the pool
            (I, lambda: _prefill(h, 0, [a], [1], out=Q)), (I, lambda: _prefill(h, 0, [a, b], [3, 2], out=K + 512)),
            (I, lambda: _prefill(h, 0, [a], [1], out=V - 16)), (I, lambda: _prefill(h, 0, [a], [1], lse=OUT + 16)),
            (I, lambda: _prefill(h, 0, [a], [1], lse=V)), (I, lambda: _prefill(h, 0, [a], [1], out=POOL + 4096)),
            (I, lambda: _prefill(h, 0, [a], [1], q=POOL, lse=POOL + 8192)),
            (I, lambda: lib.duo_pool_prefill(h, 0, 1, None, one, Q, K, V, OUT, None, None)),
            (I, lambda: lib.duo_pool_prefill(h, 0, 1, arr, None, Q, K, V, OUT, None, None)),
            (C, lambda: _prefill(h, 0, [a], [601])), (C, lambda: _prefill(h, 0, [a, b], [500, 200])),
            (duo.DUO_ERR_CUDA, lambda: _fail(0, lambda: _prefill(h, 0, [a, b], [200, 300]))),
            (duo.DUO_ERR_CUDA, lambda: _fail(1, lambda: _prefill(h, 0, [a, b], [200, 300])))]:
        assert call() == st
        assert _free(h) == 5 and duo.duo_pool_len(h, a, 0)[1] == 100 and duo.duo_pool_len(h, b, 0)[1] == 0
    assert _prefill(h, 0, [a, b], [200, 300]) == duo.DUO_OK and _free(h) == 0
    duo.duo_pool_destroy(h)


# ---------------------------------------------------------------- on the GPU

def attended(q, k, v, retrieval, S, W, pos0, out, lse, pick, scale, what):
    """out and lse of query tokens (all, or the listed ones) against the fp64 oracle.  Element
    by element: the weights p are rounded to bf16 for the tensor core (half a step, 2^-8, of
    each term: 2^-8 sum p |v|) and the result once more (2^-8 |out|).  Everything else is
    fp32: a logit is a sum of 128 exact products, off by at most 128 * 2^-24 sum |q k| scale
    (the sum is below 160 for normal inputs), which is 2^-12 relative to its weight at most;
    the sum of weights adds (tiles + 64) 2^-24, below 5e-5."""
    n, Hq, _ = q.shape
    rows = None if pick is None else [r * Hq + h for r in pick for h in range(Hq)]
    args = dict(pos0=pos0, scale=scale, rows=rows)
    w, wl = oracle.attend(bits(q[None]), bits(k[None]), bits(v[None]), retrieval, S, W, **args)
    size, _ = oracle.attend(bits(q[None]), bits(k[None]), bits(v[None].abs()), retrieval, S, W, **args)
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    if pick is not None:
        o, l = o[pick], l[pick]
    w, size, wl = (x.reshape(y.shape) for x, y in ((w, o), (size, o), (wl, l)))
    off = np.abs(o - w) / (2.0 ** -8 * np.abs(w) + (2.0 ** -8 + 2.0 ** -12) * size + 1e-30)
    assert off.max() <= 1, f"{what}: {off.max()} of the tolerance at {np.unravel_index(off.argmax(), off.shape)}"
    off = np.abs(l - wl).max()
    assert off <= 128 * 2.0 ** -24 * 160 * (scale or 128 ** -0.5) + 5e-5, f"{what}: lse off by {off}"
    assert_close(o, w, torch.bfloat16, l, wl, what)


class Tokens:
    """Sequences of a pool with every token they hold, for the oracle."""

    def __init__(self, pool, seed):
        self.pool, self.seed, self.kv = pool, seed, {}

    def draw(self, n, heads):
        self.seed += 1
        return inputs.randn((n, heads, 128), self.seed, device=DEV)

    def open(self, length=0):
        s = self.pool.open()
        self.kv[s] = [(self.draw(length, self.pool.kv_heads), self.draw(length, self.pool.kv_heads))
                      for _ in range(self.pool.layers)]
        for layer, (k, v) in enumerate(self.kv[s]):
            if length:
                self.pool.append_kv(layer, s, k, v)
        return s

    def fork(self, s, n=1):
        kids = self.pool.fork(s, n)
        for c in kids:
            self.kv[c] = list(self.kv[s])
        return kids

    def prefill(self, layer, seqs, n, rows=None, scale=None):
        """One call, checked against the oracle (all rows, or `rows` of each sequence)."""
        pool, T = self.pool, sum(n)
        q, k, v = (self.draw(T, h) for h in (pool.q_heads, pool.kv_heads, pool.kv_heads))
        out, lse = pool.prefill(layer, seqs, n, q, k, v)
        at = 0
        for s, m in zip(seqs, n):
            kk, vv = self.kv[s][layer]
            pos0 = kk.shape[0]
            kk, vv = torch.cat((kk, k[at:at + m])), torch.cat((vv, v[at:at + m]))
            self.kv[s][layer] = (kk, vv)
            pick = None if rows is None or m <= rows else sorted(
                {0, m - 1} | set(np.random.default_rng(s).integers(0, m, rows - 2).tolist()))
            self.check(layer, q[at:at + m], kk, vv, pos0, out[at:at + m], lse[at:at + m], pick, scale,
                       f"sequence {s}: {m} on {pos0}, layer {layer}")
            at += m
        return out, lse

    def check(self, layer, q, k, v, pos0, out, lse, pick, scale, what):
        pool = self.pool
        attended(q, k, v, pool.mask[layer].numpy().astype(bool), pool.S, pool.W, pos0, out, lse, pick, scale, what)

    def check_cache(self):
        for s, layers in self.kv.items():
            k = torch.nn.utils.rnn.pad_sequence([x[0] for x in layers], batch_first=True)
            v = torch.nn.utils.rnn.pad_sequence([x[1] for x in layers], batch_first=True)
            check_rows(self.pool, s, k, v, [x[0].shape[0] for x in layers])


def _gpu_pool(Hq, Hkv, mask, S, W, max_seqs=12, max_len=4000, num_pages=200, layers=1, **kw):
    return DuoPool(layers, Hkv, [mask] * layers if not torch.is_tensor(mask) else mask, S, W, max_seqs, max_len,
                   num_pages, q_heads=Hq, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("S,W", [(4, 40), (0, 1), (0, 128), (1, 129), (130, 300), (16, 512)])
@pytest.mark.parametrize("Hq,mask", [(8, [1, 0]), (2, [0, 1]), (15, [1, 0, 0]), (16, [0]), (16, [1])])
def test_prefill_ragged_small(Hq, mask, S, W):
    """Prompts, continued chunks, single tokens and drafts together, around pages, tiles and
    a wrapping ring; several calls on the same sequences."""
    tk = Tokens(_gpu_pool(Hq, len(mask), mask, S, W), 1000)
    seqs = [tk.open(x) for x in (0, 1, 127, 128, 129, 600, 1500, 0)]
    tk.prefill(0, seqs, [1, 300, 1, 64, 129, 33, 5, 700], rows=40)
    tk.prefill(0, seqs[::-1], [1, 1, 130, 2, 17, 256, 128, 3], rows=40)
    tk.prefill(0, seqs[2:4], [255, 1], rows=40)
    tk.check_cache()
    assert tk.pool.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 11, 12, 13, 16])
def test_prefill_group_sizes(G):
    """Groups that divide a tile's 128 rows and groups that leave rows idle."""
    tk = Tokens(_gpu_pool(2 * G, 2, [1, 0], 4, 60), 2000 + G)
    seqs = [tk.open(x) for x in (0, 200, 77)]
    tk.prefill(0, seqs, [300, 1, 128 // G * 2 + 1], rows=64)
    tk.check_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("length,n", [(20000, [64]), (20000, [1]), (30011, [130]), (9000, [7, 3, 500]), (700, [2])])
def test_prefill_split_over_keys(length, n):
    """Few queries over a long history: keys split over CTAs and joined."""
    tk = Tokens(_gpu_pool(32, 8, [1, 0, 1, 0, 0, 1, 1, 0], 16, 512, max_len=40000, num_pages=1200), 3000)
    seqs = [tk.open(length // (i + 1)) for i in range(len(n))]
    out1, lse1 = tk.prefill(0, seqs, n, rows=8)
    tk.prefill(0, seqs, n, rows=8)
    tk.check_cache()


@pytest.mark.gpu
def test_prefill_long_chunk():
    """A chunk of many CTAs on a history, sampled rows; then its continuation."""
    tk = Tokens(_gpu_pool(32, 8, [1, 0, 1, 0, 0, 1, 1, 0], 16, 512, max_len=20000, num_pages=300), 3500)
    s, t = tk.open(5000), tk.open(0)
    tk.prefill(0, [s, t], [4097, 1000], rows=24)
    tk.prefill(0, [t, s], [2000, 1111], rows=24)
    tk.check_cache()


@pytest.mark.gpu
def test_prefill_many_sequences():
    """128 sequences in one call, most of one token; then all again."""
    tk = Tokens(_gpu_pool(8, 2, [1, 0], 4, 60, max_seqs=128, max_len=900, num_pages=500), 7000)
    seqs = [tk.open(x) for x in np.random.default_rng(3).integers(0, 400, 128).tolist()]
    n = [1 + (i % 7 == 0) * i for i in range(128)]
    tk.prefill(0, seqs, n, rows=4)
    tk.prefill(0, seqs[::-1], n, rows=4)
    tk.check_cache()


@pytest.mark.gpu
def test_prefill_many_heads():
    """As many KV heads as a pool takes, every third one a retrieval head."""
    tk = Tokens(_gpu_pool(128, 128, [int(h % 3 == 0) for h in range(128)], 2, 33, max_len=700, num_pages=20), 7500)
    seqs = [tk.open(x) for x in (0, 300)]
    tk.prefill(0, seqs, [150, 41], rows=3)
    tk.check_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("mask", [[1], [0]])
def test_prefill_largest_call(mask):
    """The most tokens that one call takes, one query head: 1024 items, sampled rows."""
    tk = Tokens(_gpu_pool(1, 1, mask, 16, 512, max_len=262144 + 40, num_pages=2050, max_seqs=2), 8000)
    s = tk.open(37)
    tk.prefill(0, [s], [262144], rows=12)
    assert tk.pool.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mask,replays", [([1, 0, 1, 0], 1), ([1, 1, 1, 1], 3)])
def test_prefill_on_another_stream_and_captured(mask, replays):
    """The call on a stream of the caller's and inside a captured graph, replayed, gives what
    it gives eagerly: outputs and rows.  (With streaming heads a second replay would start
    from rings in which the first has already replaced the oldest tokens; retrieval rows
    are only written again.)"""
    tk = Tokens(_gpu_pool(16, 4, mask, 4, 100, max_len=9000, num_pages=300), 9000)
    s = tk.open(5000)
    a, b, c = tk.fork(s, 3)
    q, k, v = tk.draw(75, 16), tk.draw(75, 4), tk.draw(75, 4)
    want = tk.pool.prefill(0, [a], [75], q, k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tk.pool.prefill(0, [b], [75], q, k, v, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.zeros_like(q), torch.zeros(75, 16, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tk.pool.prefill(0, [c], [75], q, k, v, out=out, lse=lse)
    for _ in range(replays):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for x in (a, b, c):
        kk, vv = tk.kv[x][0]
        tk.kv[x][0] = (torch.cat((kk, k)), torch.cat((vv, v)))
    tk.check_cache()
    assert tk.pool.device_status() == 0


@pytest.mark.gpu
def test_prefill_wait_runs_out_and_the_pool_goes_on():
    """A pre-fill whose softmax waits for what never comes reports the timeout after about the
    wait limit, frees what it holds, and the pool's other sequences go on as before."""
    tk = Tokens(_gpu_pool(32, 8, [1, 0, 1, 0, 0, 1, 1, 0], 16, 512, max_len=9000, num_pages=300), 9700)
    s, t = tk.open(3000), tk.open(100)
    (c,) = tk.pool.fork(s)
    q, k, v = tk.draw(900, 32), tk.draw(900, 8), tk.draw(900, 8)
    assert tk.pool.device_status() == duo.DUO_OK
    assert duo.duo_debug_device_stall(1) == duo.DUO_OK
    try:
        t0 = time.perf_counter()
        tk.pool.prefill(0, [c], [900], q, k, v)
        status = tk.pool.device_status()
        seconds = time.perf_counter() - t0
    finally:
        assert duo.duo_debug_device_stall(0) == duo.DUO_OK
    assert status == duo.DUO_ERR_TIMEOUT and 1.0 < seconds < 60.0, (status, seconds)
    assert tk.pool.device_status() == duo.DUO_OK
    tk.pool.close_seq(c)
    tk.prefill(0, [t, s], [700, 900], rows=8)
    tk.check_cache()
    assert tk.pool.device_status() == duo.DUO_OK


@pytest.mark.gpu
def test_calls_back_to_back():
    """Norms, pre-fills, forks, decodes and copies right behind one another (each launch's
    start overlaps the one before) give what they give with a wait after every call."""
    Hq, Hkv, mask = 16, 4, [1, 0, 1, 0]

    def run(wait):
        done = torch.cuda.synchronize if wait else (lambda: None)
        pool, to = (_gpu_pool(Hq, Hkv, mask, 4, 100, max_len=8000, num_pages=300) for _ in range(2))
        rope = DuoRope(128, freqs(128))
        outs, seqs = [], [pool.open() for _ in range(3)]
        for step in range(6):
            n = [700 + 150 * step, 130, 5 + step]
            x = inputs.randn((sum(n), Hq + 2 * Hkv, 128), 9100 + step, device=DEV)
            q, k, v = x.split((Hq, Hkv, Hkv), 1)
            pos = torch.arange(sum(n), dtype=torch.int32, device=DEV)
            done()
            q, k, v = rope.norm_rope(q, k, pos, v=v)
            done()
            outs += pool.prefill(0, seqs, n, q, k, v)
            done()
            kids = pool.fork(seqs[step % 3], 2)
            done()
            q, k, v = (inputs.randn((1, 5, h, 128), 9200 + 10 * step + i, device=DEV)
                       for i, h in enumerate((Hq, Hkv, Hkv)))
            done()
            outs += pool.decode_step(0, 1, seqs + kids, q, k, v)
            done()
            moved = pool.copy(kids[0], to)
            done()
            outs += to.prefill(0, [moved], [5], *(t[0] for t in (q, k, v)))
            done()
            outs += pool.decode_step(0, 1, kids, *(t[:, :2].contiguous() for t in (q, k, v)))
            done()
            for c in kids:
                pool.close_seq(c)
        assert pool.device_status() == 0 and to.device_status() == 0
        return [t.clone() for t in outs]

    waited = run(True)
    for _ in range(3):
        for i, (a, b) in enumerate(zip(run(False), waited)):
            assert torch.equal(a, b), f"output {i} differs"


@pytest.mark.gpu
def test_two_pools_on_two_streams():
    """Calls on two pools at the same time, each on a stream of its own."""
    made = [Tokens(_gpu_pool(16, 4, [1, 0, 1, 0], 4, 100, max_len=9000, num_pages=200), 9500 + i) for i in range(2)]
    x = [[t.draw(400, h) for h in (16, 4, 4)] for t in made]
    seqs = [t.open(3000 + 500 * i) for i, t in enumerate(made)]
    alone, kids = [], []
    for t, s, (q, k, v) in zip(made, seqs, x):
        kids.append(t.pool.fork(s, 4))
        alone.append(t.pool.prefill(0, kids[-1][:1], [400], q, k, v))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in made], [[], []]
    for j in range(1, 4):
        for i, t in enumerate(made):
            got[i].append(t.pool.prefill(0, kids[i][j:j + 1], [400], *x[i], stream=streams[i]))
    torch.cuda.synchronize()
    for want, rows in zip(alone, got):
        for out, lse in rows:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_prefill_repeats_bit_for_bit():
    """The same call on forks of the same sequence gives the same bits, alone or beside
    others (the split may differ then: alone twice), and whatever a neighbour holds."""
    tk = Tokens(_gpu_pool(16, 4, [1, 0, 1, 0], 4, 100, max_len=9000, num_pages=400), 4000)
    s = tk.open(6000)
    a, b = tk.fork(s, 2)
    q, k, v = tk.draw(50, 16), tk.draw(50, 4), tk.draw(50, 4)
    o1 = tk.pool.prefill(0, [a], [50], q, k, v)
    o2 = tk.pool.prefill(0, [b], [50], q, k, v)
    assert torch.equal(o1[0], o2[0]) and torch.equal(o1[1], o2[1])
    # a neighbour of NaN and infinities, on either side
    c, d, e = tk.fork(s, 3)
    bad = torch.full((37, 4, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    bad[::2] = float("inf")
    qq = torch.cat((tk.draw(37, 16), q, tk.draw(37, 16)))
    good = tk.pool.prefill(0, [d, c, e], [37, 50, 37], qq, torch.cat((tk.draw(37, 4), k, tk.draw(37, 4))),
                           torch.cat((tk.draw(37, 4), v, tk.draw(37, 4))))
    for x in (d, c, e):
        tk.pool.close_seq(x)
    c, d, e = tk.fork(s, 3)
    broken = tk.pool.prefill(0, [d, c, e], [37, 50, 37], qq, torch.cat((bad, k, bad)), torch.cat((bad, v, bad)))
    assert torch.equal(good[0][37:87], broken[0][37:87]) and torch.equal(good[1][37:87], broken[1][37:87])
    assert bool(broken[0][87:].isnan().any())


@pytest.mark.gpu
def test_prefill_writes_its_rows_only():
    """Rows around out and lse keep their values; a scale of the caller's; no lse asked."""
    tk = Tokens(_gpu_pool(10, 2, [1, 0], 4, 60, softmax_scale=0.3), 5000)
    s = tk.open(300)
    (c,) = tk.fork(s)
    q, k, v = tk.draw(70, 10), tk.draw(70, 2), tk.draw(70, 2)
    big = torch.full((72, 10, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    big_lse = torch.full((72, 10), 7.0, device=DEV)
    tk.pool.prefill(0, [s], [70], q, k, v, out=big[1:71], lse=big_lse[1:71])
    out, lse = tk.pool.prefill(0, [c], [70], q, k, v, want_lse=False)
    assert lse is None and torch.equal(out, big[1:71])
    for x in (big, big_lse):
        assert bool((x[0] == 7).all()) and bool((x[71] == 7).all())
    kk, vv = (torch.cat((x, y)) for x, y in zip(tk.kv[s][0], (k, v)))
    tk.check(0, q, kk, vv, 300, out, big_lse[1:71], None, 0.3, "scale 0.3")
    with pytest.raises(ValueError):
        tk.pool.prefill(0, [s], [70], q[:69], k, v)
    with pytest.raises(ValueError):
        tk.pool.prefill(0, [s], [70], q, k.float(), v)
    with pytest.raises(ValueError):
        tk.pool.prefill(0, [s], [70, 1], q, k, v)
    with pytest.raises(duo.DuoError):
        tk.pool.prefill(0, [s, s], [35, 35], q, k, v)


@pytest.mark.gpu
def test_serving_run():
    """The operators as a server uses them: projection rows normed and rotated, a prompt
    pre-filled in chunks on every layer, forked, drafts checked in the forks, one of them
    dropped, the other moved to a larger pool, decoded there."""
    layers, Hq, Hkv, S, W = 2, 8, 4, 4, 50
    mask = inputs.retrieval_mask(layers, Hkv, 2, seed=9)
    pool = _gpu_pool(Hq, Hkv, mask, S, W, layers=layers, num_pages=12, max_len=900)
    f = freqs(128)
    rope = DuoRope(128, f)
    wq, wk = (1 + 0.1 * inputs.randn((128,), x, device=DEV) for x in (61, 62))
    kv, seed = {}, [6000]

    def project(seq, n):
        seed[0] += 1
        x = inputs.randn((n, Hq + 2 * Hkv, 128), seed[0], device=DEV)
        q, k, v = x.split((Hq, Hkv, Hkv), 1)
        at = 0 if seq is None else kv[seq][0][0].shape[0]
        pos = torch.arange(at, at + n, dtype=torch.int32, device=DEV)
        got = rope.norm_rope(q, k, pos, v=v, q_weight=wq, k_weight=wk)
        want, size = reference(k, wk, 1e-6, pos[None], f, [0] * 64, False, 1.0)
        assert bool(((got[1].double() - want).abs() <= 2.0 ** -8 * want.abs() + 40 * 2.0 ** -24 * size).all())
        return got

    def step(seq, layer, q, k, v, out, lse):
        kk, vv = kv[seq][layer]
        pos0 = kk.shape[0]
        kv[seq][layer] = (torch.cat((kk, k)), torch.cat((vv, v)))
        attended(q, *kv[seq][layer], mask[layer].numpy().astype(bool), S, W, pos0, out, lse, None, None,
                 f"sequence {seq}, layer {layer}")

    s = pool.open()
    none = torch.empty(0, Hkv, 128, dtype=torch.bfloat16, device=DEV)
    kv[s] = [(none, none)] * layers
    for n in (200, 190):
        x = [project(s, n) for _ in range(layers)]
        for layer in range(layers):
            step(s, layer, *x[layer], *pool.prefill(layer, [s], [n], *x[layer]))
    a, b = pool.fork(s, 2)
    kv[a], kv[b] = list(kv[s]), list(kv[s])
    for layer in range(layers):
        xa, xb = project(a, 3), project(b, 5)
        out, lse = pool.prefill(layer, [a, b], [3, 5], *(torch.cat(p) for p in zip(xa, xb)))
        step(a, layer, *xa, out[:3], lse[:3])
        step(b, layer, *xb, out[3:], lse[3:])
        # the next layer's rows are at the same positions: take back the count for project()
        if layer == 0:
            tail = kv[a][0], kv[b][0]
            kv[a][0], kv[b][0] = kv[a][1], kv[b][1]
    kv[a][0], kv[b][0] = tail
    pool.close_seq(a)
    pool.close_seq(s)
    to = _gpu_pool(Hq, Hkv, mask, S, W, layers=layers, num_pages=30, max_len=3000, max_seqs=2)
    t = pool.copy(b, to)
    pool.close_seq(b)
    assert pool.free_pages() == 12
    kv = {t: kv[b]}
    for _ in range(2):
        x = [project(t, 1) for _ in range(layers)]
        q, k, v = (torch.stack(p) for p in zip(*x))
        o, lse = to.decode_step(0, layers, [t], q, k, v)
        for layer in range(layers):
            step(t, layer, *x[layer], o[layer], lse[layer])
    assert pool.device_status() == 0 and to.device_status() == 0
