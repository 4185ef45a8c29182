"""Sequences that branch and move (duo_pool_fork, duo_pool_copy): page accounting and
refusals on the CPU with launches skipped; cached rows bit for bit and decoding of parents
and children against the fp64 oracle on the GPU."""
import numpy as np
import pytest
import torch

import oracle
from head_split_kv_duo_b200 import duo, inputs
from head_split_kv_duo_b200.duo import DuoPool
from parity import assert_close, bits

FAKE = 1 << 40
DEV = "cuda"


@pytest.fixture
def dry_run():
    assert duo.duo_debug_launch_controls(1, -1) == duo.DUO_OK
    yield
    assert duo.duo_debug_launch_controls(0, -1) == duo.DUO_OK


def _pool(layers=2, Hkv=4, Hq=8, mask=None, S=4, W=16, max_seqs=6, max_len=1000, num_pages=20):
    if mask is None:
        mask = np.array([[1, 0, 1, 0]] * layers, dtype=np.uint8)
    opts = duo._opts(q_heads=Hq)
    need = duo.duo_pool_bytes(layers, Hkv, 128, mask, S, W, max_seqs, max_len, num_pages, opts)
    st, h = duo.duo_pool_create(layers, Hkv, 128, mask, S, W, max_seqs, max_len, num_pages, opts, FAKE, need)
    assert st == duo.DUO_OK
    return h


def _fill(h, seq, lens):
    for layer, n in enumerate(lens):
        if n:
            assert duo.duo_pool_append_kv(h, layer, seq, FAKE, FAKE, n) == duo.DUO_OK


def _listed(h, seq):
    pages = []
    while True:
        st, p = duo.duo_pool_page(h, seq, len(pages))
        if st != duo.DUO_OK:
            return pages
        pages.append(p)


def _free(h):
    return duo.duo_pool_free_pages(h)[1]


def _fail(n, call):
    assert duo.duo_debug_launch_controls(1, n) == duo.DUO_OK
    st = call()
    assert duo.duo_debug_launch_controls(1, -1) == duo.DUO_OK
    return st


# ---------------------------------------------------------------- host side

@pytest.mark.parametrize("lens,shared", [([0, 0], 0), ([1, 1], 0), ([128, 128], 1), ([300, 300], 2), ([300, 130], 1),
                                         ([300, 0], 0), ([511, 512], 3)])
def test_fork_shares_only_full_pages(dry_run, lens, shared):
    """Pages full on every layer are shared; the others are each child's own; every page
    returns exactly when the last sequence that lists it closes, in any order."""
    h = _pool(num_pages=30)
    s = duo.duo_pool_open(h)[1]
    _fill(h, s, lens)
    pages = _listed(h, s)
    assert len(pages) == -(-max(lens) // 128)
    free0 = _free(h)
    st, kids = duo.duo_pool_fork(h, s, 3)
    assert st == duo.DUO_OK and len(set(kids + [s])) == 4
    own = len(pages) - shared
    assert _free(h) == free0 - 3 * own
    held = list(pages)
    for c in kids:
        got = _listed(h, c)
        assert got[:shared] == pages[:shared] and len(got) == len(pages)
        held += got[shared:]
        assert [duo.duo_pool_len(h, c, layer)[1] for layer in range(2)] == lens
    assert len(set(held)) == len(held)
    # a child forks too; the parent closes first: shared pages stay
    st, (grand,) = duo.duo_pool_fork(h, kids[0], 1)
    assert st == duo.DUO_OK and _listed(h, grand)[:shared] == pages[:shared]
    assert duo.duo_pool_close(h, s) == duo.DUO_OK
    assert _free(h) == free0 - 4 * own + own
    for c in [grand, kids[2], kids[0]]:
        assert duo.duo_pool_close(h, c) == duo.DUO_OK
    assert _free(h) == 30 - len(pages)
    assert duo.duo_pool_close(h, kids[1]) == duo.DUO_OK
    assert _free(h) == 30
    duo.duo_pool_destroy(h)


def test_forked_sequences_grow_apart(dry_run):
    """After a fork at a page boundary the next token of each takes a page of its own; in
    the middle of a page neither touches the other's page."""
    h = _pool(num_pages=12)
    s = duo.duo_pool_open(h)[1]
    _fill(h, s, [256, 256])
    c = duo.duo_pool_fork(h, s, 1)[1][0]
    free0 = _free(h)
    assert duo.duo_pool_decode_step(h, 0, 2, [s, c], FAKE, FAKE, FAKE, FAKE, None) == duo.DUO_OK
    assert _free(h) == free0 - 2
    a, b = _listed(h, s), _listed(h, c)
    assert a[:2] == b[:2] and a[2] != b[2]
    d = duo.duo_pool_fork(h, c, 1)[1][0]  # 257 tokens: page 2 is copied
    assert _listed(h, d)[:2] == b[:2] and _listed(h, d)[2] not in (a[2], b[2])
    assert duo.duo_pool_append_kv(h, 0, d, FAKE, FAKE, 200) == duo.DUO_OK
    assert duo.duo_pool_len(h, c, 0)[1] == 257 and duo.duo_pool_len(h, d, 0)[1] == 457
    duo.duo_pool_destroy(h)


def test_fork_refusals_change_nothing(dry_run):
    h = _pool(max_seqs=4, num_pages=5)
    s = duo.duo_pool_open(h)[1]
    _fill(h, s, [300, 300])  # 3 pages; 2 free
    for args, st in [((s, 0), duo.DUO_ERR_INVALID), ((s, -1), duo.DUO_ERR_INVALID), ((s, 129), duo.DUO_ERR_INVALID),
                     ((1, 1), duo.DUO_ERR_INVALID), ((-1, 1), duo.DUO_ERR_INVALID), ((99, 1), duo.DUO_ERR_INVALID),
                     ((s, 4), duo.DUO_ERR_CAPACITY), ((s, 3), duo.DUO_ERR_CAPACITY)]:
        assert duo.duo_pool_fork(h, *args)[0] == st, args
        assert _free(h) == 2
    assert duo.duo_pool_fork(None, 0, 1)[0] == duo.DUO_ERR_INVALID
    assert duo.lib().duo_pool_fork(h, s, 1, None, None) == duo.DUO_ERR_INVALID
    # a failed launch: no page and no slot is kept
    assert _fail(0, lambda: duo.duo_pool_fork(h, s, 2)[0]) == duo.DUO_ERR_CUDA
    assert _free(h) == 2
    assert duo.duo_pool_fork(h, s, 2) == (duo.DUO_OK, [1, 2])
    assert _free(h) == 0
    duo.duo_pool_destroy(h)


def test_fork_over_several_launches(dry_run):
    """More copied pages than one launch lists (layers of different lengths); a failure of
    the second launch leaves everything as it was."""
    h = _pool(num_pages=1000, max_len=200000, max_seqs=20)
    s = duo.duo_pool_open(h)[1]
    _fill(h, s, [128 * 200, 0])
    free0 = _free(h)
    assert _fail(1, lambda: duo.duo_pool_fork(h, s, 3)[0]) == duo.DUO_ERR_CUDA
    assert _free(h) == free0
    st, kids = duo.duo_pool_fork(h, s, 3)
    assert st == duo.DUO_OK and _free(h) == free0 - 600
    pages = [p for x in kids + [s] for p in _listed(h, x)]
    assert len(set(pages)) == 800
    duo.duo_pool_destroy(h)


def test_copy_host_side(dry_run):
    a, b = _pool(), _pool(max_seqs=1, num_pages=4, max_len=600)
    s = duo.duo_pool_open(a)[1]
    _fill(a, s, [300, 200])
    assert duo.duo_pool_copy(a, s, b) == (duo.DUO_OK, 0)
    assert _free(b) == 1 and [duo.duo_pool_len(b, 0, layer)[1] for layer in range(2)] == [300, 200]
    assert duo.duo_pool_copy(a, s, b)[0] == duo.DUO_ERR_CAPACITY  # no slot
    assert duo.duo_pool_close(b, 0) == duo.DUO_OK
    _fill(a, s, [230, 0])
    assert duo.duo_pool_copy(a, s, b)[0] == duo.DUO_ERR_CAPACITY and _free(b) == 4  # 5 pages
    _fill(a, s, [100, 0])
    assert duo.duo_pool_copy(a, s, b)[0] == duo.DUO_ERR_CAPACITY  # 630 tokens past max_len 600
    # within one pool nothing is shared
    free0 = _free(a)
    st, c = duo.duo_pool_copy(a, s, a)
    assert st == duo.DUO_OK and _free(a) == free0 - 5 and not set(_listed(a, s)) & set(_listed(a, c))
    assert _fail(0, lambda: duo.duo_pool_copy(a, s, a)[0]) == duo.DUO_ERR_CUDA
    assert _free(a) == free0 - 5
    # pools that do not match, closed sequences, null handles
    other = [_pool(layers=1), _pool(S=5), _pool(W=17), _pool(mask=np.array([[1, 0, 0, 1]] * 2, np.uint8)),
             _pool(Hkv=2, Hq=4, mask=np.array([[1, 0]] * 2, np.uint8))]
    for o in other:
        assert duo.duo_pool_copy(a, s, o)[0] == duo.DUO_ERR_INVALID
    assert duo.duo_pool_copy(a, 5, b)[0] == duo.DUO_ERR_INVALID
    assert duo.duo_pool_copy(None, 0, b)[0] == duo.DUO_ERR_INVALID
    assert duo.duo_pool_copy(a, s, None)[0] == duo.DUO_ERR_INVALID
    for x in [a, b] + other:
        duo.duo_pool_destroy(x)


def test_pages_come_lowest_first(dry_run):
    h = _pool(num_pages=10)
    a, b = duo.duo_pool_open(h)[1], duo.duo_pool_open(h)[1]
    _fill(h, a, [300, 0])
    _fill(h, b, [300, 0])
    assert _listed(h, a) == [0, 1, 2] and _listed(h, b) == [3, 4, 5]
    duo.duo_pool_close(h, a)
    _fill(h, b, [500, 0])
    assert _listed(h, b) == [3, 4, 5, 0, 1, 2, 6]
    duo.duo_pool_destroy(h)


def test_append_that_fails_on_the_way_keeps_the_other_layers_pages(dry_run):
    """An append of several launches whose second one fails: the pages that another, longer
    layer holds -- shared ones among them -- stay listed."""
    h = _pool(max_len=100000, num_pages=1200)
    s = duo.duo_pool_open(h)[1]
    _fill(h, s, [70000, 0])
    before, free = _listed(h, s), _free(h)
    assert len(before) == 547
    append = lambda seq, n: duo.duo_pool_append_kv(h, 1, seq, FAKE, FAKE, n)  # noqa: E731
    assert _fail(1, lambda: append(s, 40000)) == duo.DUO_ERR_CUDA
    assert duo.duo_pool_len(h, s, 1)[1] == 32512 and duo.duo_pool_len(h, s, 0)[1] == 70000
    assert _listed(h, s) == before and _free(h) == free
    # past the longer layer: only what the call itself took goes back
    assert _fail(1, lambda: append(s, 50000)) == duo.DUO_ERR_CUDA
    assert duo.duo_pool_len(h, s, 1)[1] == 65024 and _listed(h, s) == before and _free(h) == free
    duo.duo_pool_destroy(h)


# ---------------------------------------------------------------- on the GPU

def _tokens(layers, T, Hkv, seed):
    return (inputs.randn((layers, T, Hkv, 128), seed, device=DEV),
            inputs.randn((layers, T, Hkv, 128), seed + 1, device=DEV))


def _append(pool, seq, k, v, a, b):
    for layer in range(pool.layers):
        if b > a:
            pool.append_kv(layer, seq, k[layer, a:b].contiguous(), v[layer, a:b].contiguous())


def check_rows(pool, seq, k, v, lens):
    """The sequence's retrieval rows through its pages and its ring slots hold the tokens
    bit for bit; rows past its length and unwritten ring slots are zero."""
    for layer in range(pool.layers):
        n, mask = lens[layer], pool.mask[layer].bool()
        ridx, sidx = mask.nonzero()[:, 0].tolist(), (~mask).nonzero()[:, 0].tolist()
        slots = pool.S + pool.W
        replay = oracle.ring_replay(pool.S, pool.W, [n])[0] if n else -np.ones(slots, dtype=np.int64)
        at = torch.tensor(np.maximum(replay, 0), device=DEV)
        live = torch.tensor(replay >= 0, device=DEV)[None, :, None]
        for x, which_r, which_s in ((k, duo.DUO_REGION_RETR_K, duo.DUO_REGION_STRM_K),
                                    (v, duo.DUO_REGION_RETR_V, duo.DUO_REGION_STRM_V)):
            if ridx and n:
                pages = [pool.page(seq, i) for i in range(-(-n // 128))]
                got = pool.region(layer, which_r).view(torch.int16).view(pool.num_pages, len(ridx), 128, 128)[pages]
                got = got.transpose(1, 2).reshape(-1, len(ridx), 128)
                assert torch.equal(got[:n], x[layer, :n, ridx].view(torch.int16)), (seq, layer)
                assert not got[n:].any(), (seq, layer)
            if sidx:
                got = pool.region(layer, which_s).view(torch.int16).view(pool.max_seqs, len(sidx), slots, 128)[seq]
                src = x[layer][at][:, sidx] if n else torch.zeros(slots, len(sidx), 128, dtype=x.dtype, device=DEV)
                want = torch.where(live, src.transpose(0, 1).view(torch.int16), torch.zeros_like(got))
                assert torch.equal(got, want), (seq, layer)


@pytest.mark.gpu
@pytest.mark.parametrize("length", [0, 1, 5, 127, 128, 129, 300, 640])
@pytest.mark.parametrize("S,W,mask", [(4, 40, [1, 0, 1, 0]), (0, 200, [0, 0, 0, 1]), (130, 7, [0, 0, 0, 0]),
                                      (3, 3, [1, 1, 1, 1])])
def test_forked_rows_are_the_parents(S, W, mask, length):
    """Children hold the parent's tokens, in pages and rings that were somebody else's
    before; then parent and children go their own ways."""
    layers, Hkv, n = 2, 4, 3
    pool = DuoPool(layers, Hkv, [mask] * layers, S, W, 8, 800, 60, q_heads=8)
    pool.open()
    k0, v0 = _tokens(layers, 700, Hkv, 90)
    old = [pool.open() for _ in range(4)]
    for s in old:  # every slot and many pages are used ones
        _append(pool, s, k0, v0, 0, 700)
    for s in old:
        pool.close_seq(s)
    parent = pool.open()
    k, v = _tokens(layers, 800, Hkv, 92)
    _append(pool, parent, k, v, 0, length)
    kids = pool.fork(parent, n)
    for s in [parent] + kids:
        check_rows(pool, s, k, v, [length] * layers)
    own = []
    for i, s in enumerate([parent] + kids):
        kk, vv = _tokens(layers, 800, Hkv, 100 + 2 * i)
        kk[:, :length], vv[:, :length] = k[:, :length], v[:, :length]
        more = [1, 130, 3, 0][i]
        _append(pool, s, kk, vv, length, length + more)
        own.append((s, kk, vv, length + more))
    for s, kk, vv, m in own:
        check_rows(pool, s, kk, vv, [m] * layers)
    assert pool.device_status() == 0


@pytest.mark.gpu
def test_fork_with_layers_of_different_lengths():
    layers, Hkv = 3, 4
    lens = [300, 20, 129]
    pool = DuoPool(layers, Hkv, [[1, 0, 1, 0], [0, 1, 1, 1], [1, 1, 1, 1]], 2, 50, 4, 600, 30, q_heads=4)
    s = pool.open()
    k, v = _tokens(layers, 400, Hkv, 120)
    for layer, n in enumerate(lens):
        pool.append_kv(layer, s, k[layer, :n].contiguous(), v[layer, :n].contiguous())
    (c,) = pool.fork(s)
    to = DuoPool(layers, Hkv, pool.mask, 2, 50, 1, 400, 3, q_heads=4)
    d = pool.copy(s, to)
    check_rows(pool, s, k, v, lens)
    check_rows(pool, c, k, v, lens)
    check_rows(to, d, k, v, lens)
    for layer, n in enumerate(lens):  # the child grows to equal lengths; the parent stays
        pool.append_kv(layer, c, k[layer, n:310].contiguous(), v[layer, n:310].contiguous())
    check_rows(pool, c, k, v, [310] * 3)
    check_rows(pool, s, k, v, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("length", [1, 128, 1000, 90000])
def test_copied_rows(length):
    """To a larger pool, back into a pool that just fits, and within a pool (90000 tokens:
    more pages than one launch lists)."""
    Hkv = 2
    pages = -(-length // 128)
    a = DuoPool(1, Hkv, [[1, 0]], 4, 64, 2, length, 2 * pages, q_heads=2)
    s = a.open()
    k, v = _tokens(1, length, Hkv, 130)
    _append(a, s, k, v, 0, length)
    b = DuoPool(1, Hkv, [[1, 0]], 4, 64, 3, length + 500, pages + 9, q_heads=2)
    b.open()
    t = a.copy(s, b)
    c = a.copy(s, a)
    a.close_seq(s)
    back = b.copy(t, a)
    for pool, x in ((b, t), (a, c), (a, back)):
        check_rows(pool, x, k, v, [length])


@pytest.mark.gpu
def test_decoding_forks():
    """A prompt, its forks and forks of forks decode in one ragged batch, each against the
    oracle over its own tokens; closed and reopened slots in between."""
    layers, Hq, Hkv, S, W = 2, 16, 4, 4, 60
    mask = inputs.retrieval_mask(layers, Hkv, 2, seed=140)
    pool = DuoPool(layers, Hkv, mask, S, W, 8, 700, 40, q_heads=Hq)
    hist = {}

    def grow(seqs, steps, seed):
        for t in range(steps):
            q = inputs.randn((layers, len(seqs), Hq, 128), seed + 3 * t, device=DEV)
            k = inputs.randn((layers, len(seqs), Hkv, 128), seed + 3 * t + 1, device=DEV)
            v = inputs.randn((layers, len(seqs), Hkv, 128), seed + 3 * t + 2, device=DEV)
            o, lse = pool.decode_step(0, layers, seqs, q, k, v)
            for i, s in enumerate(seqs):
                kk, vv = hist[s]
                hist[s] = (torch.cat((kk, k[:, i:i + 1]), 1), torch.cat((vv, v[:, i:i + 1]), 1))
                for layer in range(layers):
                    kk, vv = hist[s]
                    w, wl = oracle.attend(bits(q[layer, i][None, None]), bits(kk[layer][None]), bits(vv[layer][None]),
                                          mask[layer].numpy().astype(bool), S, W, pos0=kk.shape[1] - 1)
                    assert_close(o[layer, i].float().cpu().numpy()[None], w[0], torch.bfloat16,
                                 lse[layer, i].cpu().numpy()[None], wl[0], f"sequence {s} layer {layer}")

    root = pool.open()
    k, v = _tokens(layers, 254, Hkv, 150)
    _append(pool, root, k, v, 0, 254)
    hist[root] = (k, v)
    a, b = pool.fork(root, 2)
    hist[a] = hist[b] = hist[root]
    grow([b, root, a], 3, 200)  # across a page boundary
    (c,) = pool.fork(b)
    hist[c] = hist[b]
    pool.close_seq(root)
    grow([a, c, b], 2, 300)
    pool.close_seq(b)
    d = pool.fork(c)[0]
    hist[d] = hist[c]
    grow([d, a, c], 2, 400)
    for s in (a, c, d):
        check_rows(pool, s, *hist[s], [hist[s][0].shape[1]] * layers)
    assert pool.device_status() == 0
