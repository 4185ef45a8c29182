"""Pre-fills on histories of tens of millions of tokens (launches skipped): a call in which one
CTA would work on a single piece for longer than the kernel's bounded waits allow is refused,
and changes nothing; calls of fewer tokens, whose items are cut, go through."""
import numpy as np
import pytest

from head_split_kv_duo_b200 import duo

FAKE = 2 << 40
Q, K, V, OUT = (FAKE + (i << 36) for i in range(4))


@pytest.fixture
def long_pool():
    """One retrieval head, one sequence of 2^27 tokens."""
    assert duo.duo_debug_launch_controls(1, -1) == duo.DUO_OK
    mask, opts = np.ones((1, 1), dtype=np.uint8), duo._opts(q_heads=1)
    args = (1, 1, 128, mask, 4, 16, 2, 1 << 28, (1 << 21) - 10, opts)
    st, h = duo.duo_pool_create(*args, 1 << 40, duo.duo_pool_bytes(*args))
    assert st == duo.DUO_OK
    s = duo.duo_pool_open(h)[1]
    yield h, s
    duo.duo_pool_destroy(h)
    assert duo.duo_debug_launch_controls(0, -1) == duo.DUO_OK


def _state(h, s):
    return duo.duo_pool_len(h, s, 0), duo.duo_pool_free_pages(h)


@pytest.mark.parametrize("length,n,status", [
    (1 << 27, 262144, duo.DUO_ERR_UNSUPPORTED), (1 << 27, 65536, duo.DUO_ERR_UNSUPPORTED),
    (1 << 27, 2048, duo.DUO_OK), (1 << 27, 1, duo.DUO_OK), (20_000_000, 262144, duo.DUO_ERR_UNSUPPORTED),
    (16_000_000, 262144, duo.DUO_OK), (100_000, 262144, duo.DUO_OK)])
def test_pieces_end_before_waits_do(long_pool, length, n, status):
    h, s = long_pool
    assert duo.duo_pool_append_kv(h, 0, s, FAKE, FAKE, length) == duo.DUO_OK
    before = _state(h, s)
    assert duo.duo_pool_prefill(h, 0, [s], [n], Q, K, V, OUT, None) == status
    if status == duo.DUO_OK:
        assert duo.duo_pool_len(h, s, 0) == (duo.DUO_OK, length + n)
    else:
        assert _state(h, s) == before
        assert duo.duo_pool_prefill(h, 0, [s], [512], Q, K, V, OUT, None) == duo.DUO_OK
