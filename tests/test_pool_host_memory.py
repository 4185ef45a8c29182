"""Pool calls that run out of host memory report it: no exception crosses the C boundary (it
would end the process), and nothing is taken.  Each case runs in a process of its own, whose
address space is limited right before the call; launches are skipped."""
import subprocess
import sys
import textwrap

import pytest

PRELUDE = """
import resource
import numpy as np
from head_split_kv_duo_b200 import duo
FAKE = 1 << 40
assert duo.duo_debug_launch_controls(1, -1) == duo.DUO_OK
opts = duo._opts(q_heads=1)
mask = np.zeros((1, 1), dtype=np.uint8)

def limit(more):
    used = int(open('/proc/self/statm').read().split()[0]) * resource.getpagesize()
    resource.setrlimit(resource.RLIMIT_AS, (used + more, resource.RLIM_INFINITY))

def unlimited():
    resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))

def create(num_pages, max_len, max_seqs=2):
    need = duo.duo_pool_bytes(1, 1, 128, mask, 4, 16, max_seqs, max_len, num_pages, opts)
    assert need > 0
    return lambda: duo.duo_pool_create(1, 1, 128, mask, 4, 16, max_seqs, max_len, num_pages, opts, FAKE, need)
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(code)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, f"{r.returncode}\n{r.stderr[-2000:]}"


@pytest.mark.parametrize("mebibytes", [512, 1536])
def test_create(mebibytes):
    """2^28 pages: 1 GiB for the free pages, 1 GiB for their counts; either may be what fails."""
    run(f"""
    make = create(1 << 28, 1000)
    limit({mebibytes} << 20)
    st, h = make()
    unlimited()
    assert st == duo.DUO_ERR_INVALID and not h, (st, h)
    """)


def test_append():
    """2^23 pages of one sequence are a list of 32 MiB."""
    run("""
    st, h = create(1 << 23, 1 << 30)()
    assert st == duo.DUO_OK
    s = duo.duo_pool_open(h)[1]
    free = duo.duo_pool_free_pages(h)[1]
    limit(4 << 20)
    st = duo.duo_pool_append_kv(h, 0, s, FAKE, FAKE, 1 << 30)
    unlimited()
    assert st == duo.DUO_ERR_INVALID, st
    assert duo.duo_pool_free_pages(h)[1] == free and duo.duo_pool_len(h, s, 0)[1] == 0
    assert duo.duo_pool_append_kv(h, 0, s, FAKE, FAKE, 300) == duo.DUO_OK
    assert duo.duo_pool_free_pages(h)[1] == free - 3
    """)


def test_decode_step():
    """A call whose own bookkeeping (a byte for each of 2^20 slots) does not fit."""
    run("""
    st, h = create(4, 300, 1 << 20)()
    assert st == duo.DUO_OK
    s = duo.duo_pool_open(h)[1]
    step, args = duo.lib().duo_pool_decode_step, (h, 0, 1, 1, (duo.ctypes.c_int * 1)(s), FAKE, FAKE, FAKE, FAKE, None, None)
    # use up what the allocator still holds
    kept = []
    limit(0)
    try:
        while True:
            kept.append(bytearray(1 << 19))
    except MemoryError:
        pass
    st = step(*args)
    unlimited()
    assert st == duo.DUO_ERR_INVALID, st
    assert duo.duo_pool_len(h, s, 0)[1] == 0 and duo.duo_pool_free_pages(h)[1] == 4
    assert step(*args) == duo.DUO_OK
    assert duo.duo_pool_len(h, s, 0)[1] == 1
    """)
