"""The block pool when host memory runs out: PA_ERR_OOM, nothing changed, no exception out of a C entry (it would end
the process).  In a process of its own whose address space is limited.  No GPU."""
import subprocess
import sys
import textwrap

import pytest

from paged_kv_cache_75_gb300 import build as pkg_build

START = """
import ctypes as C, resource, sys
L = C.CDLL(sys.argv[1])
def room(megabytes):
    used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
    resource.setrlimit(resource.RLIMIT_AS, (used + (megabytes << 20), resource.RLIM_INFINITY))
def pool(n, bs=1):
    h = C.c_void_p()
    return L.pa_pool_create(C.c_int64(n), bs, None, C.byref(h)), h
def seq(h, i):
    return L.pa_pool_add_seq(h, C.c_int64(i))
L.pa_pool_num_free.restype = C.c_int64
"""


def run(body):
    lib = pkg_build.build()
    r = subprocess.run([sys.executable, "-c", START + textwrap.dedent(body), lib], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.split()[-1:] == ["fine"], (r.returncode, r.stdout, r.stderr)


def test_create():
    run("""
        room(256)
        for n in (2 ** 31 - 1, 100_000_000):
            st, h = pool(n)
            assert st == 3 and h.value is None
        assert pool(1000)[0] == 0
        print("fine")
    """)


def test_append_and_fork():
    run("""
        N = 60_000_000
        st, h = pool(N)
        assert st == 0 and seq(h, 1) == 0
        n = 50_000_000
        slots = (C.c_int64 * n)()
        room(64)  # not what 50 million block ids take
        assert L.pa_pool_append(h, C.c_int64(1), n, slots, None, None) == 3
        assert L.pa_pool_num_free(h) == N and L.pa_pool_seq_len(h, C.c_int64(1)) == 0
        room(256)
        assert L.pa_pool_append(h, C.c_int64(1), n, slots, None, None) == 0
        assert slots[0] == 0 and slots[n - 1] == n - 1
        room(64)
        assert L.pa_pool_fork(h, C.c_int64(1), C.c_int64(2)) == 3
        assert L.pa_pool_seq_len(h, C.c_int64(2)) == -1 and L.pa_pool_ref_count(h, C.c_int64(0)) == 1
        # giving back allocates nothing
        assert L.pa_pool_free_seq(h, C.c_int64(1)) == 0 and L.pa_pool_num_free(h) == N
        print("fine")
    """)


def test_sequences():
    run("""
        st, h = pool(10)
        room(16)
        i = 0
        while (st := seq(h, i)) == 0:
            i += 1
            assert i < 10 ** 8
        assert st == 3 and L.pa_pool_seq_len(h, C.c_int64(i)) == -1 and L.pa_pool_seq_len(h, C.c_int64(i - 1)) == 0
        L.pa_pool_destroy(h)
        print("fine")
    """)


@pytest.mark.parametrize("n", [1, 7, 64])
def test_a_ring_many_times_round(n):
    """First in, first out, over many turns of the free list."""
    import random

    import paged_kv_cache_75_gb300 as pk

    rng = random.Random(n)
    p, free, held = pk.BlockPool(n, 1, free_order=list(reversed(range(n)))), list(reversed(range(n))), {}
    for step in range(3000):
        if free and (not held or rng.random() < 0.5):
            k = rng.randint(1, len(free))
            p.add_seq(step)
            slots, _ = p.append(step, k)
            held[step], free = free[:k], free[k:]
            assert slots == held[step]
        else:
            i = rng.choice(list(held))
            p.free_seq(i)
            free += held.pop(i)
        assert p.num_free() == len(free)
