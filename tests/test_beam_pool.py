"""pa_pool_reserve / pa_pool_reorder / pa_pool_unreserve: beams' blocks in the host pool.  No GPU."""
import ctypes as C
import random

import numpy as np
import pytest

import beam_ref as R
import paged_kv_cache_75_gb300 as pk
from oracle.pool_model import BlockPoolModel
from paged_kv_cache_75_gb300 import build as pkg_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg_build.build()


class Model(BlockPoolModel):
    """The pool model with reserved blocks and reordered beams."""

    def reserve(self, n):
        assert n <= len(self.free)
        return [self._take() for _ in range(n)]

    def give(self, blocks):
        for b in blocks:
            self.ref[b] -= 1
            if self.ref[b] == 0:
                self.free.append(b)

    def reorder(self, old, new, parents, spare):
        width = max([len(self.seqs[s][0]) for s in old] + [0]) + 1
        table = np.array([list(self.seqs[s][0]) + [-1] * (width - len(self.seqs[s][0])) for s in old], np.int32)
        t, lens, slots, used, _ = R.reorder(parents, table.reshape(len(old), width), [self.seqs[s][1] for s in old], spare,
                                            self.block_size)
        rows = [[int(b) for b in t[i, :-(-int(lens[i]) // self.block_size)]] for i in range(len(new))]
        for i, row in enumerate(rows):
            for b in row:
                if not (used[i] and b == spare[i]):
                    self.ref[b] += 1  # (a spare's one reference goes over to its sequence)
        for s in old:
            self.give(self.seqs.pop(s)[0])
        for i, s in enumerate(new):
            self.seqs[s] = [rows[i], int(lens[i])]
        return slots.tolist(), [bool(u) for u in used]


def same(pool, m):
    ids = sorted(m.seqs)
    t, lens = pool.block_table(ids, 200)
    for s, row, n in zip(ids, t, lens):
        assert row == m.seqs[s][0] + [-1] * (200 - len(m.seqs[s][0])) and n == m.seqs[s][1]
    assert pool.num_free() == len(m.free)
    assert all(pool.ref_count(b) == m.ref[b] for b in range(m.num_blocks))


@pytest.mark.parametrize("bs", [1, 3, 16])
@pytest.mark.parametrize("seed", range(4))
def test_against_the_model(bs, seed):
    rng = random.Random(100 * seed + bs)
    n = 400
    order = list(range(n))
    rng.shuffle(order)
    pool, m = pk.BlockPool(n, bs, free_order=order), Model(n, bs, free_order=order)
    beams, next_id = {}, 0
    for req in range(3):
        pool.add_seq(next_id)
        m.add_seq(next_id)
        prompt = rng.randint(0, 3 * bs)
        assert pool.append(next_id, prompt) == m.append(next_id, prompt)
        beams[req], next_id = [next_id], next_id + 1
    spares = []
    for step in range(60):
        req = rng.randrange(3)
        old = beams[req]
        w = rng.randint(1, 6)
        if rng.random() < 0.5:
            new = [next_id + i for i in range(w)]
        else:
            new = (old + [next_id + i for i in range(w)])[:w]
            rng.shuffle(new)
        next_id += w
        parents = [rng.randrange(len(old)) if rng.random() < 0.95 else -1 for _ in range(w)]
        if w > len(spares):
            more = w - len(spares)
            if more > len(m.free):
                break
            got = pool.reserve(more)
            assert got == m.reserve(more)
            spares += got
        now = spares[:w]
        slots, used = pool.reorder(old, new, parents, now)
        assert (slots, used) == m.reorder(old, new, parents, now)
        spares = [b for b, u in zip(now, used) if not u] + spares[w:]
        beams[req] = new
        same(pool, m)
        if rng.random() < 0.1 and len(spares) > 1:
            back = [spares.pop(), spares.pop(0)]
            pool.unreserve(back)
            m.give(back)
            same(pool, m)
    for old in beams.values():
        for s in old:
            pool.free_seq(s)
    pool.unreserve(spares)
    assert pool.num_free() == n


def refused(pool, code, f):
    free, refs = pool.num_free(), [pool.ref_count(b) for b in range(12)]
    with pytest.raises(pk.PaError) as e:
        f()
    assert e.value.status == code
    assert pool.num_free() == free and [pool.ref_count(b) for b in range(12)] == refs


def test_refusals_change_nothing():
    pool = pk.BlockPool(12, 4)
    pool.add_seq(7)
    pool.append(7, 6)
    pool.add_seq(8)
    a, b = pool.reserve(2)
    refused(pool, 3, lambda: pool.reserve(100))
    refused(pool, 1, lambda: pool.reserve(-1))
    refused(pool, 1, lambda: pool.unreserve([a, a]))
    refused(pool, 1, lambda: pool.unreserve([a, 0]))      # a sequence's block
    refused(pool, 1, lambda: pool.unreserve([12]))
    refused(pool, 1, lambda: pool.unreserve([-1]))
    refused(pool, 1, lambda: pool.reorder([9], [1], [0], [a]))             # unknown
    refused(pool, 1, lambda: pool.reorder([7, 7], [1], [0], [a]))          # twice
    refused(pool, 1, lambda: pool.reorder([7], [1, 1], [0, 0], [a, b]))
    refused(pool, 1, lambda: pool.reorder([7], [8], [0], [a]))             # another's id
    refused(pool, 1, lambda: pool.reorder([7], [1], [1], [a]))             # no such parent
    refused(pool, 1, lambda: pool.reorder([7], [1, 2, 3], [0, 0, 0], [a, b, b]))
    refused(pool, 1, lambda: pool.reorder([7], [1, 2], [0, 0], [a, 5]))    # not reserved
    refused(pool, 1, lambda: pool.reorder([7], [1, 2], [0, 0], [a, -1]))
    pool.fork(7, 70)
    refused(pool, 1, lambda: pool.reorder([7], [1], [0], [a]))             # the partly filled block is shared
    pool.free_seq(70)
    # the spare of a first child of a partly filled block is not looked at
    assert pool.reorder([7], [1, 2], [0, 0], [-5, b]) == ([1 * 4 + 2, b * 4 + 2], [False, True])
    assert pool.seq_len(7) == -1 and pool.seq_len(1) == 7 and pool.seq_len(8) == 0
    pool.unreserve([a])


def test_an_empty_parent_and_no_rows():
    pool = pk.BlockPool(8, 4)
    pool.add_seq(0)
    spare = pool.reserve(2)
    assert pool.reorder([0], [0, 1], [0, 0], spare) == ([4 * spare[0], 4 * spare[1]], [True, True])
    assert pool.reorder([0, 1], [], [], []) == ([], [])
    assert pool.num_free() == 8


def test_null_pointers():
    L = pk.library()
    pool = pk.BlockPool(4, 4)
    assert L.pa_pool_reserve(pool._h, 1, None) == 1 and L.pa_pool_reserve(None, 0, None) == 1
    assert L.pa_pool_unreserve(pool._h, None, 1) == 1
    ids = (C.c_int64 * 1)(0)
    assert L.pa_pool_reorder(pool._h, None, 1, None, 0, None, None, None, None) == 1
    assert L.pa_pool_reorder(pool._h, None, 0, ids, 1, None, None, None, None) == 1
    assert L.pa_pool_reorder(pool._h, None, 0, None, 0, None, None, None, None) == 0
