"""pa_pool_release_window: blocks that left a sliding window go back to the pool.  No GPU."""
import random

import pytest

import paged_kv_cache_75_gb300 as pk
import window_ref as R
from oracle.pool_model import BlockPoolModel
from paged_kv_cache_75_gb300 import build as pkg_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg_build.build()


class Model(BlockPoolModel):
    """The pool model with holes."""

    def release_window(self, seq_id, window, sinks):
        blocks, length = self.seqs[seq_id]
        n = 0
        seen = R.seen_blocks(length, length - 1, window, sinks, self.block_size).tolist() if length else []
        for j, b in enumerate(blocks):
            # a block past the sinks is released when it ends before the window
            if b is not None and not seen[j]:
                self.ref[b] -= 1
                if self.ref[b] == 0:
                    self.free.append(b)
                blocks[j] = None
                n += 1
        return n

    def fork(self, parent, child):
        blocks, length = self.seqs[parent]
        for b in blocks:
            if b is not None:
                self.ref[b] += 1
        self.seqs[child] = [list(blocks), length]

    def free_seq(self, seq_id):
        for b in self.seqs.pop(seq_id)[0]:
            if b is not None:
                self.ref[b] -= 1
                if self.ref[b] == 0:
                    self.free.append(b)


def table(m, s, width):
    return [-1 if b is None else b for b in m.seqs[s][0]] + [-1] * (width - len(m.seqs[s][0]))


def test_blocks_leave_one_by_one():
    pool = pk.BlockPool(6, 4)
    pool.add_seq(0)
    pool.append(0, 4)
    for n in range(5, 400):
        pool.append(0, 1)
        pool.release_window(0, 6, 1)
        t, lens = pool.block_table([0], 100)
        held = [j for j, b in enumerate(t[0]) if b >= 0]
        # the sink's block, and the window's (positions n-6 .. n-1)
        assert held == sorted({0} | set(range(max(0, n - 6) // 4, (n - 1) // 4 + 1))), n
        assert lens == [n] and pool.num_free() == 6 - len(held)
    pool.free_seq(0)
    assert pool.num_free() == 6


def test_a_shared_block_goes_back_with_its_last_user():
    pool = pk.BlockPool(10, 4)
    pool.add_seq(1)
    pool.append(1, 18)
    pool.fork(1, 2)
    assert pool.release_window(1, 5, 0) == 3
    assert pool.num_free() == 5 and pool.ref_count(0) == 1
    assert pool.release_window(1, 5, 0) == 0
    pool.fork(1, 3)  # with its holes
    assert pool.block_table([3], 5)[0] == [[-1, -1, -1, 3, 4]]
    assert pool.release_window(2, 5, 0) == 3
    assert pool.num_free() == 8
    for s in (1, 2, 3):
        pool.free_seq(s)
    assert pool.num_free() == 10


def test_refusals():
    pool = pk.BlockPool(4, 4)
    pool.add_seq(1)
    assert pool.release_window(1, 1, 0) == 0
    for args in ((9, 4, 0), (1, 0, 0), (1, -3, 0), (1, 4, -1)):
        with pytest.raises(pk.PaError) as e:
            pool.release_window(*args)
        assert e.value.status == 1
    pool.append(1, 9)
    assert pool.release_window(1, 2 ** 31 - 1, 0) == 0 and pool.release_window(1, 1, 2 ** 31 - 1) == 0
    assert pk.library().pa_pool_release_window(None, 1, 4, 0, None) == 1
    assert pk.library().pa_pool_release_window(pool._h, 1, 1, 0, None) == 0
    assert pool.block_table([1], 3)[0] == [[-1, -1, 2]]


@pytest.mark.parametrize("seed", range(30))
def test_random_operations_against_the_model(seed):
    rng = random.Random(seed)
    bs, nb = rng.choice([1, 3, 4, 16]), 200
    order = rng.sample(range(nb), nb)
    pool, m = pk.BlockPool(nb, bs, order), Model(nb, bs, order)
    nxt = 0
    for _ in range(300):
        op = rng.random()
        ids = list(m.seqs)
        if op < 0.15 or not ids:
            pool.add_seq(nxt), m.add_seq(nxt)
            nxt += 1
        elif op < 0.55:
            s, n = rng.choice(ids), rng.randint(1, 3 * bs)
            need = -(-(m.seqs[s][1] + n) // bs) - len(m.seqs[s][0]) + 1
            if need <= len(m.free):
                assert pool.append(s, n) == m.append(s, n)
        elif op < 0.85:
            s, w, k = rng.choice(ids), rng.randint(1, 6 * bs), rng.choice([0, 1, bs, 2 * bs + 1])
            assert pool.release_window(s, w, k) == m.release_window(s, w, k)
        elif op < 0.93 and len(ids) < 8:
            s = rng.choice(ids)
            pool.fork(s, nxt), m.fork(s, nxt)
            nxt += 1
        else:
            s = rng.choice(ids)
            pool.free_seq(s), m.free_seq(s)
        assert pool.num_free() == len(m.free)
        width = max([len(m.seqs[s][0]) for s in m.seqs] + [1])
        if m.seqs:
            t, lens = pool.block_table(list(m.seqs), width)
            assert t == [table(m, s, width) for s in m.seqs]
            assert lens == [m.seqs[s][1] for s in m.seqs]
        assert [pool.ref_count(b) for b in range(nb)] == m.ref


def test_windows_past_32_bits_mean_everything():
    """A window or a sink count that no 32-bit argument holds is the largest one, not its low bits."""
    pkg_build.build()
    p = pk.BlockPool(64, 4)
    p.add_seq(1)
    p.append(1, 200)
    free = p.num_free()
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 + 5):
        assert p.release_window(1, window) == 0 and p.num_free() == free
    for sinks in (2 ** 31 - 1, 2 ** 32, 2 ** 64 + 3):
        assert p.release_window(1, 8, sinks) == 0
    for window, sinks in ((0, 0), (-1, 0), (5 - 2 ** 32, 0), (8, -1), (8, 5 - 2 ** 32)):
        with pytest.raises(pk.PaError):
            p.release_window(1, window, sinks)
    size = pk.pa_decode_window_workspace_size
    assert size(4, 8, 128, 300, 16, 2 ** 32 + 5, 0, 64) == size(4, 8, 128, 300, 16, 2 ** 31 - 1, 0, 64) > 0
    assert size(4, 8, 128, 300, 16, 5 - 2 ** 32, 0, 64) == 0
    assert size(4, 8, 128, 300, 16, 8, 2 ** 40, 64) == size(4, 8, 128, 300, 16, 8, 300, 64)
    assert p.release_window(1, 8) > 0
