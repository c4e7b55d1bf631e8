"""The windowed path together, as a layer's attention runs it (GPU): projections normed, rotated and written to the
paged cache, a windowed prefill of the prompts, then decode steps, the pool taking back what left the window, its
blocks given to the other sequences -- in a pool that could not hold the sequences whole."""
import numpy as np
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import rope_ref
import window_ref as R
from gpu_util import dev_status

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


class Layer:
    """One layer's cache, pool and kernels; beside it, what it must be equivalent to: every token of every sequence
    kept, in order, in a cache of its own."""

    def __init__(self, n_seqs, H, Hkv, dt, kd, bs, window, sinks, num_blocks, longest, interleaved):
        g = torch.Generator().manual_seed(1)
        self.H, self.Hkv, self.dt, self.bs, self.window, self.sinks = H, Hkv, dt, bs, window, sinks
        self.scale = D ** -0.5
        self.pool = pk.BlockPool(num_blocks, bs)
        ks, vs = (0.05, 0.02) if kd == torch.float8_e4m3fn else (1.0, 1.0)
        mk = lambda nb: pk.KVCache(torch.zeros(nb, Hkv, bs, D, device=DEV).to(kd),  # noqa: E731
                                   torch.zeros(nb, Hkv, bs, D, device=DEV).to(kd), ks, vs)
        self.cache = mk(num_blocks)
        self.per = -(-longest // bs)
        self.whole = mk(n_seqs * self.per)
        self.qw, self.kw = 1 + 0.1 * torch.randn(D, generator=g), 1 + 0.1 * torch.randn(D, generator=g)
        rope = pk.rope_frequencies(96, 50000.0, "yarn", factor=4.0, original_max_position=64, device=DEV)
        self.tr = pk.QKTransform(rope, interleaved, self.qw.to(DEV), self.kw.to(DEV), 1e-6)
        self.st = dev_status()
        self.lens = [0] * n_seqs
        for s in range(n_seqs):
            self.pool.add_seq(s)
        self.g = g

    def write(self, counts):
        """Appends counts[s] tokens to each sequence -> their queries, normed and rotated (device, packed)."""
        T = sum(counts)
        x = torch.randn(T, self.H + 2 * self.Hkv, D, generator=self.g).to(self.dt)
        slots, pos, own = [], [], []
        for s, n in enumerate(counts):
            sl, cow = self.pool.append(s, n)
            assert cow == []
            slots += sl
            pos += list(range(self.lens[s], self.lens[s] + n))
            own += [s * self.per * self.bs + self.lens[s] + i for i in range(n)]
            self.lens[s] += n
        xd = x.to(DEV)
        q, k, v = xd[:, :self.H], xd[:, self.H:self.H + self.Hkv], xd[:, self.H + self.Hkv:]
        q_out = torch.empty(T, self.H, D, dtype=self.dt, device=DEV)
        again = torch.empty_like(q_out)
        p = torch.tensor(pos, device=DEV)
        pk.pa_qk_norm_rope_write(q_out, q, k, v, self.cache, p, torch.tensor(slots, device=DEV), self.tr, self.st)
        pk.pa_qk_norm_rope_write(again, q, k, v, self.whole, p, torch.tensor(own, device=DEV), self.tr, self.st)
        assert torch.equal(q_out, again)
        ref, pair = rope_ref.rows(x[:, :self.H], pos, self.tr.rope.theta, self.tr.rope.factor, self.tr.interleaved,
                                  self.qw, 1e-6)
        rope_ref.check(q_out.cpu(), ref, pair, self.dt)
        return q_out

    def table(self):
        width = max(-(-n // self.bs) for n in self.lens)
        t, lens = self.pool.block_table(list(range(len(self.lens))), width)
        assert lens == self.lens
        return torch.tensor(t, dtype=torch.int32, device=DEV)

    def release(self, chunk=1):
        return sum(self.pool.release_window(s, self.window + chunk - 1, self.sinks) for s in range(len(self.lens)))

    def check(self, out, q, counts):
        at = 0
        kc, vc = self.whole.k_cache.cpu(), self.whole.v_cache.cpu()
        for s, n in enumerate(counts):
            row = torch.arange(s * self.per, (s + 1) * self.per, dtype=torch.int32)
            pick = sorted({0, n - 1, n // 2}) if n else []
            sel = torch.tensor(pick, dtype=torch.long)
            ref, mag = R.attend(q.cpu()[at + sel], (self.lens[s] - n + sel).tolist(), self.lens[s], row, kc, vc, self.scale,
                                self.window, self.sinks, self.whole.k_scale, self.whole.v_scale)
            R.check(out.cpu()[at + sel], ref, mag, "sequence %d" % s)
            at += n


@pytest.mark.parametrize("dt,G,bs,window,sinks", [(torch.bfloat16, 4, 16, 40, 4), (torch.float16, 1, 32, 64, 0),
                                                  (torch.bfloat16, 8, 16, 17, 20)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_prefill_then_decode_in_a_small_pool(dt, G, bs, window, sinks, interleaved):
    n, Hkv = 3, 2
    # blocks a sequence may hold: the sinks', the window's and the longest chunk's
    most = -(-sinks // bs) + (window + 33) // bs + 3
    L = Layer(n, G * Hkv, Hkv, dt, dt, bs, window, sinks, n * most, 600, interleaved)
    total = 0
    for counts in ([33, 9, 1], [20, 33, 33], [33, 1, 30]):  # chunks of the prompts
        q = L.write(counts)
        cu_q = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
        cu_k = torch.tensor([0] + list(np.cumsum(L.lens)), dtype=torch.int32, device=DEV)
        out = torch.empty_like(q)
        pk.pa_prefill_varlen_window(out, q, L.cache, L.table(), cu_q, cu_k, max(counts), max(L.lens), L.scale, window, sinks,
                                    L.st)
        L.check(out, q, counts)
        total += L.release()
    ws = torch.empty(pk.pa_decode_window_workspace_size(n, G * Hkv, D, 600, bs, window, sinks, bs), dtype=torch.uint8, device=DEV)
    for step in range(150):
        q = L.write([1] * n)
        out = torch.empty_like(q)
        lens = torch.tensor(L.lens, dtype=torch.int32, device=DEV)
        pk.pa_decode_window(out, q, L.cache, L.table(), lens, max(L.lens), L.scale, window, sinks, bs if step % 2 else 0, ws, L.st)
        if step % 7 == 0 or step > 145:
            L.check(out, q, [1] * n)
        total += L.release()
    assert L.st.item() == 0
    # more blocks went through than the pool has
    assert sum(-(-x // bs) for x in L.lens) > n * most and total > 0


def test_decode_over_an_e4m3_cache():
    n, H, Hkv, bs, window, sinks = 4, 8, 1, 32, 50, 3
    L = Layer(n, H, Hkv, torch.bfloat16, torch.float8_e4m3fn, bs, window, sinks, n * 5, 400, False)
    for step in range(200):
        counts = [1, 1 + (step == 0) * 30, 1, 1]
        q = L.write(counts)
        if step:
            out = torch.empty_like(q)
            lens = torch.tensor(L.lens, dtype=torch.int32, device=DEV)
            need = pk.pa_decode_window_workspace_size(n, H, D, 400, bs, window, sinks)
            ws = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
            pk.pa_decode_window(out, q, L.cache, L.table(), lens, max(L.lens), L.scale, window, sinks, 0, ws, L.st)
            if step % 9 == 0 or step > 196:
                L.check(out, q, counts)
        L.release()
    assert L.st.item() == 0


def test_a_whole_step_in_one_graph():
    """Write and attend captured once, replayed as the sequences grow: positions, slots, lengths and the table are
    buffers that the host refills."""
    n, H, Hkv, bs, window, sinks = 2, 8, 2, 16, 30, 2
    L = Layer(n, H, Hkv, torch.bfloat16, torch.bfloat16, bs, window, sinks, 64, 200, False)
    g = torch.Generator().manual_seed(5)
    x = torch.zeros(n, H + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    pos, slots = torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV)
    lens, table = torch.zeros(n, dtype=torch.int32, device=DEV), torch.full((n, 16), -1, dtype=torch.int32, device=DEV)
    q_out, out = torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV), torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(pk.pa_decode_window_workspace_size(n, H, D, 200, bs, window, sinks, 16), dtype=torch.uint8, device=DEV)

    def step():
        pk.pa_qk_norm_rope_write(q_out, x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], L.cache, pos, slots, L.tr, L.st)
        pk.pa_decode_window(out, q_out, L.cache, table, lens, 200, L.scale, window, sinks, 16, ws, L.st)

    slots.fill_(-1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(120):
        xi = torch.randn(x.shape, generator=g).to(torch.bfloat16)
        new = [L.pool.append(b, 1)[0][0] for b in range(n)]
        x.copy_(xi), pos.fill_(i), slots.copy_(torch.tensor(new))
        L.lens = [i + 1] * n
        lens.fill_(i + 1)
        t = L.table()
        table.fill_(-1), table[:, :t.shape[1]].copy_(t)
        graph.replay()
        pk.pa_qk_norm_rope_write(torch.empty_like(q_out), x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], L.whole, pos,
                                 torch.tensor([b * L.per * bs + i for b in range(n)], device=DEV), L.tr)
        torch.cuda.synchronize()
        if i % 10 == 0 or i > 115:
            L.check(out, q_out, [1] * n)
        L.release()
    assert L.st.item() == 0
