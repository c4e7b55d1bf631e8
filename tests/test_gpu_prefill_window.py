"""pa_prefill_varlen_window against the definition in 64 bits (GPU)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import window_ref as R
from gpu_util import dev_status
from paged_kv_cache_75_gb300 import workloads as W
from test_gpu_canaries import Guarded, all_intact

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    def __init__(self, lq, lk, G, Hkv, bs, dt, seed=0, extra=2):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lq, self.lk, self.bs, self.D = list(lq), list(lk), bs, 128
        nb = sum(W.pages_for(x, bs) for x in lk) + extra
        self.table = torch.from_numpy(W.assign_blocks(rng, lk, bs, nb))
        self.q = torch.randn(sum(lq), G * Hkv, 128, generator=g).to(dt)
        self.kc = torch.randn(nb, Hkv, bs, 128, generator=g).to(dt)
        self.vc = torch.randn(nb, Hkv, bs, 128, generator=g).to(dt)
        self.scale = 128 ** -0.5
        self.cu_q = torch.tensor([0] + list(np.cumsum(lq)), dtype=torch.int32)
        self.cu_k = torch.tensor([0] + list(np.cumsum(lk)), dtype=torch.int32)

    def reference(self, window, sinks, rows=None):
        """rows: {sequence: query indices}; all by default. -> index, out, mag"""
        idx, outs, mags = [], [], []
        for b, (n, L) in enumerate(zip(self.lq, self.lk)):
            i = torch.arange(n) if rows is None else torch.tensor(rows.get(b, []), dtype=torch.long)
            if i.numel() == 0:
                continue
            at = int(self.cu_q[b]) + i
            o, m = R.attend(self.q[at], (L - n + i).tolist(), L, self.table[b], self.kc, self.vc, self.scale, window, sinks)
            idx.append(at), outs.append(o), mags.append(m)
        return torch.cat(idx), torch.cat(outs), torch.cat(mags)

    def poisoned(self, window, sinks):
        """NaN wherever no query of a sequence looks, unseen blocks -> -1."""
        kc, vc, table = self.kc.clone(), self.vc.clone(), self.table.clone()
        keep = torch.zeros(kc.shape[0], self.bs, dtype=torch.bool)
        for b, (n, L) in enumerate(zip(self.lq, self.lk)):
            if n == 0 or L == 0:
                continue
            t = torch.arange(L)
            t = t[(t >= L - n - window + 1) | (t < sinks)]
            keep[self.table[b][t // self.bs].long(), t % self.bs] = True
            seen = R.seen_blocks(L, L - n, window, sinks, self.bs)
            table[b, :len(seen)][~seen] = -1
        for c in (kc, vc):
            c.masked_fill_(~keep[:, None, :, None], float("nan"))
        return kc, vc, table

    def run(self, window, sinks, kc=None, vc=None, table=None, max_q=None, max_k=None):
        out = torch.full_like(self.q, float("nan")).to(DEV)
        st = dev_status()
        cache = pk.KVCache((self.kc if kc is None else kc).to(DEV), (self.vc if vc is None else vc).to(DEV))
        pk.pa_prefill_varlen_window(out, self.q.to(DEV), cache, (self.table if table is None else table).to(DEV),
                                    self.cu_q.to(DEV), self.cu_k.to(DEV), max(self.lq) if max_q is None else max_q,
                                    max(self.lk) if max_k is None else max_k, self.scale, window, sinks, st)
        torch.cuda.synchronize()
        return out.cpu(), st.item()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 16), (33, 3), (65, 130), (100, 0), (200, 20)])
def test_masks(dt, G, bs, window, sinks):
    """Sequences with fewer keys than queries, none of either, chunks on a long prior part; windows and sinks
    that begin and end inside blocks and tiles; everything out of sight NaN or unallocated."""
    lq = [10, 3, 1, 0, 40, 33, 1, 70, 5]
    lk = [0, 1, 7, 20, 40, 300, 290, 411, 3]
    c = Batch(lq, lk, G, 1 if G > 2 else 2, bs, TYPES[dt], seed=window + bs)
    idx, ref, mag = c.reference(window, sinks)
    out, st = c.run(window, sinks, *c.poisoned(window, sinks))
    assert st == 0
    R.check(out[idx], ref, mag)
    assert bool((out[:10] == 0).all())  # queries without keys


@pytest.mark.parametrize("dt,G,bs", [("bf16", 4, 16), ("f16", 1, 32), ("bf16", 8, 64), ("f16", 2, 16)])
@pytest.mark.parametrize("window,sinks", [(128, 4), (129, 0), (700, 40), (1, 300), (1000, 1)])
def test_long_chunks(dt, G, bs, window, sinks):
    lq, lk = [600, 1, 259, 130], [600, 2100, 1900, 1500]
    c = Batch(lq, lk, G, 1, bs, TYPES[dt], seed=5)
    rows = {0: [0, 1, 127, 128, 130, 399, 598, 599], 1: [0], 2: [0, 5, 31, 32, 64, 127, 128, 200, 258], 3: [0, 1, 63, 128, 129]}
    idx, ref, mag = c.reference(window, sinks, rows)
    out, st = c.run(window, sinks, *c.poisoned(window, sinks))
    assert st == 0
    R.check(out[idx], ref, mag)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("dt,G,Hkv,bs", [("bf16", 8, 2, 16), ("f16", 4, 4, 32), ("bf16", 1, 8, 64)])
@pytest.mark.parametrize("window,sinks", [(300, 4), (130, 0), (17, 33)])
def test_several_items_a_block(dt, G, Hkv, bs, window, sinks):
    """More items than blocks, of unlike costs: the sorted order, both tensor-memory buffers, the deferred output."""
    rng = np.random.default_rng(window)
    lq = [int(x) for x in rng.integers(1, 500, size=14)] + [0, 1, 1, 2000]
    lk = [n + int(x) for n, x in zip(lq, rng.integers(0, 1500, size=len(lq)))]
    c = Batch(lq, lk, G, Hkv, bs, TYPES[dt], seed=G)
    assert sum(-(-n // (128 // G)) for n in lq) * Hkv > 2 * 152
    rows = {b: sorted({int(i) for i in rng.integers(0, n, size=5)} | {0, n - 1}) for b, n in enumerate(lq) if n}
    out, st = c.run(window, sinks, *c.poisoned(window, sinks))
    assert st == 0 and bool(out.isfinite().all())
    idx, ref, mag = c.reference(window, sinks, rows)
    R.check(out[idx], ref, mag)


def test_more_items_than_a_blocks_table_of_them():
    """Over 64 items a block: the rest are worked out on the way."""
    n, lq = 330, 60
    c = Batch([lq] * n, [lq + 40 + b % 90 for b in range(n)], 8, 8, 16, torch.bfloat16, seed=2)
    assert n * -(-lq // 16) * 8 > 64 * 152
    out, st = c.run(50, 3)
    assert st == 0 and bool(out.isfinite().all())
    idx, ref, mag = c.reference(50, 3, {b: [0, b % lq, lq - 1] for b in range(0, n, 23)})
    R.check(out[idx], ref, mag)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [1, 4])
def test_a_window_of_everything_is_plain_causal_prefill(dt, G):
    c = Batch([200, 1, 77], [500, 300, 77], G, 2, 16, TYPES[dt])
    want = torch.empty_like(c.q).to(DEV)
    cache = pk.KVCache(c.kc.to(DEV), c.vc.to(DEV))
    pk.pa_prefill_varlen(want, c.q.to(DEV), cache, c.table.to(DEV), c.cu_q.to(DEV), c.cu_k.to(DEV), 200, 500, c.scale, True)
    for window, sinks in ((500, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 500), (250, 250)):
        out, st = c.run(window, sinks)
        assert st == 0
        assert torch.equal(out.view(torch.int16), want.cpu().view(torch.int16)), (window, sinks)
    # one key short: the query at position 499 does not see key 249
    out, st = c.run(250, 249)
    assert st == 0 and not torch.equal(out[199], want[199].cpu())
    assert torch.equal(out[:199].view(torch.int16), want[:199].cpu().view(torch.int16))
    idx, ref, mag = c.reference(250, 249)
    R.check(out, ref, mag)


@pytest.mark.parametrize("G,bs", [(1, 16), (4, 16), (8, 32)])
def test_one_token_rows_agree_with_decode(G, bs):
    lk = [1, 40, 333, 900, 1500]
    c = Batch([1] * 5, lk, G, 2, bs, torch.bfloat16, seed=9)
    out, st = c.run(120, 5)
    assert st == 0
    idx, ref, mag = c.reference(120, 5)
    R.check(out, ref, mag)
    dec = torch.empty_like(c.q).to(DEV)
    pk.pa_decode_window(dec, c.q.to(DEV), pk.KVCache(c.kc.to(DEV), c.vc.to(DEV)), c.table.to(DEV),
                        torch.tensor(lk, dtype=torch.int32, device=DEV), 1500, c.scale, 120, 5)
    R.check(dec.cpu(), ref, mag)


def test_scores_that_climb_past_the_reference_maximum():
    """Keys whose scores grow along the sequence, and a sink that dominates or vanishes: the running maximum moves
    inside the window."""
    c = Batch([300], [900], 4, 1, 16, torch.bfloat16, seed=3)
    d = torch.randn(128, generator=torch.Generator().manual_seed(1))
    d /= d.norm()
    c.q[:] = (8 * d).to(torch.bfloat16)
    for t in range(900):
        blk = int(c.table[0, t // 16])
        c.kc[blk, 0, t % 16] = (0.3 * t * d).to(torch.bfloat16)
    for sink_size in (-50.0, 0.0, 400.0):
        blk = int(c.table[0, 0])
        c.kc[blk, 0, :2] = (sink_size * d).to(torch.bfloat16)
        rows = {0: [0, 31, 32, 150, 299]}
        idx, ref, mag = c.reference(200, 2, rows)
        out, st = c.run(200, 2)
        assert st == 0
        # scores up to 8 * 400 * 128^-0.5 = 283 in binary32: off by 283 * 2^-24 * 8 (log2 scale, product, sum) = 1.4e-4 each
        R.check(out[idx], ref, mag * (1 + 3e-4 / R.WEIGHTS))


def test_bad_blocks_and_lengths_are_reported():
    c = Batch([40, 30], [400, 300], 4, 1, 16, torch.float16)
    idx, ref, mag = c.reference(100, 4)
    table = c.table.clone()
    table[0, 10] = 1 << 30  # no query of sequence 0 looks there
    out, st = c.run(100, 4, table=table)
    assert st == 0
    R.check(out[idx], ref, mag)
    for j in (0, 17, 24):
        table = c.table.clone()
        table[0, j] = -7
        out, st = c.run(100, 4, table=table)
        assert st == 6
        R.check(out[40:], ref[40:], mag[40:])
    out, st = c.run(100, 4, max_k=350)
    assert st == 1
    R.check(out[40:], ref[40:], mag[40:])
    assert bool(out[:40].isnan().all())  # not written


def test_writes_only_out():
    c = Batch([1, 130, 33], [1, 700, 500], 4, 2, 16, torch.bfloat16, extra=6)
    gk, gv = Guarded(c.kc.shape, c.kc.dtype, init=c.kc.to(DEV)), Guarded(c.vc.shape, c.vc.dtype, init=c.vc.to(DEV))
    gq, go = Guarded(c.q.shape, c.q.dtype, init=c.q.to(DEV)), Guarded(c.q.shape, c.q.dtype)
    st = dev_status()
    pk.pa_prefill_varlen_window(go.t, gq.t, pk.KVCache(gk.t, gv.t), c.table.to(DEV), c.cu_q.to(DEV), c.cu_k.to(DEV), 130,
                                700, c.scale, 90, 3, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    all_intact(gk, gv, gq, go)
    assert torch.equal(gk.t.cpu(), c.kc) and torch.equal(gv.t.cpu(), c.vc)
    idx, ref, mag = c.reference(90, 3)
    R.check(go.t.cpu(), ref, mag)


@pytest.mark.parametrize("dt,G,bs", [("bf16", 4, 16), ("f16", 8, 32)])
def test_rows_past_the_last_sequence_stay_as_they_were(dt, G, bs):
    """A batch padded to a fixed count of rows, as a captured step keeps it: empty sequences at its end, rows behind the
    last one, in q (NaN) and in out."""
    c = Batch([37, 1, 70, 0, 0], [137, 20, 300, 0, 0], G, 2, bs, TYPES[dt])
    pad = 45
    q = torch.cat([c.q, torch.full((pad, *c.q.shape[1:]), float("nan"), dtype=c.q.dtype)]).to(DEV)
    out = torch.full_like(q, 7.0)
    st = dev_status()
    pk.pa_prefill_varlen_window(out, q, pk.KVCache(c.kc.to(DEV), c.vc.to(DEV)), c.table.to(DEV), c.cu_q.to(DEV),
                                c.cu_k.to(DEV), 128, 512, c.scale, 60, 3, st)
    torch.cuda.synchronize()
    assert st.item() == 0 and bool((out[-pad:] == 7.0).all())
    idx, ref, mag = c.reference(60, 3)
    R.check(out[:-pad].cpu()[idx], ref, mag)


def test_captured_and_replayed():
    c = Batch([64, 9], [300, 200], 4, 2, 16, torch.bfloat16)
    out = torch.empty_like(c.q).to(DEV)
    q, cache = c.q.to(DEV), pk.KVCache(c.kc.to(DEV), c.vc.to(DEV))
    args = (cache, c.table.to(DEV), c.cu_q.to(DEV), c.cu_k.to(DEV), 64, 300, c.scale, 50, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pk.pa_prefill_varlen_window(out, q, *args)
    s.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.pa_prefill_varlen_window(out, q, *args)
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    idx, ref, mag = c.reference(50, 2)
    R.check(out.cpu(), ref, mag)


def test_the_binding_refuses_wrong_tensors():
    c = Batch([4, 2], [30, 20], 2, 2, 16, torch.float16)
    out, q, cache = torch.empty_like(c.q).to(DEV), c.q.to(DEV), pk.KVCache(c.kc.to(DEV), c.vc.to(DEV))
    t, cq, ck = c.table.to(DEV), c.cu_q.to(DEV), c.cu_k.to(DEV)
    with pytest.raises(ValueError):
        pk.pa_prefill_varlen_window(out[:3], q, cache, t, cq, ck, 4, 30, 0.1, 8)
    with pytest.raises(ValueError):
        pk.pa_prefill_varlen_window(out, q, cache, t[:1], cq, ck, 4, 30, 0.1, 8)
    with pytest.raises(ValueError):
        pk.pa_prefill_varlen_window(out, q, cache, t, cq, ck[:2], 4, 30, 0.1, 8)
    for window, sinks, scale in ((0, 0, 0.1), (8, -1, 0.1), (8, 0, 0.0), (8, 0, -1.0), (8, 0, float("inf"))):
        with pytest.raises(pk.PaError):
            pk.pa_prefill_varlen_window(out, q, cache, t, cq, ck, 4, 30, scale, window, sinks)
