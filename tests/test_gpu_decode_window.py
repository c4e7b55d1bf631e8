"""pa_decode_window against the definition in 64 bits (GPU)."""
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
KINDS = {"f16": (W.F16, W.F16), "bf16": (W.BF16, W.BF16), "e4m3": (W.BF16, W.E4M3), "e4m3_f16": (W.F16, W.E4M3)}


def poison(case, window, sinks, block=None):
    """NaN wherever nothing may look: positions that are not seen, positions past
    the length, blocks outside the table; entries of unseen blocks -> -1 (or
    `block`)."""
    kc, vc = case.k_cache.clone(), case.v_cache.clone()
    table = case.block_table.clone()
    bs = case.block_size
    keep = torch.zeros(kc.shape[0], bs, dtype=torch.bool)
    for b, L in enumerate(case.seq_lens.tolist()):
        seen = R.seen_blocks(L, L - 1, window, sinks, bs)
        for j in range(len(seen)):
            if not seen[j]:
                table[b, j] = -1 if block is None else block
        t = torch.arange(L)
        t = t[(t >= L - window) | (t < sinks)]
        keep[case.block_table[b][t // bs].long(), t % bs] = True
    for c in (kc, vc):
        bits = c.view(torch.uint8 if c.element_size() == 1 else torch.int16)
        nan = {torch.float16: 0x7e00, torch.bfloat16: 0x7fc0, torch.float8_e4m3fn: 0x7f}[c.dtype]
        bits.masked_fill_(~keep[:, None, :, None], nan)
    return kc, vc, table


def run(case, window, sinks, P=0, kc=None, vc=None, table=None, ks=1.0, vs=1.0, max_len=None):
    cache = pk.KVCache((case.k_cache if kc is None else kc).to(DEV), (case.v_cache if vc is None else vc).to(DEV), ks, vs)
    q = case.q.to(DEV)
    out = torch.full_like(q, float("nan"))
    max_len = max(1, int(case.seq_lens.max())) if max_len is None else max_len
    n = pk.pa_decode_window_workspace_size(q.shape[0], q.shape[1], q.shape[2], max_len, case.block_size, window, sinks, P)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    st = dev_status()
    pk.pa_decode_window(out, q, cache, (case.block_table if table is None else table).to(DEV), case.seq_lens.to(DEV),
                        max_len, case.scale, window, sinks, P, ws, st)
    torch.cuda.synchronize()
    return out.cpu(), st.item()


def reference(case, window, sinks, ks=1.0, vs=1.0):
    outs, mags = [], []
    for b, L in enumerate(case.seq_lens.tolist()):
        o, m = R.attend(case.q[b:b + 1], [L - 1], L, case.block_table[b], case.k_cache, case.v_cache, case.scale, window,
                        sinks, ks, vs)
        outs.append(o), mags.append(m)
    return torch.cat(outs), torch.cat(mags)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 16), (33, 3), (64, 65), (100, 0), (250, 20)])
def test_masks(kind, G, bs, window, sinks):
    """Windows and sinks that begin and end inside blocks, meet, overlap; lengths
    from none on; everything out of sight NaN or unallocated."""
    qd, kd = KINDS[kind]
    D = 64 if (G + bs + window) % 3 == 0 else 128
    lens = [0, 1, 2, bs - 1, bs, bs + 1, window, window + 1, window + sinks + bs, 3 * bs + 5, 271, 300]
    case = W.make_decode_case(window * 7 + bs, lens, 2 * G, 2, D, bs, sum(W.pages_for(x, bs) for x in lens) + 2, qd, kd)
    ks, vs = (0.5, 2.0) if kd == W.E4M3 else (1.0, 1.0)
    ref, mag = reference(case, window, sinks, ks, vs)
    kc, vc, table = poison(case, window, sinks)
    out, st = run(case, window, sinks, 0, kc, vc, table, ks, vs)
    assert st == 0
    R.check(out, ref, mag)
    assert bool((out[0] == 0).all())
    # split into partitions of one block, and of a few
    for P in (bs, 64 if bs < 64 else 128):
        out, st = run(case, window, sinks, P, kc, vc, table, ks, vs)
        assert st == 0
        R.check(out, ref, mag, "P=%d" % P)


@pytest.mark.parametrize("kind,G,D,bs", [("f16", 1, 128, 16), ("bf16", 4, 128, 16), ("e4m3", 8, 128, 32), ("bf16", 2, 64, 64),
                                         ("f16", 8, 64, 32)])
@pytest.mark.parametrize("P", [0, 512])
def test_long_sequences(kind, G, D, bs, P):
    qd, kd = KINDS[kind]
    lens = [5000, 4097, 2500, 1, 3001, 700]
    window, sinks = 1500, 70
    case = W.make_decode_case(11, lens, 2 * G, 2, D, bs, sum(W.pages_for(x, bs) for x in lens) + 2, qd, kd)
    ref, mag = reference(case, window, sinks)
    kc, vc, table = poison(case, window, sinks)
    out, st = run(case, window, sinks, P, kc, vc, table)
    assert st == 0
    R.check(out, ref, mag)


@pytest.mark.parametrize("kind,G,bs", [("f16", 1, 16), ("bf16", 4, 16), ("e4m3", 8, 32), ("bf16", 2, 64)])
@pytest.mark.parametrize("P", [0, 64, 128])
def test_more_items_than_blocks(kind, G, bs, P):
    """A batch whose items the blocks take several of, in the work list's order (smaller ones build no list)."""
    qd, kd = KINDS[kind]
    rng = np.random.default_rng(P + G)
    lens = [int(x) for x in rng.integers(0, 700, size=330)]
    window, sinks = 260, 9
    case = W.make_decode_case(4, lens, 2 * G, 2, 64, bs, sum(W.pages_for(x, bs) for x in lens) + 2, qd, kd)
    kc, vc, table = poison(case, window, sinks)
    out, st = run(case, window, sinks, P, kc, vc, table)
    assert st == 0
    ref, mag = reference(case, window, sinks)
    R.check(out, ref, mag)
    # a batch in which one length is beyond the maximum: the others as they were
    lens[5] = 701
    broken = W.PagedCase(**{**case.__dict__, "seq_lens": torch.tensor(lens, dtype=torch.int32)})
    again, st = run(broken, window, sinks, P, kc, vc, table, max_len=700)
    assert st == 1 and bool((again[5] == 0).all())
    keep = torch.arange(330) != 5
    R.check(again[keep], ref[keep], mag[keep])


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 4])
def test_a_window_of_everything_is_plain_decode(kind, G):
    qd, kd = KINDS[kind]
    lens = [0, 1, 40, 1100, 1599]
    case = W.make_decode_case(5, lens, 2 * G, 2, 128, 16, sum(W.pages_for(x, 16) for x in lens) + 1, qd, kd)
    cache = pk.KVCache(case.k_cache.to(DEV), case.v_cache.to(DEV))
    q = case.q.to(DEV)
    B, H, D = q.shape
    for P in (256, 2048):
        want = torch.empty_like(q)
        ws = torch.empty(pk.pa_decode_workspace_size(B, H, D, 1600, 16, P) + 16, dtype=torch.uint8, device=DEV)
        pk.pa_decode(want, q, cache, case.block_table.to(DEV), case.seq_lens.to(DEV), 1600, case.scale, P, ws)
        for window, sinks in ((1600, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 1600), (800, 799)):
            out, st = run(case, window, sinks, P, max_len=1600)
            assert st == 0
            assert torch.equal(out.view(torch.int16), want.cpu().view(torch.int16)), (P, window, sinks)


def test_infinite_and_nan_scores_out_of_sight_do_not_count():
    lens = [400]
    case = W.make_decode_case(3, lens, 4, 1, 128, 16, 26, W.BF16, W.BF16)
    ref, mag = reference(case, 50, 2)
    for value in (float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min, float("nan")):
        kc, vc = case.k_cache.clone(), case.v_cache.clone()
        for t in list(range(2, 350)):
            blk = int(case.block_table[0, t // 16])
            kc[blk, :, t % 16], vc[blk, :, t % 16] = value, value
        out, st = run(case, 50, 2, 0, kc, vc)
        assert st == 0
        R.check(out, ref, mag, str(value))


def test_bad_blocks_and_lengths_are_reported():
    lens = [300, 280]
    case = W.make_decode_case(8, lens, 4, 1, 128, 16, 40, W.F16, W.F16)
    # an unseen entry may be anything, a seen one may not
    table = case.block_table.clone()
    table[0, 5] = 1 << 30
    out, st = run(case, 100, 4, 0, table=table)
    assert st == 0
    ref, mag = reference(case, 100, 4)
    R.check(out, ref, mag)
    for j in (0, 15, 18):  # the sinks' block, one of the window's, the last
        table = case.block_table.clone()
        table[0, j] = case.k_cache.shape[0]
        out, st = run(case, 100, 4, 0, table=table)
        assert st == 6
        R.check(out[1:], ref[1:], mag[1:])
    for bad in (-1, 10 ** 6):
        broken = W.PagedCase(**{**case.__dict__, "seq_lens": torch.tensor([bad, 280], dtype=torch.int32)})
        out, st = run(broken, 100, 4, 0, max_len=300)
        assert st == 1 and bool((out[0] == 0).all())
        R.check(out[1:], ref[1:], mag[1:])


@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("P", [0, 64])
def test_writes_only_out_and_workspace(G, P):
    lens = [1, 700, 33, 1500]
    case = W.make_decode_case(61, lens, 2 * G, 2, 128, 16, sum(W.pages_for(x, 16) for x in lens) + 6, W.BF16, W.BF16)
    window, sinks = 200, 5
    gk = Guarded(case.k_cache.shape, case.k_cache.dtype, init=case.k_cache.to(DEV))
    gv = Guarded(case.v_cache.shape, case.v_cache.dtype, init=case.v_cache.to(DEV))
    gq, gout = Guarded(case.q.shape, case.q.dtype, init=case.q.to(DEV)), Guarded(case.q.shape, case.q.dtype)
    B, H, D = case.q.shape
    n = pk.pa_decode_window_workspace_size(B, H, D, 1500, 16, window, sinks, P)
    gws = Guarded((max(n, 16),), torch.uint8)
    gbt = Guarded(case.block_table.shape, torch.int32, init=case.block_table.to(DEV))
    gsl = Guarded(case.seq_lens.shape, torch.int32, init=case.seq_lens.to(DEV))
    st = dev_status()
    pk.pa_decode_window(gout.t, gq.t, pk.KVCache(gk.t, gv.t), gbt.t, gsl.t, 1500, case.scale, window, sinks, P, gws.t, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    all_intact(gk, gv, gq, gout, gws, gbt, gsl)
    assert np.array_equal(W.as_bits(gk.t), W.as_bits(case.k_cache))
    ref, mag = reference(case, window, sinks)
    R.check(gout.t, ref, mag)


def test_captured_and_replayed_as_the_sequences_grow():
    lens = [300, 95, 17]
    case = W.make_decode_case(2, [310, 105, 27], 8, 2, 128, 16, 60, W.BF16, W.BF16)
    cache = pk.KVCache(case.k_cache.to(DEV), case.v_cache.to(DEV))
    q, table = case.q.to(DEV), case.block_table.to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    ws = torch.empty(pk.pa_decode_window_workspace_size(3, 8, 128, 310, 16, 64, 4, 32), dtype=torch.uint8, device=DEV)
    call = lambda: pk.pa_decode_window(out, q, cache, table, sl, 310, case.scale, 64, 4, 32, ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(10):
        graph.replay()
        torch.cuda.synchronize()
        for b in range(3):
            L = lens[b] + step
            ref, mag = R.attend(case.q[b:b + 1], [L - 1], L, case.block_table[b], case.k_cache, case.v_cache, case.scale, 64, 4)
            R.check(out[b:b + 1], ref, mag)
        sl.add_(1)


def test_the_binding_refuses_wrong_tensors():
    case = W.make_decode_case(2, [30, 20], 4, 2, 128, 16, 6, W.F16, W.F16)
    cache = pk.KVCache(case.k_cache.to(DEV), case.v_cache.to(DEV))
    q, table, sl = case.q.to(DEV), case.block_table.to(DEV), case.seq_lens.to(DEV)
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        pk.pa_decode_window(out[:1], q, cache, table, sl, 30, 0.1, 8)
    with pytest.raises(ValueError):
        pk.pa_decode_window(out, q, cache, table[:1], sl, 30, 0.1, 8)
    with pytest.raises(ValueError):
        pk.pa_decode_window(out, q, cache, table, sl[:1], 30, 0.1, 8)
    with pytest.raises(ValueError):
        pk.pa_decode_window(out, q, cache, table.cpu(), sl, 30, 0.1, 8)
    with pytest.raises(TypeError):
        pk.pa_decode_window(out, q, cache, table, sl.long(), 30, 0.1, 8)
    with pytest.raises(OverflowError):
        pk.pa_decode_window(out, q, cache, table, sl, 30, 0.1, 1 << 31)
    with pytest.raises(TypeError):
        pk.pa_decode_window(out, q, cache, table, sl, 30.5, 0.1, 8)
    # numpy's numbers are numbers
    pk.pa_decode_window(out, q, cache, table, sl, np.int64(30), np.float32(0.1), np.int32(8))
    with pytest.raises(pk.PaError):
        pk.pa_decode_window(out, q, cache, table, sl, 30, 0.1, 0)
    with pytest.raises(pk.PaError):
        pk.pa_decode_window(out, q, cache, table, sl, 30, 0.1, 8, -1)


def test_calls_on_two_streams_and_threads_at_once():
    """Two threads, each with a stream, a workspace and inputs of its own."""
    import threading
    cases = [W.make_decode_case(20 + i, [900, 77, 400], 8, 2, 128, 16, 100, W.BF16, W.BF16) for i in range(2)]
    refs = [reference(c, 300, 7) for c in cases]
    outs, errors = [None, None], []

    def work(i):
        try:
            c, s = cases[i], torch.cuda.Stream()
            with torch.cuda.stream(s):
                cache, q = pk.KVCache(c.k_cache.to(DEV), c.v_cache.to(DEV)), c.q.to(DEV)
                table, sl, out = c.block_table.to(DEV), c.seq_lens.to(DEV), torch.empty_like(c.q, device=DEV)
                n = pk.pa_decode_window_workspace_size(3, 8, 128, 900, 16, 300, 7, 64)
                ws = torch.empty(n, dtype=torch.uint8, device=DEV)
                for _ in range(200):
                    pk.pa_decode_window(out, q, cache, table, sl, 900, c.scale, 300, 7, 64, ws)
                s.synchronize()
            outs[i] = out.cpu()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for o, (ref, mag) in zip(outs, refs):
        R.check(o, ref, mag)


def test_blocks_past_four_gigabytes():
    """Blocks whose byte offset in the cache passes 32 bits: write, decode and prefill."""
    nb, bs, Hkv, H, D = 1_100_000, 16, 1, 4, 128  # 4.5 GB each of K and V
    kc = torch.zeros(nb, Hkv, bs, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros(nb, Hkv, bs, D, dtype=torch.bfloat16, device=DEV)
    cache = pk.KVCache(kc, vc)
    g = torch.Generator().manual_seed(0)
    T = 100
    ids = [nb - 1, 5, nb - 3, 1_048_577, 1_048_576, nb - 70, 3]
    x = torch.randn(T, H + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    slots = torch.tensor([ids[t // bs] * bs + t % bs for t in range(T)])
    xd = x.to(DEV)
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    st = dev_status()
    pk.pa_qk_norm_rope_write(q, xd[:, :H], xd[:, H:H + 1], xd[:, H + 1:], cache, None, slots.to(DEV), pk.QKTransform(), st)
    assert torch.equal(kc[ids[3], 0, 2], xd[50, H]) and torch.equal(vc[nb - 1, 0, 9], xd[9, H + 1])
    small_k = torch.zeros(7, Hkv, bs, D, dtype=torch.bfloat16)
    small_v = torch.zeros(7, Hkv, bs, D, dtype=torch.bfloat16)
    t = torch.arange(T)
    small_k[t // bs, 0, t % bs], small_v[t // bs, 0, t % bs] = x[:, H], x[:, H + 1]
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    pk.pa_prefill_varlen_window(out, q, cache, table, torch.tensor([0, T], dtype=torch.int32, device=DEV),
                                torch.tensor([0, T], dtype=torch.int32, device=DEV), T, T, D ** -0.5, 40, 3, st)
    ref, mag = R.attend(x[:, :H], range(T), T, torch.arange(7), small_k, small_v, D ** -0.5, 40, 3)
    R.check(out.cpu(), ref, mag)
    one = torch.empty(1, H, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(pk.pa_decode_window_workspace_size(1, H, D, T, bs, 40, 3, 16), dtype=torch.uint8, device=DEV)
    pk.pa_decode_window(one, q[-1:], cache, table, torch.tensor([T], dtype=torch.int32, device=DEV), T, D ** -0.5, 40, 3, 16,
                        ws, st)
    R.check(one.cpu(), ref[-1:], mag[-1:])
    assert st.item() == 0
