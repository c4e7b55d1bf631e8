"""pa_prefill_varlen_window over values that are not finite, or nearly not (GPU): what a query does not see takes no
part in it, also where other queries see it."""
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import window_ref as R
from gpu_util import dev_status
from test_gpu_prefill_window import TYPES, Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


def put(c, cache, b, t, head, dim, x):
    cache[int(c.table[b, t // c.bs]), head, t % c.bs, dim] = x


def same(got, ref, mag):
    """Finite elements as window_ref has them, the others alike."""
    g = got.to(torch.float64)
    odd = ~ref.isfinite()
    assert bool(odd.any()) and torch.equal(g.isnan(), ref.isnan())
    assert torch.equal(torch.where(odd, g, 0.0).nan_to_num(5.0, 6.0, 7.0), torch.where(odd, ref, 0.0).nan_to_num(5.0, 6.0, 7.0))
    zero = torch.zeros((), dtype=torch.float64)
    R.check(torch.where(odd, zero, g).to(got.dtype), torch.where(odd, zero, ref), torch.where(odd, zero, mag))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("window,sinks,bs", [(70, 3, 16), (70, 0, 32), (1, 0, 16), (130, 20, 64)])
def test_values_that_are_not_finite(dt, G, window, sinks, bs):
    c = Batch([200, 1, 60], [500, 333, 60], G, 2, bs, TYPES[dt], seed=window + G)
    for b, t, head, dim, x in ((0, 350, 0, 5, INF), (0, 410, 0, 77, NAN), (0, 411, 1, 127, -INF), (0, 499, 1, 0, INF),
                               (2, 21, 0, 64, -INF), (2, 22, 0, 64, INF), (2, 30, 1, 63, NAN)):
        put(c, c.vc, b, t, head, dim, x)
    idx, ref, mag = c.reference(window, sinks)
    out, st = c.run(window, sinks)
    assert st == 0
    same(out[idx], ref, mag)
    # rows that see none of it are finite
    assert bool(out[:40].isfinite().all()) and bool(out[200].isfinite().all()) and bool(out[201:222].isfinite().all())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_keys_that_are_not_finite(dt):
    c = Batch([200], [500], 4, 2, 16, TYPES[dt], seed=3)
    for t, head, x in ((350, 0, NAN), (420, 1, INF)):
        put(c, c.kc, 0, t, head, slice(None), x)
    out, st = c.run(70, 3)
    assert st == 0
    # (a query's own keys: its scores are what they are; the others do not notice)
    hit = torch.zeros(200, 8, dtype=torch.bool)
    hit[50:120, :4] = True   # positions 350 .. 419
    hit[120:190, 4:] = True  # positions 420 .. 489
    for t, head in ((350, 0), (420, 1)):
        put(c, c.kc, 0, t, head, slice(None), 0.0)
    idx, ref, mag = c.reference(70, 3)
    keep = ~hit
    R.check(out[idx][keep], ref[keep], mag[keep])


@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("climb", [0.0, 40.0])
def test_values_near_the_types_end(G, climb):
    """A sum of values under weights that are not divided by their sum yet passes binary32's range; the output does not."""
    c = Batch([150], [400], G, 1, 16, torch.bfloat16, seed=2)
    c.vc[:] = (c.vc.float().abs().clamp(0.5, 2.0) * 1.5e38).to(torch.bfloat16)
    if climb:
        d = c.q[-1, 0].float()
        c.q[:] = d.to(torch.bfloat16)
        for t in (300, 390):
            put(c, c.kc, 0, t, 0, slice(None), (climb / 1.4427 / c.scale / d.dot(d) * d).to(torch.bfloat16))
    idx, ref, mag = c.reference(200, 4)
    out, st = c.run(200, 4)
    assert st == 0 and bool(out.isfinite().all())
    R.check(out[idx], ref, mag)


@pytest.mark.parametrize("G,Hkv", [(4, 8), (1, 2)])
def test_in_a_large_batch_and_replayed(G, Hkv):
    """Several items a block, every third sequence with such a value; nothing but out written, twice the same bits."""
    n = 40
    c = Batch([130 + 3 * b for b in range(n)], [200 + 7 * b for b in range(n)], G, Hkv, 16, torch.bfloat16, seed=8)
    for b in range(0, n, 3):
        put(c, c.vc, b, 120 + b, b % Hkv, b, INF if b % 2 else NAN)
    rows = {b: [0, 60, 61, 100, c.lq[b] - 1] for b in range(n)}
    idx, ref, mag = c.reference(50, 2, rows)
    kc, vc, table = c.poisoned(50, 2)
    cache = pk.KVCache(kc.to(DEV), vc.to(DEV))
    q, t, cq, ck = c.q.to(DEV), table.to(DEV), c.cu_q.to(DEV), c.cu_k.to(DEV)
    out, st = torch.zeros_like(q), dev_status()
    args = (out, q, cache, t, cq, ck, max(c.lq), max(c.lk), c.scale, 50, 2, st)
    pk.pa_prefill_varlen_window(*args)
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.pa_prefill_varlen_window(*args)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert st.item() == 0 and torch.equal(out.view(torch.int16), first.view(torch.int16))
    same(out.cpu()[idx], ref, mag)
    assert torch.equal(cache.v_cache.cpu().view(torch.int16), vc.view(torch.int16))
