"""Prefill over keys whose scores climb past the first tile's by less than what moves the reference of bf16 weights
(GPU): fp16 weights end at 65504."""
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import window_ref as R
from gpu_util import dev_status
from test_gpu_prefill_window import TYPES, Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def climbing(dt, G, height, bs=16):
    """200 queries on 700 keys; a few keys past the first tiles score `height` (in log2) above the others, for every
    row alike, so that no other row moves a tile's reference."""
    c = Batch([200], [700], G, 2, bs, dt, seed=int(10 * height))
    d = torch.randn(128, generator=torch.Generator().manual_seed(1))
    d /= d.norm()
    c.q[:] = (8 * d + 0.05 * c.q.float()).to(dt)
    c.kc[:] = (0.05 * c.kc.float()).to(dt)
    per = 8 * c.scale * 1.4426950408889634  # log2 score of a key's unit along d
    for t in (260, 431, 510):
        c.kc[int(c.table[0, t // bs]), :, t % bs] += (height / per * d).to(dt)
    return c


# Scores reach height / 1.44 in binary32, off by 8 * 2^-24 of that (log2 scale, product, sum), and so their weights:
# 2e-5 at 60, beside what window_ref counts.
EXTRA = 1 + 2e-5 / R.WEIGHTS


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("height", [12.0, 15.5, 16.5, 20.0, 40.0, 60.0, 70.0])
@pytest.mark.parametrize("window,sinks", [(400, 4), (250, 0), (700, 0)])
def test_windowed(dt, G, height, window, sinks):
    c = climbing(TYPES[dt], G, height)
    idx, ref, mag = c.reference(window, sinks, {0: [0, 1, 31, 32, 100, 128, 199]})
    out, st = c.run(window, sinks)
    assert st == 0 and bool(out.isfinite().all())
    R.check(out[idx], ref, mag * EXTRA)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("height", [15.5, 16.5, 20.0, 40.0, 60.0])
@pytest.mark.parametrize("packed", [False, True])
def test_unwindowed(dt, G, height, packed):
    c = climbing(TYPES[dt], G, height)
    idx, ref, mag = c.reference(700, 0, {0: [0, 1, 31, 32, 100, 128, 199]})
    out, st = torch.full_like(c.q, float("nan")).to(DEV), dev_status()
    cu_q, cu_k = c.cu_q.to(DEV), c.cu_k.to(DEV)
    if packed:
        t = torch.arange(700)
        rows = [x[c.table[0][t // 16].long(), :, t % 16].contiguous().to(DEV) for x in (c.kc, c.vc)]
        pk.pa_prefill_varlen_packed(out, c.q.to(DEV), *rows, cu_q, cu_k, 200, 700, c.scale, True, st)
    else:
        pk.pa_prefill_varlen(out, c.q.to(DEV), pk.KVCache(c.kc.to(DEV), c.vc.to(DEV)), c.table.to(DEV), cu_q, cu_k, 200,
                             700, c.scale, True, st)
    torch.cuda.synchronize()
    assert st.item() == 0 and bool(out.isfinite().all())
    R.check(out.cpu()[idx], ref, mag * EXTRA)
