"""A windowed decode or a prefill whose waits run out ends with PA_ERR_TIMEOUT and leaves the GPU usable.

As tests/test_gpu_wait_timeout.py: the hooks launch the kernels with loader warps that issue no copy at all, so the
waits for the queries and the pages run out (2 s) with nothing in flight.  The same calls in earnest, on the same stream
afterwards, still match the definition in 64 bits.
"""
import time

import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import test_gpu_decode_window as DW
import window_ref as R
from gpu_util import dev_status
from paged_kv_cache_75_gb300 import workloads as W
from test_gpu_prefill_window import TYPES, Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def timed(call):
    torch.cuda.synchronize()
    t0 = time.monotonic()
    call()
    torch.cuda.synchronize()
    assert 1.0 < time.monotonic() - t0 < 60.0  # the wait limit ran out, then the kernel returned


@pytest.mark.parametrize("G,P", [(1, 0), (4, 0), (4, 32)])
def test_windowed_decode(G, P):
    """P 0: every item has a block of its own, no work list; P 32 on many sequences: a work list."""
    lens = [100, 700, 33, 1] * (1 if P == 0 else 40)
    case = W.make_decode_case(21 + G, lens, 4 * G, 4, 128, 16, 80 * (len(lens) // 4), W.BF16, W.BF16)
    ref, mag = DW.reference(case, 90, 3)
    q = case.q.to(DEV)
    cache = pk.KVCache(case.k_cache.to(DEV), case.v_cache.to(DEV))
    n = pk.pa_decode_window_workspace_size(len(lens), 4 * G, 128, 700, 16, 90, 3, P)
    ws, st = torch.empty(max(16, n), dtype=torch.uint8, device=DEV), dev_status()
    timed(lambda: pk.pa_decode_window_test_wait_timeout(torch.zeros_like(q), q, cache, case.block_table.to(DEV),
                                                        case.seq_lens.to(DEV), 700, case.scale, 90, 3, P, ws, st))
    assert int(st.item()) == 5  # PA_ERR_TIMEOUT
    out, status = DW.run(case, 90, 3, P)
    assert status == 0
    R.check(out, ref, mag)


@pytest.mark.parametrize("dt,G", [("bf16", 4), ("f16", 1)])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("lq", [[20], [200, 1, 0, 77], [150] * 60])
def test_prefill(dt, G, window, lq):
    """One item, a few, several a block."""
    c = Batch(lq, [n + 100 if n else 0 for n in lq], G, 4, 16, TYPES[dt])
    cache, st = pk.KVCache(c.kc.to(DEV), c.vc.to(DEV)), dev_status()
    q, table, cq, ck = c.q.to(DEV), c.table.to(DEV), c.cu_q.to(DEV), c.cu_k.to(DEV)
    out = torch.zeros_like(q)
    timed(lambda: pk.pa_prefill_test_wait_timeout(out, q, cache, table, cq, ck, max(lq), max(c.lk), c.scale, window, 2, st))
    assert int(st.item()) == 5
    st = dev_status()
    if window:
        pk.pa_prefill_varlen_window(out, q, cache, table, cq, ck, max(lq), max(c.lk), c.scale, window, 2, st)
    else:
        pk.pa_prefill_varlen(out, q, cache, table, cq, ck, max(lq), max(c.lk), c.scale, True, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    rows = {b: [0, n // 2, n - 1] for b, n in enumerate(lq) if n and b < 6}
    idx, ref, mag = c.reference(window or 10 ** 6, 2, rows)
    R.check(out.cpu()[idx], ref, mag)
