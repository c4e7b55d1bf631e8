"""Decode over an E4M3 cache (GPU): a query head's size, or a value in it that is not finite, is nothing to the heads
and the sequences that are worked on beside it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import window_ref as R
from gpu_util import dev_status
from paged_kv_cache_75_gb300 import workloads as W
from test_gpu_cascade import group_case, run_cascade
from test_gpu_decode_window import reference, run

pytestmark = pytest.mark.gpu
DEV = "cuda"


def plain(case):
    q = case.q.to(DEV)
    out = torch.full_like(q, float("nan"))
    L = int(case.seq_lens.max())
    n = pk.pa_decode_workspace_size(*q.shape, L, case.block_size)
    st = dev_status()
    pk.pa_decode(out, q, pk.KVCache(case.k_cache.to(DEV), case.v_cache.to(DEV)), case.block_table.to(DEV),
                 case.seq_lens.to(DEV), L, case.scale, workspace=torch.empty(max(n, 16), dtype=torch.uint8, device=DEV),
                 dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    return out.cpu()


@pytest.mark.parametrize("qd", [W.BF16, W.F16])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("x", [float("inf"), float("nan"), 3e38, 3e4])
def test_heads(x, D, G, qd):
    if qd == W.F16 and x == 3e38:
        x = 65504.0
    case = W.make_decode_case(50 + G, [40, 300, 700, 1], 2 * G, 2, D, 32, 40, qd, W.E4M3)
    clean = [plain(case)] + [run(case, 100, 5)[0]]
    ref, mag = reference(case, 100, 5)
    R.check(clean[1], ref, mag)
    for h in range(0, 2 * G, max(1, G // 2)):
        q = case.q.clone()
        case.q[1:, h, 7] = x
        got = [plain(case)] + [run(case, 100, 5)[0]]
        case.q = q
        for a, b in zip(got, clean):
            keep = torch.ones(a.shape[:2], dtype=torch.bool)
            keep[1:, h] = False
            assert torch.equal(a[keep].view(torch.int16), b[keep].view(torch.int16))


@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("x", [float("inf"), 3e38])
def test_members_of_a_group(x, G):
    case, cu, shared = group_case(9, [3, 8, 1], [6, 4, 2], list(range(1, 25, 2)), 2 * G, 2, 32, W.BF16)
    case.k_cache, case.v_cache = (t.float().clamp(-448, 448).to(torch.float8_e4m3fn) for t in (case.k_cache, case.v_cache))
    clean, st = run_cascade(case, cu, shared)
    assert st == 0
    q = case.q.clone()
    case.q[4, :, 3] = x
    got, st = run_cascade(case, cu, shared)
    assert st == 0
    case.q = q
    keep = np.arange(len(q)) != 4
    assert np.array_equal(got[keep], clean[keep])
