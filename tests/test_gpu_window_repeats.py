"""The calls around the cache repeat themselves bit for bit (GPU): whatever the workspace and the outputs held, on any
stream, beside other work."""
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
from gpu_util import dev_status
from paged_kv_cache_75_gb300 import workloads as W
from test_gpu_decode_window import KINDS
from test_gpu_prefill_window import TYPES, Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def repeats(call, outs, times=25):
    """call() into outs, again and again: on another stream every third time, a matrix product beside it every second."""
    x = torch.randn(2048, 2048, device=DEV)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    first = None
    for i in range(times):
        for j, o in enumerate(outs):
            o.view(torch.uint8).fill_((37 * i + j) % 251)
        torch.cuda.synchronize()
        if i % 2:
            with torch.cuda.stream(side):
                x @ x
        with torch.cuda.stream(other if i % 3 == 2 else torch.cuda.current_stream()):
            call(i)
        torch.cuda.synchronize()
        got = [o.view(torch.uint8).clone() for o in outs]
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first)), i


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("P", [0, 64])
def test_windowed_decode(kind, G, P):
    lens = [33, 900, 1, 2000, 511, 0, 77] * 9
    qd, kd = KINDS[kind]
    case = W.make_decode_case(3, lens, 4 * G, 4, 128, 16, sum(W.pages_for(x, 16) for x in lens) + 1, qd, kd)
    q, table, sl = case.q.to(DEV), case.block_table.to(DEV), case.seq_lens.to(DEV)
    cache = pk.KVCache(case.k_cache.to(DEV), case.v_cache.to(DEV), 1.0, 1.0)
    n = pk.pa_decode_window_workspace_size(len(lens), 4 * G, 128, 2000, 16, 700, 4, P)
    out, ws, st = torch.empty_like(q), torch.empty(max(n, 16), dtype=torch.uint8, device=DEV), dev_status()

    def call(i):
        ws.fill_(i * 9 % 256)
        pk.pa_decode_window(out, q, cache, table, sl, 2000, case.scale, 700, 4, P, ws, st)
    repeats(call, [out])
    assert st.item() == 0


@pytest.mark.parametrize("dt,G", [("bf16", 4), ("f16", 1), ("f16", 8)])
@pytest.mark.parametrize("odd", [False, True])
def test_windowed_prefill(dt, G, odd):
    c = Batch([300, 1, 77, 640, 5, 128] * 4, [400, 900, 77, 2000, 300, 128] * 4, G, 4, 16, TYPES[dt])
    if odd:
        c.vc[int(c.table[3, 100]), 1, 3, 9] = float("inf")
    cache, st, q = pk.KVCache(c.kc.to(DEV), c.vc.to(DEV)), dev_status(), c.q.to(DEV)
    table, cq, ck, out = c.table.to(DEV), c.cu_q.to(DEV), c.cu_k.to(DEV), torch.empty_like(q)
    repeats(lambda i: pk.pa_prefill_varlen_window(out, q, cache, table, cq, ck, 640, 2000, c.scale, 300, 4, st), [out])
    assert st.item() == 0


@pytest.mark.parametrize("T", [1, 700, 9000])
def test_norm_rotation_and_write(T):
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, 24, 128, generator=g, device=DEV).to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn(128, generator=g, device=DEV)
    tr = pk.QKTransform(pk.rope_frequencies(128, 500000.0, device=DEV), q_weight=w, k_weight=w)
    pos = torch.randint(0, 100000, (T,), generator=g, device=DEV)
    kc = torch.empty(T // 16 + 1, 4, 16, 128, dtype=torch.bfloat16, device=DEV)
    cache, qo, slots = pk.KVCache(kc, kc.clone()), torch.empty(T, 16, 128, dtype=torch.bfloat16, device=DEV), torch.arange(T, device=DEV)
    repeats(lambda i: (cache.k_cache.zero_(), cache.v_cache.zero_(), pk.pa_qk_norm_rope_write(
        qo, x[:, :16], x[:, 16:20], x[:, 20:], cache, pos, slots, tr)), [qo, cache.k_cache, cache.v_cache])
