"""pa_varlen_cascade against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
from cascade_ref import Batch

pytestmark = pytest.mark.gpu

ONE = [(1, 1)]


def own(n, seed, hi, q_hi=1, q_lo=1):
    rng = np.random.default_rng(seed)
    q = rng.integers(q_lo, q_hi + 1, n)
    return [(int(a + b), int(b)) for a, b in zip(rng.integers(0, hi + 1, n), q)]


LAYOUTS = {
    "decode": lambda bs: [(40 * bs, own(5, 1, 300)), (bs, own(3, 2, 20)), (7 * bs, own(1, 3, 100))],
    "one_token_own": lambda bs: [(5 * bs, ONE * 9)],
    "no_prefix": lambda bs: [(0, own(4, 4, 500)), (0, own(1, 5, 3)), (3 * bs, own(2, 6, 3))],
    "short": lambda bs: [(64 * bs, own(7, 7, 90, 19)), (2 * bs, own(6, 8, 3, 3))],
    "ragged": lambda bs: [(11 * bs, own(3, 9, 400, 230, 0)), (33 * bs, own(2, 10, 10, 1)), (0, own(2, 11, 0, 70))],
    "wide": lambda bs: [(1024, own(70, 12, 130, 2))],
    "long": lambda bs: [(9984 // bs * bs, own(3, 13, 700, 9))],
    "no_queries": lambda bs: [(4 * bs, [(30, 0), (5, 2), (9, 0)]), (6 * bs, [(0, 0), (0, 0)]), (bs, [(3, 3)])],
}


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,bs", [(8, 1, 16), (8, 2, 32), (6, 3, 64), (5, 5, 16), (32, 8, 16), (64, 8, 32)])
def test_layouts(layout, dtype, heads, kv_heads, bs):
    b = Batch(LAYOUTS[layout](bs), heads, kv_heads, dtype, bs, len(layout) + bs).device()
    b.check(b.run())


@pytest.mark.parametrize("shared", [16, 112, 128, 144, 240, 256, 272, 512, 528, 2048])
@pytest.mark.parametrize("mine", [1, 2, 127, 128, 129, 255, 256, 257, 513])
def test_lengths_about_tiles_and_parts(shared, mine):
    for q in (1, min(mine, 33)):
        b = Batch([(shared, [(mine, q), (mine, min(q, 2))])], 8, 2, "bf16", 16, shared + mine).device()
        b.check(b.run())


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(seed)
    bs = int(rng.choice([16, 32, 64]))
    kvh, per = int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 2, 4, 8]))
    groups = []
    for _ in range(rng.integers(1, 9)):
        groups.append((int(rng.integers(0, 60)) * bs, own(int(rng.integers(1, 12)), int(rng.integers(1 << 30)), int(rng.integers(1, 700)),
                                                          int(rng.choice([1, 2, 17, 90])), int(rng.integers(0, 2)))))
    b = Batch(groups, kvh * per, kvh, ["bf16", "f16"][seed % 2], bs, seed, pad_rows=int(rng.integers(0, 3))).device()
    b.check(b.run())


def test_loose_bounds_and_a_row_behind():
    b = Batch([(160, own(4, 1, 50)), (32, own(2, 2, 5))], 8, 2, "bf16", 16, 3, pad_rows=5).device()
    b.check(b.run())
    b.check(b.run(max_q=40, max_k=9000, max_group=50, max_shared=4096))


def test_steep_softmax():
    """Large scores: the reference moves within and between parts."""
    b = Batch([(2048, own(5, 1, 600, 7))], 8, 2, "bf16", 16, 4, spread=1.0).device()
    b.scale = 1.5  # scores of about +-50
    out = b.run()
    ref, mag = b.reference()
    # 128 accumulations at 2^-23 of sum |q k| scale <= 1.5 * 150 move a weight by 3.5e-3
    lim = 2.0 ** -8 * ref.abs() + mag * (2.0 ** -15 + 7e-3 + 4e-4)
    assert bool(((out.double() - ref).abs() <= lim).all())


def test_many_queries_delegate_nothing_away():
    """Long chunks behind a prefix."""
    b = Batch([(1024, [(700, 600), (300, 257), (513, 512)]), (64, [(900, 900)])], 16, 4, "bf16", 16, 8).device()
    b.check(b.run())


def test_other_sequences_values_take_no_part():
    """Infinities and NaN in one member's own keys stay with it, and in one group's with the group."""
    b = Batch([(160, [(40, 3), (60, 1), (200, 2)]), (64, [(30, 1), (20, 4)])], 8, 2, "bf16", 16, 5)
    last = b.table[1, (b.lk[1] - 1) // 16]
    b.v[last] = float("inf")
    b.k[b.table[3, 0]] = float("nan")
    b.v[b.table[3, 1]] = float("nan")
    b.device()
    out = b.run()
    keep = torch.tensor([0, 1, 2, 4, 5], device="cuda")  # rows of sequences 0 and 2
    b.check(out, keep)


def test_strange_workspace_addresses_and_unaligned_out():
    b = Batch([(160, own(4, 1, 50, 4))], 8, 2, "bf16", 16, 3).device()
    want = b.run()
    n = b.workspace().numel()
    big = torch.full((n + 64,), 0x5a, dtype=torch.uint8, device="cuda")
    for off in (0, 16, 32, 48):
        big.fill_(0x5a)
        wide = torch.empty(b.qd.numel() + 8, dtype=b.dtype, device="cuda")
        out = wide[8:].view(b.qd.shape)  # 16-byte aligned, not 32
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        b.call(out, big[off:off + n], st)
        assert torch.equal(out, want) and int(st) == 0
        assert bool((big[:off] == 0x5a).all()) and bool((big[off + n:] == 0x5a).all())


def test_the_same_results_every_time():
    b = Batch(LAYOUTS["short"](16), 32, 8, "bf16", 16, 9).device()
    first = b.run()
    for _ in range(5):
        assert torch.equal(b.run(), first)


def test_captured_twice_and_on_another_stream():
    b = Batch(LAYOUTS["decode"](16), 32, 8, "bf16", 16, 9).device()
    want = b.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(2):
            out, ws = torch.empty_like(b.qd), b.workspace()
            b.call(out, ws, st)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                b.call(out, ws, st)
            runs.append((g, out, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, out, _ in runs:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for _, o, _ in runs) and int(st) == 0


@pytest.mark.parametrize("what", ["late", "partial", "long", "group", "uncovered", "row", "block", "max_q", "max_k", "total"])
def test_reported(what):
    b = Batch([(64, [(20, 2), (9, 1)]), (96, [(40, 5), (33, 1)])], 8, 2, "bf16", 16, 6).device()
    more, code = {}, 1
    if what == "late":
        b.sh[1] = 128       # past the queries' first keys
        more = dict(max_shared=128)
    elif what == "partial":
        b.sh[1] = 90
    elif what == "long":
        more = dict(max_shared=80)
    elif what == "group":
        more = dict(max_group=1)
    elif what == "uncovered":
        b.cu_g[2] = 3
    elif what == "row":
        b.tab[3, 2] = b.tab[0, 0]
    elif what == "block":
        b.tab[2:, 1], code = b.kc.shape[0], 6
    elif what == "max_q":
        more = dict(max_q=4)
    elif what == "max_k":
        more = dict(max_k=130)
    else:
        b.cu_q[4] += 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.run(status, **more)
    assert int(status) == code
    if what in ("late", "partial", "row", "block", "uncovered", "max_q", "total", "max_k"):
        b.cu_q = b.cu_q.clone()
        b.tab = torch.from_numpy(b.table).cuda()
        b.check(out, torch.arange(3, device="cuda"))  # the other group's rows


def test_a_cache_past_four_gigabytes():
    b = Batch([(160, own(3, 1, 50, 4))], 16, 8, "bf16", 16, 3, first_id=139_900)
    n = b.first_id + b.k.shape[0]
    kc = torch.empty(n, 8, 16, 128, dtype=b.dtype, device="cuda")  # 4.6 GB
    vc = torch.empty_like(kc)
    kc[b.first_id:], vc[b.first_id:] = b.k.cuda(), b.v.cuda()
    b.device()
    b.kc, b.vc = kc, vc
    b.cache = pk.KVCache(kc, vc)
    b.check(b.run())


def test_binding_refusals():
    b = Batch([(64, [(20, 2), (9, 1)])], 8, 2, "bf16", 16, 6).device()
    out, ws = torch.empty_like(b.qd), b.workspace()
    a = lambda **kw: {**dict(out=out, q=b.qd, cache=b.cache, block_table=b.tab, cu_seq_lens_q=b.cu_q,  # noqa: E731
                             cu_seq_lens_k=b.cu_k, max_seqlen_q=2, max_seqlen_k=84, scale=0.1, cu_groups=b.cu_g,
                             shared_lens=b.sh, max_group_size=2, max_shared_len=64, workspace=ws), **kw}
    for kw, e in ((dict(out=out[:1]), ValueError), (dict(out=out.float()), TypeError), (dict(q=b.qd[0]), ValueError),
                  (dict(q=b.qd.cpu()), ValueError), (dict(block_table=b.tab[:1]), ValueError),
                  (dict(block_table=b.tab.long()), TypeError), (dict(cu_seq_lens_k=b.cu_k[:2]), ValueError),
                  (dict(cu_groups=b.cu_g[:1]), ValueError), (dict(shared_lens=b.sh.cpu()), ValueError),
                  (dict(workspace=ws[:100]), pk.PaError), (dict(workspace=ws.cpu()), ValueError),
                  (dict(max_shared_len=65), pk.PaError), (dict(scale=-1.0), pk.PaError)):
        with pytest.raises(e):
            pk.pa_varlen_cascade(**a(**kw))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,bs", [(8, 8, 16), (16, 8, 32), (32, 8, 64), (64, 8, 16)])
def test_decode_batches(dtype, heads, kv_heads, bs):
    """One token a sequence, enough of them that the decode kernel takes their own keys: groups of many, of one, without
    a prefix, own keys of one token and of more than one part."""
    groups = [(20 * bs, own(15, 1, 300)), (bs, own(1, 2, 40)), (0, own(3, 3, 200)), (2048, [(2500, 1), (1, 1), (1024, 1), (1025, 1)]),
              (7 * bs, own(2, 4, 5))]
    b = Batch(groups, heads, kv_heads, dtype, bs, 21, pad_rows=4).device()
    b.check(b.run())
    b.check(b.run(max_k=9000, max_shared=4096, max_group=99))


def test_padded_decode_batch():
    """Sequences without a query behind the others (their rows too are left as they were)."""
    b = Batch([(320, own(20, 5, 90)), (64, own(2, 6, 9)), (0, [(0, 0)] * 4)], 32, 8, "bf16", 16, 22, pad_rows=4).device()
    b.check(b.run())


def test_decode_batch_with_a_gap():
    """Sequences without a query between the others: by tiles where q has a row a query, else reported."""
    groups = [(320, [(9, 1), (5, 0), (40, 1)] * 8)]
    b = Batch(groups, 32, 8, "bf16", 16, 23).device()
    b.check(b.run())
    b = Batch(groups, 32, 8, "bf16", 16, 23, pad_rows=8).device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.run(status)
    assert int(status) == 1


@pytest.mark.parametrize("what", ["late", "partial", "row", "block", "max_k"])
def test_decode_reported(what):
    b = Batch([(64, own(20, 1, 50)), (96, own(3, 2, 40))], 32, 8, "bf16", 16, 24).device()
    more, code = {}, 1
    if what == "late":
        b.sh[1] = 192
        more = dict(max_shared=192, max_k=300)
    elif what == "partial":
        b.sh[1] = 90
    elif what == "row":
        b.tab[22, 2] = b.tab[0, 0]
    elif what == "block":
        b.tab[20:, 1], code = b.kc.shape[0], 6
    else:
        more = dict(max_k=int(b.lk[20:].max()) - 1)
        assert int(b.lk[:20].max()) <= more["max_k"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.run(status, **more)
    assert int(status) == code
    b.tab = torch.from_numpy(b.table).cuda()
    b.check(out, torch.arange(20, device="cuda"))


def test_decode_captured():
    b = Batch([(640, own(30, 1, 90))], 32, 8, "bf16", 16, 25).device()
    want = b.run()
    out, ws, st = torch.empty_like(b.qd), b.workspace(), torch.zeros(1, dtype=torch.int32, device="cuda")
    b.call(out, ws, st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call(out, ws, st)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shared,members,q", [(2048, 32, 20), (1040, 64, 10), (4096, 31, 21), (272, 80, 8), (2048, 20, 33)])
def test_a_last_round_in_smaller_parts(dtype, shared, members, q):
    """One group whose query tiles fill some rounds of the SMs and a part of one more."""
    b = Batch([(shared, [(1 + (7 * i) % 90 + q - i % 3, q - i % 3) for i in range(members)])], 32, 8, dtype, 16, members, pad_rows=2)
    b.device()
    b.check(b.run())
