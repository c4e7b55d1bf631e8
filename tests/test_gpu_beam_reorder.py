"""pa_beam_reorder against its definition (everything is whole numbers and moved bits: equal)."""
import numpy as np
import pytest
import torch

import beam_ref as R
import paged_kv_cache_75_gb300 as pk

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def state(requests, w_in, w_out, layers, kvh, d, bs, dtype, lens, seed, width=None, drop=0.1):
    rng = np.random.default_rng(seed)
    rows = requests * w_in
    lens = np.repeat(np.resize(np.asarray(lens), requests), w_in).astype(np.int32)
    width = width or int(lens.max()) // bs + 1
    n = requests * w_out
    have = -(-lens // bs)
    blocks = int(have.sum()) + n + 2
    ids = rng.permutation(blocks).astype(np.int32)
    table = np.full((rows, width), -1, np.int32)
    at = 0
    for r in range(rows):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    parents = np.concatenate([b * w_in + rng.integers(0, w_in, w_out) for b in range(requests)]).astype(np.int32)
    parents[rng.random(n) < drop] = -1
    # any bits, the odd patterns among them
    caches = [tuple(torch.from_numpy(rng.integers(0, 256, (blocks, kvh, bs, d * DT[dtype].itemsize), np.uint8)).cuda().view(DT[dtype])
                    for _ in range(2)) for _ in range(layers)]
    return dict(parents=parents, table=table, lens=lens, spare=ids[at:at + n], caches=caches, bs=bs, blocks=blocks)


def run(s, status=None):
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    n, width = len(s["parents"]), s["table"].shape[1]
    out = (torch.full((n, width), 77, dtype=torch.int32, device="cuda"), torch.full((n,), 77, dtype=torch.int32, device="cuda"),
           torch.full((n,), 77, dtype=torch.int64, device="cuda"), torch.full((n,), 77, dtype=torch.int32, device="cuda"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    pk.pa_beam_reorder(pk.KVLayers([pk.KVCache(k, v) for k, v in s["caches"]]), dev(s["parents"]), dev(s["table"]),
                       dev(s["lens"]), dev(s["spare"]), *out, dev_status=st)
    torch.cuda.synchronize()
    if status is None:
        assert int(st) == 0
    return [o.cpu().numpy() for o in out]


def bits(x):
    return x.view(torch.uint8).cpu().numpy()


def check(s):
    before = [[bits(x) for x in pair] for pair in s["caches"]]
    got = run(s)
    t, ln, slots, used, copies = R.reorder(s["parents"], s["table"], s["lens"], s["spare"], s["bs"])
    for g, want in zip(got, (t, ln, slots, used)):
        assert np.array_equal(g, want)
    for pair, old in zip(s["caches"], before):
        for x, y in zip(pair, old):
            for a, b, rest in copies:
                y[b, :, :rest] = y[a, :, :rest]
            assert np.array_equal(bits(x), y)
    return copies


@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("kvh,d", [(1, 64), (8, 128), (3, 128)])
def test_beams(dtype, bs, kvh, d):
    lens = [0, 1, bs - 1, bs, bs + 1, 3 * bs + 5, 200]
    copies = check(state(7, 4, 4, 2, kvh, d, bs, dtype, lens, bs + d, width=14))
    assert copies
    check(state(7, 1, 5, 1, kvh, d, bs, dtype, lens, bs, width=70))   # the first step
    check(state(7, 3, 1, 1, kvh, d, bs, dtype, lens, bs))             # a best one alone


@pytest.mark.parametrize("layers", [1, 95, 96, 97, 200])
def test_layers(layers):
    check(state(2, 3, 4, layers, 2, 64, 16, "bf16", [5, 31], layers))


@pytest.mark.parametrize("d,dtype,bs", [(4, "f16", 5), (24, "e4m3", 7), (1, "e4m3", 1), (8, "bf16", 3)])
def test_other_shapes(d, dtype, bs):
    """Head and block sizes that the attention does not take, rows of any number of bytes."""
    check(state(3, 3, 5, 2, 2, d, bs, dtype, [0, 1, 2 * bs, 3 * bs + bs // 2, 9], d, width=64))


def test_many_rows():
    check(state(700, 2, 3, 1, 1, 64, 16, "f16", list(range(1, 60)), 1))
    one = state(1, 900, 900, 1, 1, 64, 16, "f16", [21], 2)
    one["parents"][:] = np.minimum(one["parents"], 40)
    check(one)


def test_all_rows_gone_and_none():
    s = state(2, 3, 3, 1, 2, 64, 16, "bf16", [20, 33], 3)
    s["parents"][:] = -1
    check(s)
    s["parents"], s["spare"] = s["parents"][:0], s["spare"][:0]
    assert run(s)[0].shape == (0, s["table"].shape[1])


def test_released_blocks_go_along():
    s = state(1, 2, 3, 1, 1, 64, 16, "bf16", [70], 4, drop=0.0)
    s["table"][:, 1:3] = -1
    check(s)


@pytest.mark.parametrize("what", ["parent", "length", "negative", "full", "spare", "source"])
def test_reported(what):
    s = state(1, 2, 3, 1, 1, 64, 16, "bf16", [37], 5, width=4, drop=0.0)
    s["parents"][:] = [1, 1, 0]
    code, bad, empty = 1, 1, True
    if what == "parent":
        s["parents"][1] = 2
    elif what == "length":
        s["lens"][1], bad = 64, None
    elif what == "full":
        s["lens"][:], s["parents"][:], bad = 64, [0, 0, 0], None
    elif what == "negative":
        s["lens"][1], bad = -1, None
    elif what == "spare":
        s["spare"][1], code, empty = s["blocks"], 6, False
    else:
        s["table"][1, 2], code, empty, bad = -1, 6, False, 0
    before = [bits(x) for x in s["caches"][0]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, ln, slots, used = run(s, status)
    assert int(status) == code
    if what == "full":
        assert (t == -1).all() and (ln == 0).all() and (slots == -1).all()
    elif empty:
        rows = [1] if bad == 1 else [0, 1]
        assert (t[rows] == -1).all() and (ln[rows] == 0).all() and (slots[rows] == -1).all()
        assert ln[2] == 38 and slots[2] == s["table"][0, 2] * 16 + 5
    else:
        assert t[bad, 2] == -1 and slots[bad] == -1 and ln[bad] == 38
        if what == "spare":
            assert all(np.array_equal(bits(x), y) for x, y in zip(s["caches"][0], before))


def test_captured():
    s = state(4, 4, 4, 3, 2, 128, 16, "bf16", [21, 32, 47, 5], 6, drop=0.0)
    want = R.reorder(s["parents"], s["table"], s["lens"], s["spare"], 16)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    a = [dev(s[k]) for k in ("parents", "table", "lens", "spare")]
    out = (torch.empty(16, s["table"].shape[1], dtype=torch.int32, device="cuda"),
           torch.empty(16, dtype=torch.int32, device="cuda"), torch.empty(16, dtype=torch.int64, device="cuda"),
           torch.empty(16, dtype=torch.int32, device="cuda"))
    layers = pk.KVLayers([pk.KVCache(k, v) for k, v in s["caches"]])
    pk.pa_beam_reorder(layers, *a, *out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_beam_reorder(layers, *a, *out)
    for o in out:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(o.cpu().numpy(), w) for o, w in zip(out, want[:4]))


def test_binding_refusals():
    s = state(2, 2, 2, 2, 2, 64, 16, "bf16", [20, 33], 7)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    a = [dev(s[k]) for k in ("parents", "table", "lens", "spare")]
    w = s["table"].shape[1]
    out = [torch.empty(4, w, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda"),
           torch.empty(4, dtype=torch.int64, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")]
    caches = [pk.KVCache(k, v) for k, v in s["caches"]]
    layers = pk.KVLayers(caches)
    with pytest.raises(TypeError):
        pk.pa_beam_reorder(caches, *a, *out)
    for i in range(4):
        bad = list(a)
        bad[i] = a[i].cpu()
        with pytest.raises(ValueError):
            pk.pa_beam_reorder(layers, *bad, *out)
        bad = list(out)
        bad[i] = out[i][:3].contiguous()
        with pytest.raises(ValueError):
            pk.pa_beam_reorder(layers, *a, *bad)
        bad = list(out)
        bad[i] = out[i].float()
        with pytest.raises(TypeError):
            pk.pa_beam_reorder(layers, *a, *bad)
    with pytest.raises(pk.PaError):
        pk.pa_beam_reorder(layers, *a, a[1], *out[1:])  # in place
    with pytest.raises(ValueError):
        pk.KVLayers([])
    with pytest.raises(ValueError):
        pk.KVLayers([caches[0], pk.KVCache(s["caches"][0][0][1:], s["caches"][0][1][1:])])
