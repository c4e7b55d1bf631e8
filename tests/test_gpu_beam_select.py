"""pa_beam_select against its definition in 64 bits.

Tolerance of a score.  Beside its one rounding to binary32 (2^-24 of itself) it carries the error of a row's
log-sum: a chunk's sum adds at most 64 exponentials a thread in binary32 (64 * 2^-24 of their sum, at the most),
each off by ex2.approx's 2^-22, and by |d| 2^-24 through its argument d = x - top rounded once and multiplied by
log2 e (2 roundings), where |d| exp(d) <= 0.37: together below 2^-17.5 of the sum, so 6e-6 of the logarithm.
Candidates nearer than twice that may stand in either order when they are of different rows; within a row the order
is that of the logits, exactly.
"""
import numpy as np
import pytest
import torch

import beam_ref as R
import paged_kv_cache_75_gb300 as pk

pytestmark = pytest.mark.gpu

LSE = 6e-6
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def call(logits, scores, cu, k, allowed=None, ended=None, end_token=0, status=None):
    B = len(cu) - 1
    out = (torch.full((B, k), 7.0, device="cuda"), torch.full((B, k), 7, dtype=torch.int32, device="cuda"),
           torch.full((B, k), 7, dtype=torch.int32, device="cuda"))
    n = pk.pa_beam_select_workspace_size(logits.shape[0], logits.shape[1], k)
    ws = torch.full((n + 16,), 0x5a, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    pk.pa_beam_select(*out, logits, scores, torch.tensor(cu, dtype=torch.int32, device="cuda"), allowed=allowed, ended=ended,
                      end_token=end_token, workspace=ws[:n], dev_status=st)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 0x5a).all())
    if status is None:
        assert int(st) == 0
    return [x.cpu().numpy() for x in out]


def words_of(allowed):
    R_, V = allowed.shape
    pad = np.zeros((R_, -(-V // 32) * 32), bool)
    pad[:, :V] = allowed
    w = np.packbits(pad.reshape(R_, -1, 32), axis=2, bitorder="little").view(np.uint32).reshape(R_, -1)
    return torch.from_numpy(w.view(np.int32).copy()).cuda()


def check(got, logits, scores, cu, k, allowed=None, ended=None, end_token=0):
    x = logits.double().cpu().numpy()
    sc = scores.cpu().numpy()
    s = R.candidate_scores(x, sc, allowed, ended, end_token)
    want = R.select(s, cu, k)
    gs, gr, gt = got
    n = want[1] >= 0
    assert np.array_equal(gr >= 0, n) and np.array_equal(gt >= 0, n)
    assert np.all(gs[~n] == -np.inf) and np.all(gr[~n] == -1) and np.all(gt[~n] == -1)
    lim = LSE + 2.0 ** -24 * np.abs(want[0][n])
    mine = s[gr[n], gt[n]]  # the chosen candidates' own scores
    assert np.all(np.abs(gs[n] - mine) <= lim)
    assert np.all(np.abs(mine - want[0][n]) <= 2 * LSE)
    for b in range(len(cu) - 1):
        m = int(n[b].sum())
        assert len({(r, t) for r, t in zip(gr[b, :m], gt[b, :m])}) == m
        assert np.all((cu[b] <= gr[b, :m]) & (gr[b, :m] < cu[b + 1]))
        assert np.all(np.diff(gs[b, :m]) <= 0)
        for r in range(cu[b], cu[b + 1]):
            # of one row: its first candidates, in the exact order
            t = gt[b, :m][gr[b, :m] == r]
            if ended is not None and ended[r]:
                assert list(t) in ([], [end_token])
                continue
            y = np.where(s[r] > -np.inf, x[r], -np.inf)
            order = np.lexsort((np.arange(len(y)), -y))[:len(t)]
            assert np.array_equal(t, order)


def values(rows, vocab, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * scale
    x[:, torch.randint(0, vocab, (5,), generator=g)] += 6.0
    return x.to(DT[dtype]), -10.0 * torch.rand(rows, generator=g)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 255, 2048, 2049, 5000, 50257])
@pytest.mark.parametrize("k", [1, 5, 64])
def test_sizes(dtype, vocab, k):
    cu = [0, 3, 3, 4, 9]
    x, sc = values(9, vocab, dtype, vocab * 3 + k)
    x, sc = x.cuda(), sc.cuda()
    check(call(x, sc, cu, k), x, sc, cu, k)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows", [400, 1300])
def test_long_chunks(dtype, rows):
    """Batches large enough for each length of chunk."""
    for vocab in (33000, 32768):
        x, sc = values(rows, vocab, dtype, rows)
        x, sc = x.cuda(), sc.cuda()
        cu = list(range(0, rows + 1, 100))
        check(call(x, sc, cu, 9), x, sc, cu, 9)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (3, 2), (8, 0), (8, 8)])
def test_strides_and_alignment(dtype, pad, off):
    x, sc = values(6, 4001, dtype, 5)
    wide = torch.full((6, 4001 + pad + off), float("nan"), dtype=DT[dtype], device="cuda")
    view = wide[:, off:off + 4001]
    view.copy_(x)
    cu = [0, 2, 6]
    got = call(view, sc.cuda(), cu, 7)
    check(got, x, sc, cu, 7)
    again = call(x.cuda(), sc.cuda(), cu, 7)
    assert all(np.array_equal(a, b) for a, b in zip(got[1:], again[1:]))


@pytest.mark.parametrize("vocab", [4096, 4097, 50257])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_equal_beams_and_equal_logits(vocab, dtype):
    """Ties go to the lower row, then the lower token, whatever the rows' addresses."""
    x, _ = values(1, vocab, dtype, 1)
    x = x.expand(4, vocab).contiguous().cuda()
    s, r, t = call(x, torch.zeros(4, device="cuda"), [0, 4], 12)
    _, _, first = call(x[:1].contiguous(), torch.zeros(1, device="cuda"), [0, 1], 3)
    order = [int(first[0, i // 4]) for i in range(12)]
    if len(set(x[0].tolist())) == vocab or x[0].topk(4).values.unique().numel() == 4:
        assert r[0].tolist() == [0, 1, 2, 3] * 3 and t[0].tolist() == order
    assert s[0, 0] == s[0, 3]
    flat = torch.zeros(3, vocab, dtype=DT[dtype], device="cuda")
    flat[:, 1::2] = -0.0
    s, r, t = call(flat, torch.zeros(3, device="cuda"), [0, 3], 64)
    assert r[0].tolist() == [0] * 64 and t[0].tolist() == list(range(64))
    assert abs(float(s[0, 0]) + np.log(vocab)) < LSE + 2.0 ** -20


def test_many_above_the_threshold():
    """The largest elements all with one thread, or more equal ones than a list holds."""
    x, sc = values(3, 20000, "bf16", 2)
    x[0, :8] = 30.0
    x[1, 100:5000] = 12.0
    x[2, 19000:] = 9.0
    x, sc = x.cuda(), sc.cuda()
    for k in (3, 64):
        check(call(x, sc, [0, 1, 2, 3], k), x, sc, [0, 1, 2, 3], k)
        check(call(x, sc, [0, 3], k), x, sc, [0, 3], k)


def test_many_beams_of_one_request():
    x, sc = values(700, 300, "f16", 3)
    sc[:] = -1.0
    x, sc = x.cuda(), sc.cuda()
    check(call(x, sc, [0, 700], 64), x, sc, [0, 700], 64)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 33, 4096, 50257])
def test_allowed(dtype, vocab):
    """Masks that leave everything, a few tokens, one, none; what they hide may be infinite or NaN."""
    x, sc = values(6, vocab, dtype, vocab)
    rng = np.random.default_rng(vocab)
    on = rng.random((6, vocab)) < 0.4
    on[1], on[2], on[3] = True, False, False
    on[3, vocab - 1] = True
    hidden = torch.from_numpy(~on & (rng.random((6, vocab)) < 0.3))
    x[hidden] = float("nan")
    x[torch.from_numpy(~on & (rng.random((6, vocab)) < 0.2))] = float("inf")
    x, sc = x.cuda(), sc.cuda()
    clean = torch.where(torch.from_numpy(on).cuda(), x, torch.zeros_like(x))
    for cu in ([0, 1, 2, 3, 4, 5, 6], [0, 3, 6]):
        check(call(x, sc, cu, 8, allowed=words_of(on)), clean, sc, cu, 8, allowed=on)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_infinite_logits_are_no_candidates(dtype):
    x, sc = values(4, 3000, dtype, 9)
    x[0, 5:] = -float("inf")
    x[1] = -float("inf")
    x[2, ::2] = -float("inf")
    x[3] = torch.finfo(DT[dtype]).min  # the type's lowest value is one
    x, sc = x.cuda(), sc.cuda()
    check(call(x, sc, [0, 1, 2, 3, 4], 9), x, sc, [0, 1, 2, 3, 4], 9)
    check(call(x, sc, [0, 4], 64), x, sc, [0, 4], 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_logits(dtype):
    """A large common part, and values at the type's ends."""
    x, sc = values(4, 3000, "f32", 10)
    x[0] += 5000.0
    x[1] -= 5000.0
    x[2, 7] = 3e38
    x[3, 9] = -3e38
    x = x.to(DT[dtype]).cuda()
    sc = sc.cuda()
    check(call(x, sc, [0, 1, 2, 3, 4], 5), x, sc, [0, 1, 2, 3, 4], 5)


def test_ended_and_absent_beams():
    x, sc = values(8, 999, "bf16", 11)
    sc[1], sc[4] = -float("inf"), -float("inf")
    ended = np.array([0, 0, 1, 0, 1, 1, 1, 0], np.uint8)
    x[2] = float("nan")  # not read
    x, sc = x.cuda(), sc.cuda()
    clean = torch.nan_to_num(x)
    for cu in ([0, 2, 5, 8], [0, 8], [0, 1, 2, 3, 4, 5, 6, 7, 8]):
        for k in (1, 6):
            for e in (torch.from_numpy(ended).cuda(), torch.from_numpy(ended).cuda().bool()):
                check(call(x, sc, cu, k, ended=e, end_token=2), clean, sc, cu, k, ended=ended, end_token=2)


@pytest.mark.parametrize("what", ["nan", "inf", "score_nan", "score_inf", "cu"])
def test_reported(what):
    x, sc = values(3, 500, "f32", 12)
    cu = [0, 1, 2, 3]
    if what == "nan":
        x[1, 400] = float("nan")
    elif what == "inf":
        x[1, 400] = float("inf")
    elif what == "score_nan":
        sc[1] = float("nan")
    elif what == "score_inf":
        sc[1] = float("inf")
    else:
        cu = [0, 1, 0, 3]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, sc = x.cuda(), sc.cuda()
    s, r, t = call(x, sc, cu, 4, status=status)
    assert int(status) == 1
    assert r[1].tolist() == [-1] * 4 and t[1].tolist() == [-1] * 4
    keep = [0] if what == "cu" else [0, 2]
    ref = R.select(R.candidate_scores(np.nan_to_num(x.double().cpu().numpy()), np.nan_to_num(sc.cpu().numpy())), [0, 1, 2, 3], 4)
    for b in keep:
        assert np.array_equal(t[b], ref[2][b]) and np.array_equal(r[b], ref[1][b])


def test_no_requests_and_no_rows():
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    i = torch.int32
    pk.pa_beam_select(e(0, 4), e(0, 4, dtype=i), e(0, 4, dtype=i), e(0, 10), e(0), torch.zeros(1, dtype=i, device="cuda"))
    out = e(2, 3), e(2, 3, dtype=i), e(2, 3, dtype=i)
    pk.pa_beam_select(*out, e(0, 10), e(0), torch.zeros(3, dtype=i, device="cuda"))
    assert bool((out[0] == -float("inf")).all()) and bool((out[1] == -1).all()) and bool((out[2] == -1).all())


def test_captured_twice_with_a_workspace_each_and_on_another_stream():
    x, sc = values(20, 9000, "bf16", 13)
    x, sc = x.cuda(), sc.cuda()
    cu = torch.tensor([0, 5, 20], dtype=torch.int32, device="cuda")
    want = call(x, sc, [0, 5, 20], 6)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    runs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            out = (torch.empty(2, 6, device="cuda"), torch.empty(2, 6, dtype=torch.int32, device="cuda"),
                   torch.empty(2, 6, dtype=torch.int32, device="cuda"))
            ws = torch.empty(pk.pa_beam_select_workspace_size(20, 9000, 6), dtype=torch.uint8, device="cuda")
            pk.pa_beam_select(*out, x, sc, cu, workspace=ws, dev_status=st)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                pk.pa_beam_select(*out, x, sc, cu, workspace=ws, dev_status=st)
            runs.append((g, out, ws))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, out, _ in runs:
            for o in out:
                o.zero_()
            g.replay()
    torch.cuda.synchronize()
    for _, out, _ in runs:
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out, want))
    assert int(st) == 0


def test_binding_refusals():
    x, sc = values(4, 64, "bf16", 14)
    x, sc = x.cuda(), sc.cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    o = [torch.empty(1, 4, device="cuda"), torch.empty(1, 4, dtype=torch.int32, device="cuda"),
         torch.empty(1, 4, dtype=torch.int32, device="cuda")]
    ws = torch.empty(pk.pa_beam_select_workspace_size(4, 64, 4), dtype=torch.uint8, device="cuda")
    f = pk.pa_beam_select
    with pytest.raises(TypeError):
        f(*o, x.double(), sc, cu, workspace=ws)
    with pytest.raises(ValueError):
        f(*o, x.t(), sc, cu, workspace=ws)
    with pytest.raises(ValueError):
        f(*o, x, sc[:3], cu, workspace=ws)
    with pytest.raises(TypeError):
        f(*o, x, sc.half(), cu, workspace=ws)
    with pytest.raises(ValueError):
        f(*o, x, sc.cpu(), cu, workspace=ws)
    with pytest.raises(ValueError):
        f(o[0], o[1][:, :3].contiguous(), o[2], x, sc, cu, workspace=ws)
    with pytest.raises(TypeError):
        f(o[0], o[1].long(), o[2], x, sc, cu, workspace=ws)
    with pytest.raises(ValueError):
        f(*o, x, sc, cu, allowed=torch.zeros(4, 1, dtype=torch.int32, device="cuda"), workspace=ws)
    with pytest.raises(TypeError):
        f(*o, x, sc, cu, ended=torch.zeros(4, device="cuda"), workspace=ws)
    with pytest.raises(pk.PaError):
        f(*o, x, sc, cu)
    with pytest.raises(pk.PaError):
        f(*o, x, sc, cu, ended=torch.zeros(4, dtype=torch.uint8, device="cuda"), end_token=64, workspace=ws)
