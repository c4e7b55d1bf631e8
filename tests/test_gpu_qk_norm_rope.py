"""pa_qk_norm_rope and pa_qk_norm_rope_write against the 64-bit formulas (GPU)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import rope_ref
from gpu_util import dev_status

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(T, H, Hkv, D, dt, seed=0, far=5000):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H + 2 * Hkv, D, generator=g) * torch.exp(0.5 * torch.randn(D, generator=g))).to(dt)
    pos = torch.randint(0, far, (T,), generator=g)
    qw, kw = 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(D, generator=g)
    return x, pos, qw, kw


def transform(rot, interleaved=False, qw=None, kw=None, eps=1e-6, **kw_rope):
    rope = pk.rope_frequencies(rot, device=DEV, **kw_rope) if rot else None
    return pk.QKTransform(rope, interleaved, None if qw is None else qw.to(DEV), None if kw is None else kw.to(DEV), eps)


def reference(x, pos, tr, weight):
    th, f = (tr.rope.theta, tr.rope.factor) if tr.rope is not None else ([], 1.0)
    return rope_ref.rows(x, pos.tolist(), th, f, tr.interleaved, weight, tr.eps)


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 64), (128, 96), (128, 128), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("norm", ["none", "both", "q", "k"])
def test_packed_rows(D, rot, interleaved, dt, norm):
    T, H, Hkv = 37, 6, 3
    x, pos, qw, kw = make(T, H, Hkv, D, TYPES[dt], seed=D + rot)
    qw, kw = (qw if norm in ("both", "q") else None), (kw if norm in ("both", "k") else None)
    tr = transform(rot, interleaved, qw, kw)
    xd = x.to(DEV)
    q, k = xd[:, :H], xd[:, H:H + Hkv]  # views of a fused buffer
    qo, ko = torch.empty(T, H, D, dtype=x.dtype, device=DEV), torch.empty(T, Hkv, D, dtype=x.dtype, device=DEV)
    pk.pa_qk_norm_rope(qo, ko, q, k, pos.to(DEV), tr)
    for got, src, w in ((qo, x[:, :H], qw), (ko, x[:, H:H + Hkv], kw)):
        ref, pair = reference(src, pos, tr, w)
        rope_ref.check(got.cpu(), ref, pair, x.dtype)
    if rot < D:
        tail = slice(rot, D)
        if qw is None:
            assert torch.equal(qo.cpu()[..., tail], x[:, :H, tail])
        if kw is None:
            assert torch.equal(ko.cpu()[..., tail], x[:, H:H + Hkv, tail])
    assert torch.equal(xd.cpu(), x)


@pytest.mark.parametrize("T", [1, 2, 5, 151, 152, 305, 2000])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (32, 8), (40, 40)])
def test_token_counts_and_heads(T, H, Hkv):
    D = 128
    x, pos, qw, kw = make(T, H, Hkv, D, torch.bfloat16, seed=T)
    tr = transform(D, False, qw, kw)
    xd = x.to(DEV)
    qo, ko = torch.empty(T, H, D, dtype=x.dtype, device=DEV), torch.empty(T, Hkv, D, dtype=x.dtype, device=DEV)
    pk.pa_qk_norm_rope(qo, ko, xd[:, :H], xd[:, H:H + Hkv], pos.to(DEV), tr)
    sample = sorted({0, T - 1, T // 2, T // 3, *range(0, T, max(1, T // 40))})
    for got, src, w in ((qo, x[:, :H], qw), (ko, x[:, H:H + Hkv], kw)):
        ref, pair = reference(src[sample], pos[sample], tr, w)
        rope_ref.check(got.cpu()[sample], ref, pair, x.dtype)


@pytest.mark.parametrize("T", [2431, 2432, 2433, 4864, 7001])
@pytest.mark.parametrize("D,H,Hkv", [(128, 32, 8), (64, 5, 3), (128, 1, 1)])
@pytest.mark.parametrize("write", [False, True])
def test_many_tokens_equal_few(T, D, H, Hkv, write):
    """Counts around whole rounds of the resident warps (and past several): the same bits as in calls of a few hundred
    tokens each, which hold no whole round."""
    dt, bs = torch.bfloat16, 16
    x, pos, qw, kw = make(T, H, Hkv, D, dt, seed=T)
    tr = transform(D // 2, D == 64, qw, kw)
    xd, pd = x.to(DEV), pos.to(DEV)
    g = torch.Generator().manual_seed(1)
    nb = T // bs + 2
    slots = torch.randperm(nb * bs, generator=g)[:T].to(DEV)
    slots[::11] = -1
    res = []
    for step in (T, 300):
        qo = torch.zeros(T, H, D, dtype=dt, device=DEV)
        if write:
            cache = pk.KVCache(torch.zeros(nb, Hkv, bs, D, dtype=dt, device=DEV), torch.zeros(nb, Hkv, bs, D, dtype=dt, device=DEV))
            out = (qo, cache.k_cache, cache.v_cache)
        else:
            ko = torch.zeros(T, Hkv, D, dtype=dt, device=DEV)
            out = (qo, ko)
        for a in range(0, T, step):
            b = min(T, a + step)
            q, k, v = xd[a:b, :H], xd[a:b, H:H + Hkv], xd[a:b, H + Hkv:]
            if write:
                pk.pa_qk_norm_rope_write(qo[a:b], q, k, v, cache, pd[a:b], slots[a:b], tr)
            else:
                pk.pa_qk_norm_rope(qo[a:b], ko[a:b], q, k, pd[a:b], tr)
        res.append(out)
    for a, b in zip(*res):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    sample = [0, 1, T // 2, T - 2, T - 1]
    ref, pair = reference(x[sample, :H], pos[sample], tr, qw)
    rope_ref.check(res[0][0].cpu()[sample], ref, pair, dt)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("D,H,Hkv,bs", [(128, 8, 2, 16), (64, 4, 4, 32), (128, 32, 8, 64), (64, 3, 1, 5)])
@pytest.mark.parametrize("T", [1, 45, 400])
def test_write_to_the_cache(kv, D, H, Hkv, bs, T):
    dt = torch.bfloat16 if kv == "e4m3" else TYPES[kv]
    kd = torch.float8_e4m3fn if kv == "e4m3" else dt
    x, pos, qw, kw = make(T, H, Hkv, D, dt, seed=bs + T)
    rot = D // 2
    tr = transform(rot, bs == 32, qw, kw, scaling="linear", factor=4.0)
    ks, vs = (0.04, 0.3) if kv == "e4m3" else (1.0, 1.0)
    nb = T // bs + 3
    g = torch.Generator().manual_seed(9)
    bits = torch.uint8 if kv == "e4m3" else torch.int16
    kc0 = torch.randn(nb, Hkv, bs, D, generator=g).to(kd)
    vc0 = torch.randn(nb, Hkv, bs, D, generator=g).to(kd)
    slots = torch.randperm(nb * bs, generator=g)[:T]
    slots[::7] = -5  # padding: queries still come out
    cache = pk.KVCache(kc0.to(DEV), vc0.to(DEV), ks, vs)
    xd = x.to(DEV)
    q, k, v = xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:]
    qo = torch.empty(T, H, D, dtype=dt, device=DEV)
    st = dev_status()
    pk.pa_qk_norm_rope_write(qo, q, k, v, cache, pos.to(DEV), slots.to(DEV), tr, st)
    assert st.item() == 0
    ref, pair = reference(x[:, :H], pos, tr, qw)
    rope_ref.check(qo.cpu(), ref, pair, dt, "q")
    real = slots >= 0
    at = slots[real]
    got_k, got_v = cache.k_cache.cpu(), cache.v_cache.cpu()
    ref, pair = reference(x[:, H:H + Hkv], pos, tr, kw)
    mine = got_k.view(bits)[at // bs, :, at % bs].view(kd)
    rope_ref.check(mine, ref[real] / ks, pair[real] / ks, kd, "k")
    # values: as pa_kv_cache_write stores them, bit for bit; and nothing else is touched
    vals = pk.KVCache(kc0.to(DEV), vc0.to(DEV), ks, vs)
    pk.pa_kv_cache_write(vals, k, v, slots.to(DEV), st)
    assert torch.equal(got_v.view(bits), vals.v_cache.cpu().view(bits))
    touched = torch.zeros(nb, bs, dtype=torch.bool)
    touched[at // bs, at % bs] = True
    keep = ~touched[:, None, :, None].expand(nb, Hkv, bs, D)
    assert torch.equal(got_k.view(bits)[keep], kc0.view(bits)[keep])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("ks,vs", [(1.0, 1.0), (0.25, 4.0), (3.0, 0.7), (2.0 ** -126, 2.0 ** 126), (2.0 ** -20, 2.0 ** 127)])
def test_e4m3_scales(dt, ks, vs):
    """Scales that are powers of two and not, at the ends of the range: keys and values that nothing turns are stored
    as pa_kv_cache_write stores them, bit for bit, saturated ones, subnormal ones and infinities among them."""
    T, H, Hkv, D, bs = 50, 2, 2, 128, 16
    x, pos, _, _ = make(T, H, Hkv, D, TYPES[dt], seed=3)
    x[5, :, 3], x[6, :, 4], x[7] = float("inf"), float("-inf"), x[7] * 1000
    x[8] = (x[8].float() * 2.0 ** -12).to(x.dtype)
    xd = x.to(DEV)
    q, k, v = xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:]
    zero = torch.zeros(4, Hkv, bs, D, device=DEV).to(torch.float8_e4m3fn)
    a, b = pk.KVCache(zero.clone(), zero.clone(), ks, vs), pk.KVCache(zero.clone(), zero.clone(), ks, vs)
    slots = torch.arange(T, device=DEV) + 5
    pk.pa_qk_norm_rope_write(torch.empty_like(q.contiguous()), q, k, v, a, pos.to(DEV), slots, pk.QKTransform())
    pk.pa_kv_cache_write(b, k, v, slots)
    assert torch.equal(a.k_cache.view(torch.uint8), b.k_cache.view(torch.uint8))
    assert torch.equal(a.v_cache.view(torch.uint8), b.v_cache.view(torch.uint8))


def test_slots_past_the_cache_are_reported_and_skipped():
    T, H, Hkv, D, bs = 9, 4, 2, 128, 16
    x, pos, qw, kw = make(T, H, Hkv, D, torch.float16)
    tr = transform(64, False, qw, kw)
    kc = torch.zeros(2, Hkv, bs, D, dtype=torch.float16)
    cache = pk.KVCache(kc.to(DEV), kc.to(DEV))
    slots = torch.tensor([0, 1, 32, 2, -1, 1 << 40, 3, 31, 33])
    xd = x.to(DEV)
    qo = torch.empty(T, H, D, dtype=x.dtype, device=DEV)
    st = dev_status()
    pk.pa_qk_norm_rope_write(qo, xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:], cache, pos.to(DEV), slots.to(DEV), tr, st)
    assert st.item() == 6
    ref, pair = reference(x[:, :H], pos, tr, qw)
    rope_ref.check(qo.cpu(), ref, pair, x.dtype)
    written = cache.v_cache.cpu().permute(0, 2, 1, 3).reshape(32, -1).abs().sum(-1) > 0
    assert written.nonzero().flatten().tolist() == [0, 1, 2, 3, 31]


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_strides_and_alignments(offset, pad, D):
    """Every tensor a view at an odd place with an odd token stride; the gaps stay as they were."""
    T, H, Hkv, bs = 21, 3, 2, 16
    dt = torch.bfloat16
    x, pos, qw, kw = make(T, H, Hkv, D, dt, seed=pad)
    tr = transform(32, False, qw, kw)

    def strided(n, fill):
        row = n * D + pad
        flat = torch.full((offset + T * row + 8,), fill, dtype=dt, device=DEV)
        return flat, flat[offset:offset + T * row].view(T, row)[:, :n * D].view(T, n, D) if pad == 0 else \
            torch.as_strided(flat, (T, n, D), (row, D, 1), offset)

    (_, q), (_, k), (_, v) = strided(H, 0.0), strided(Hkv, 0.0), strided(Hkv, 0.0)
    q.copy_(x[:, :H]), k.copy_(x[:, H:H + Hkv]), v.copy_(x[:, H + Hkv:])
    (fq, qo), (fk, ko) = strided(H, 7.0), strided(Hkv, 7.0)
    pk.pa_qk_norm_rope(qo, ko, q, k, pos.to(DEV), tr)
    for got, src, w in ((qo, x[:, :H], qw), (ko, x[:, H:H + Hkv], kw)):
        ref, pair = reference(src, pos, tr, w)
        rope_ref.check(got.cpu(), ref, pair, dt)
    for flat, n in ((fq, H), (fk, Hkv)):
        mask = torch.ones(flat.numel(), dtype=torch.bool)
        for t in range(T):
            a = offset + t * (n * D + pad)
            mask[a:a + n * D] = False
        assert bool((flat.cpu()[mask] == 7.0).all())
    kc = torch.zeros(2, Hkv, bs, D, dtype=dt, device=DEV)
    cache = pk.KVCache(kc, kc.clone())
    slots = torch.arange(T, device=DEV) + 3
    qo2 = torch.empty_like(qo.contiguous())
    pk.pa_qk_norm_rope_write(qo2, q, k, v, cache, pos.to(DEV), slots, tr)
    assert torch.equal(qo2, qo) and torch.equal(kc.permute(0, 2, 1, 3).reshape(32, Hkv, D)[3:3 + T], ko)
    assert torch.equal(cache.v_cache.permute(0, 2, 1, 3).reshape(32, Hkv, D)[3:3 + T], v)


@pytest.mark.parametrize("odd", ["q", "k", "v", "q_out"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (5, 2), (4, 4)])
def test_one_tensor_unaligned_beside_aligned_ones(odd, H, Hkv):
    T, D, bs = 9, 128, 16
    x, pos, qw, kw = make(T, H, Hkv, D, torch.float16, seed=H)
    tr = transform(64, False, qw, kw)

    def place(src, name):
        n = src.shape[1]
        flat = torch.zeros(T * n * D + 8, dtype=src.dtype, device=DEV)
        at = flat[1:1 + T * n * D] if odd == name else flat[:T * n * D]
        return at.view(T, n, D).copy_(src)

    q, k, v = place(x[:, :H], "q"), place(x[:, H:H + Hkv], "k"), place(x[:, H + Hkv:], "v")
    qo = place(torch.zeros(T, H, D, dtype=x.dtype), "q_out")
    kc = torch.zeros(2, Hkv, bs, D, dtype=x.dtype, device=DEV)
    cache = pk.KVCache(kc, kc.clone())
    pk.pa_qk_norm_rope_write(qo, q, k, v, cache, pos.to(DEV), torch.arange(T, device=DEV), tr)
    ref, pair = reference(x[:, :H], pos, tr, qw)
    rope_ref.check(qo.cpu(), ref, pair, x.dtype)
    ref, pair = reference(x[:, H:H + Hkv], pos, tr, kw)
    rope_ref.check(kc.cpu()[0, :, :T].transpose(0, 1), ref, pair, x.dtype)
    assert torch.equal(cache.v_cache.cpu()[0, :, :T].transpose(0, 1), x[:, H + Hkv:])


def test_in_place_equals_out_of_place():
    T, H, Hkv, D = 300, 32, 8, 128
    x, pos, qw, kw = make(T, H, Hkv, D, torch.bfloat16)
    tr = transform(128, False, qw, kw)
    a, b = x.to(DEV), x.to(DEV)
    qo, ko = torch.empty(T, H, D, dtype=x.dtype, device=DEV), torch.empty(T, Hkv, D, dtype=x.dtype, device=DEV)
    pk.pa_qk_norm_rope(qo, ko, a[:, :H], a[:, H:H + Hkv], pos.to(DEV), tr)
    pk.pa_qk_norm_rope(b[:, :H], b[:, H:H + Hkv], b[:, :H], b[:, H:H + Hkv], pos.to(DEV), tr)
    assert torch.equal(b[:, :H], qo) and torch.equal(b[:, H:H + Hkv], ko)
    assert torch.equal(b[:, H + Hkv:].cpu(), x[:, H + Hkv:])


@pytest.mark.parametrize("pos", [0, -1, -4096, 131071, 1 << 20, (1 << 31) + 5, -(1 << 40), (1 << 62) + 12345])
def test_far_positions(pos):
    T, H, Hkv, D = 2, 2, 1, 128
    x, _, qw, kw = make(T, H, Hkv, D, torch.float16, seed=4)
    tr = transform(128, True, qw, kw)
    p = torch.tensor([pos, pos + 1])
    xd = x.to(DEV)
    qo, ko = torch.empty(T, H, D, dtype=x.dtype, device=DEV), torch.empty(T, Hkv, D, dtype=x.dtype, device=DEV)
    pk.pa_qk_norm_rope(qo, ko, xd[:, :H], xd[:, H:H + Hkv], p.to(DEV), tr)
    # the angle that the stored 64-bit turns give (theta has 53 bits: 2^62 positions of it are no angle)
    turns = tr.rope.turns.cpu().numpy().view(np.uint64)
    if abs(pos) < 1 << 41:
        ref, pair = rope_ref.rows(x[:, :H], p.tolist(), tr.rope.theta, 1.0, True, qw, tr.eps)
        # theta's 53 bits over pos positions
        pair = pair * (1 + abs(pos) * 2.0 ** -52 * 2.0 ** 24 / rope_ref.FP32_UNITS)
        rope_ref.check(qo.cpu(), ref, pair, x.dtype)
    else:
        ang = np.array([[((int(q) * int(u)) % 2 ** 64) / 2 ** 64 * 2 * np.pi for u in turns] for q in p.tolist()])
        y = x[:, :H].double()
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + tr.eps) * qw.double()
        co, si = torch.from_numpy(np.cos(ang))[:, None], torch.from_numpy(np.sin(ang))[:, None]
        ref = torch.stack((y[..., 0::2] * co - y[..., 1::2] * si, y[..., 1::2] * co + y[..., 0::2] * si), -1).flatten(-2)
        pair = (y[..., 0::2].abs() + y[..., 1::2].abs()).repeat_interleave(2, -1)
        rope_ref.check(qo.cpu(), ref, pair, x.dtype)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1e30, 3e38])
def test_row_sizes(size):
    """Rows whose squares leave binary32's range: the norm still stands."""
    T, H, Hkv, D = 4, 2, 2, 128
    x, pos, qw, kw = make(T, H, Hkv, D, torch.bfloat16)
    x = (x.float() / x.float().abs().max() * size).to(torch.bfloat16)
    x[1, 0] = 0.0
    tr = transform(64, False, qw, kw, eps=1e-12)
    xd = x.to(DEV)
    qo, ko = torch.empty(T, H, D, dtype=x.dtype, device=DEV), torch.empty(T, Hkv, D, dtype=x.dtype, device=DEV)
    pk.pa_qk_norm_rope(qo, ko, xd[:, :H], xd[:, H:H + Hkv], pos.to(DEV), tr)
    for got, src, w in ((qo, x[:, :H], qw), (ko, x[:, H:H + Hkv], kw)):
        ref, pair = reference(src, pos, tr, w)
        rope_ref.check(got.cpu(), ref, pair, x.dtype)


def test_a_row_with_nan_or_infinity_keeps_to_itself():
    T, H, Hkv, D = 6, 4, 4, 64
    x, pos, qw, kw = make(T, H, Hkv, D, torch.float16)
    clean = x.clone()
    x[2, 1, 5], x[3, H + 2, 60], x[4, H + Hkv, 3] = float("nan"), float("inf"), float("nan")
    tr = transform(32, False, qw, kw)
    out = []
    for src in (x, clean):
        xd = src.to(DEV)
        kc = torch.zeros(1, Hkv, 16, D, dtype=x.dtype, device=DEV)
        cache = pk.KVCache(kc, kc.clone())
        qo = torch.empty(T, H, D, dtype=x.dtype, device=DEV)
        pk.pa_qk_norm_rope_write(qo, xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:], cache, pos.to(DEV),
                                 torch.arange(T, device=DEV), tr)
        out.append((qo.cpu(), cache.k_cache.cpu(), cache.v_cache.cpu()))
    (q1, k1, v1), (q0, k0, v0) = out
    assert bool(q1[2, 1].isnan().all()) and not bool(k1[0, 2, 3].isfinite().all())
    q1[2, 1], k1[0, 2, 3] = q0[2, 1], k0[0, 2, 3]
    assert torch.equal(q1, q0) and torch.equal(k1, k0)
    assert torch.equal(v1[0, :, 4].view(torch.int16), x[4, H + Hkv:].view(torch.int16))


def test_no_tokens_and_no_change():
    D, H, Hkv = 128, 4, 2
    x, pos, _, _ = make(8, H, Hkv, D, torch.float16)
    xd = x.to(DEV)
    q, k = xd[:, :H], xd[:, H:H + Hkv]
    pk.pa_qk_norm_rope(q[:0], k[:0], q[:0], k[:0], pos.to(DEV)[:0], transform(64))
    qo, ko = torch.empty(8, H, D, dtype=x.dtype, device=DEV), torch.empty(8, Hkv, D, dtype=x.dtype, device=DEV)
    pk.pa_qk_norm_rope(qo, ko, q, k, None, transform(0))
    assert torch.equal(qo.cpu(), x[:, :H]) and torch.equal(ko.cpu(), x[:, H:H + Hkv])


def test_captured_replayed_and_on_another_stream():
    T, H, Hkv, D = 64, 8, 2, 128
    x, pos, qw, kw = make(T, H, Hkv, D, torch.bfloat16)
    tr = transform(128, False, qw, kw)
    xd, pd = x.to(DEV), pos.to(DEV)
    qo, ko = torch.empty(T, H, D, dtype=x.dtype, device=DEV), torch.empty(T, Hkv, D, dtype=x.dtype, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pk.pa_qk_norm_rope(qo, ko, xd[:, :H], xd[:, H:H + Hkv], pd, tr)
    s.synchronize()
    want_q, want_k = qo.clone(), ko.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.pa_qk_norm_rope(qo, ko, xd[:, :H], xd[:, H:H + Hkv], pd, tr)
    qo.zero_(), ko.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    pd.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    ref, pair = reference(x[:, :H], pos + 17, tr, qw)
    rope_ref.check(qo.cpu(), ref, pair, x.dtype)


def test_the_binding_refuses_wrong_tensors():
    T, H, Hkv, D = 4, 4, 2, 128
    x, pos, qw, kw = make(T, H, Hkv, D, torch.float16)
    xd, pd = x.to(DEV), pos.to(DEV)
    q, k = xd[:, :H], xd[:, H:H + Hkv]
    qo, ko = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    tr = transform(128, False, qw, kw)
    with pytest.raises(ValueError):
        pk.pa_qk_norm_rope(qo, ko, q, k, pd[:3], tr)
    with pytest.raises(ValueError):
        pk.pa_qk_norm_rope(qo[:, :3], ko, q, k, pd, tr)
    with pytest.raises(ValueError):
        pk.pa_qk_norm_rope(qo, ko.bfloat16(), q, k, pd, tr)
    with pytest.raises(ValueError):
        pk.pa_qk_norm_rope(qo, ko, q.transpose(1, 2).contiguous().transpose(1, 2), k, pd, tr)
    with pytest.raises(TypeError):
        pk.pa_qk_norm_rope(qo, ko, q, k, pd.int(), tr)
    with pytest.raises(ValueError):
        pk.pa_qk_norm_rope(qo, ko, q, k, pd, pk.QKTransform(q_weight=torch.ones(64, device=DEV)))
    with pytest.raises(TypeError):
        pk.QKTransform(q_weight=torch.ones(128, device=DEV, dtype=torch.float16))
    with pytest.raises(pk.PaError):
        pk.pa_qk_norm_rope(qo, ko, q, k, None, tr)
    cache = pk.KVCache(torch.zeros(2, Hkv, 16, 64, dtype=torch.float16, device=DEV),
                       torch.zeros(2, Hkv, 16, 64, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        pk.pa_qk_norm_rope_write(qo, q, k, k, cache, pd, torch.arange(T, device=DEV), tr)


@pytest.mark.parametrize("size,eps", [(2e19, 1e38), (3e18, 3.3e38), (3e38, 3.4e38), (1.0, 3e38), (1e-3, 1e-30), (1e-18, 1e-36),
                                      (1e-21, 1e-45), (2e-22, 1e-45), (1e-25, 1e-45), (1e-37, 1e-40), (3e-39, 1e-20), (3e-39, 1e-45)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_eps_and_rows_of_any_size(size, eps, interleaved):
    """Any eps > 0 beside any row: neither the sum of the two nor the squares need fit binary32."""
    T, H, Hkv, D = 5, 3, 2, 64
    x, pos, qw, kw = make(T, H, Hkv, D, torch.bfloat16, seed=4)
    x = (x.float() / x.float().abs().max() * size).to(torch.bfloat16)
    x[1, 0], x[2] = 0.0, torch.randn(H + 2 * Hkv, D, generator=torch.Generator().manual_seed(1))
    tr = transform(32, interleaved, qw, kw, eps=float(np.float32(eps)))
    xd = x.to(DEV)
    qo, ko = torch.empty(T, H, D, dtype=x.dtype, device=DEV), torch.empty(T, Hkv, D, dtype=x.dtype, device=DEV)
    pk.pa_qk_norm_rope(qo, ko, xd[:, :H], xd[:, H:H + Hkv], pos.to(DEV), tr)
    for got, src, w in ((qo, x[:, :H], qw), (ko, x[:, H:H + Hkv], kw)):
        ref, pair = reference(src, pos, tr, w)
        rope_ref.check(got.cpu(), ref, pair, x.dtype)
