"""Measured cases of four operators around the paged cache.

* ``qk_norm_rope``        norms of the queries and keys of each head and the position rotation in one pass,
                          over packed rows (what goes to varlen attention over packed K/V)
* ``qk_norm_rope_write``  the same, with the keys and the values written to their cache slots
* ``decode_window``       single-query attention over the paged cache with a sliding window and a few first
                          tokens that stay visible (sinks)
* ``prefill_window``      causal varlen attention over the paged cache under the same mask

``run`` computes the plain form (elementary torch operations, 32 bits) where ``own`` is false, and makes the
library's calls where it is true.  ``exact`` is the definition in 64 bits, written apart from the plain form.
Sequence lengths follow from the case alone; values, block tables, positions and slots follow from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ----------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------
def _rope(op, tokens, heads, kv_heads, head_size, dtype, rotary, **more):
    c = dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, head_size=head_size, dtype=dtype, rotary=rotary,
             interleaved=False, norm=True, scaling="none", base=10000.0, max_position=4096, block_size=16,
             kv_dtype=dtype, fused_qkv=True)
    c.update(more)
    return c


def _attn(op, seqs, heads, kv_heads, head_size, dtype, window, sinks, lens, **more):
    c = dict(op=op, seqs=seqs, heads=heads, kv_heads=kv_heads, head_size=head_size, dtype=dtype, kv_dtype=dtype,
             window=window, sinks=sinks, lens=lens, lo=1, hi=2048, lens_seed=0, block_size=16, released=True)
    c.update(more)
    return c


def listed():
    return [
        # one new token of one sequence: the latency of a decode step's projections
        dict(_rope("qk_norm_rope_write", 1, 32, 8, 128, "bf16", 128), name="write_1tok"),
        # a decode batch of 256 sequences into an E4M3 cache; adjacent pairs rotated, half of the head, and the
        # positions of a long context stretched by the dimension ramp
        dict(_rope("qk_norm_rope_write", 256, 32, 8, 128, "bf16", 64, interleaved=True, kv_dtype="e4m3", block_size=32,
                   scaling="yarn", max_position=131072), name="write_256tok_e4m3"),
        # a prefill chunk: 16k tokens of several prompts in one call
        dict(_rope("qk_norm_rope_write", 16384, 32, 8, 128, "bf16", 128, base=500000.0, scaling="banded",
                   max_position=131072), name="write_16k"),
        # packed rows of a first prefill, rotation alone, an odd count of tokens, as many key as query heads
        dict(_rope("qk_norm_rope", 5461, 32, 32, 128, "f16", 128, norm=False, fused_qkv=False), name="rope_5461_mha"),
        # small heads, a quarter of each rotated, positions scaled linearly
        dict(_rope("qk_norm_rope", 333, 16, 4, 64, "f16", 16, scaling="linear", max_position=16384), name="rope_333_d64"),
        # the three-sequence batch of the decode worked example, with a window shorter than its longest sequence
        dict(_attn("decode_window", 3, 4, 4, 64, "f16", 24, 4, "tiny", block_size=32), name="decode_tiny"),
        # the single-head-per-KV-head decode batch: lengths uniform up to 2048, many shorter than the window
        dict(_attn("decode_window", 64, 32, 32, 128, "f16", 1024, 4, "uniform", lens_seed=2000), name="decode_mha"),
        # a serving batch of 256 sequences, log-normal lengths, window of 1024
        dict(_attn("decode_window", 256, 32, 8, 128, "bf16", 1024, 4, "lognormal", lo=16, hi=8192, lens_seed=3000),
             name="decode_gqa"),
        # eight long contexts over an E4M3 cache, the whole of which is kept; a wide window
        dict(_attn("decode_window", 8, 64, 8, 128, "bf16", 8192, 64, "uniform", lo=32768, hi=131072, kv_dtype="e4m3",
                   block_size=32, lens_seed=4000, released=False), name="decode_long_e4m3"),
        # three short odd prompts: the latency of a small prefill
        dict(_attn("prefill_window", 3, 8, 2, 128, "f16", 33, 3, "uniform", lo=5, hi=211, q_lo=5, q_hi=97, lens_seed=7),
             name="prefill_small"),
        # eight prefill chunks on up to 4096 cached tokens, a window of 1024
        dict(_attn("prefill_window", 8, 32, 8, 128, "bf16", 1024, 4, "prior", lo=0, hi=4096, q_lo=512, q_hi=2048,
                   lens_seed=5000), name="prefill_mixed"),
        # one long prompt from its first token, a wide window
        dict(_attn("prefill_window", 1, 32, 8, 128, "bf16", 2048, 16, "uniform", lo=8192, hi=8192, q_lo=8192, q_hi=8192,
                   block_size=32, lens_seed=1), name="prefill_8k"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope_write", "qk_norm_rope", "decode_window", "prefill_window"])
    dtype = rng.choice(["f16", "bf16"])
    kvh = rng.choice([1, 2, 4, 8])
    heads = kvh * rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32, 64])
    if op.startswith("qk"):
        d = rng.choice([64, 128])
        return _rope(op, _log(rng, 1, 12288), heads, kvh, d, dtype, 16 * rng.randint(1, d // 16),
                     interleaved=rng.random() < 0.5, norm=rng.random() < 0.7,
                     scaling=rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
                     base=rng.choice([10000.0, 500000.0]), max_position=_log(rng, 256, 1 << 20), block_size=bs,
                     kv_dtype=rng.choice([dtype, dtype, "e4m3"]), fused_qkv=rng.random() < 0.6)
    window, sinks = _log(rng, 1, 2560), rng.choice([0, 1, 4, 17, 64])
    seed = rng.randrange(1 << 30)
    if op == "decode_window":
        hi = _log(rng, 16, 16384)
        return _attn(op, _log(rng, 1, 64), heads, kvh, rng.choice([64, 128]), dtype, window, sinks, "uniform",
                     lo=0, hi=hi, block_size=bs, kv_dtype=rng.choice([dtype, dtype, "e4m3"]), lens_seed=seed,
                     released=rng.random() < 0.7)
    q_hi = _log(rng, 1, 512)
    return _attn(op, rng.randint(1, 4), heads, kvh, 128, dtype, window, sinks, "prior", lo=0, hi=_log(rng, 1, 4096),
                 q_lo=1, q_hi=q_hi, block_size=bs, lens_seed=seed, released=rng.random() < 0.7)


def _lengths(c):
    """Key lengths and query lengths of an attention case."""
    g = np.random.default_rng(c["lens_seed"])
    n = c["seqs"]
    if c["lens"] == "tiny":
        lk = np.array([31, 33, 71])
    elif c["lens"] == "lognormal":
        lk = np.clip(np.rint(np.exp(math.log(1000.0) + g.standard_normal(n))), c["lo"], c["hi"]).astype(np.int64)
    else:
        lk = g.integers(c["lo"], c["hi"] + 1, size=n)
    if c["op"] == "decode_window":
        return lk, np.ones(n, np.int64)
    lq = g.integers(c["q_lo"], c["q_hi"] + 1, size=n)
    if c["lens"] == "prior":
        return lk + lq, lq
    return np.maximum(lk, lq), lq


# ----------------------------------------------------------------------------------------------------------
# frequencies of the rotation (a host list that a program keeps)
# ----------------------------------------------------------------------------------------------------------
SCALING = {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=8.0),
           "yarn": dict(factor=16.0, original_max_position=8192, beta_fast=32.0, beta_slow=1.0),
           "banded": dict(factor=8.0, original_max_position=8192, low_freq_factor=1.0, high_freq_factor=4.0)}


def _inv_freq(c):
    """Radians per position of each rotated pair, and the factor of cos and sin."""
    rot, base, kind = c["rotary"], c["base"], c["scaling"]
    s = SCALING[kind]
    if kind == "ntk":
        base = base * s["factor"] ** (rot / (rot - 2.0))
    th = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        return [t / s["factor"] for t in th], 1.0
    if kind == "yarn":
        at = lambda r: rot * math.log(s["original_max_position"] / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(s["beta_fast"])), 0), min(math.ceil(at(s["beta_slow"])), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        return [t / s["factor"] * r + t * (1 - r) for t, r in zip(th, ramp)], 0.1 * math.log(s["factor"]) + 1.0
    if kind == "banded":
        out = []
        for t in th:
            turns = s["original_max_position"] * t / (2 * math.pi)
            w = (turns - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])
            w = min(max(w, 0.0), 1.0)
            out.append((1 - w) * t / s["factor"] + w * t)
        return out, 1.0
    return th, 1.0


# ----------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------
def _cast(x, dtype):
    return (x.clamp_(-448.0, 448.0) if dtype == torch.float8_e4m3fn else x).to(dtype)


def _prepare_rope(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t, h, kvh, d, bs = c["tokens"], c["heads"], c["kv_heads"], c["head_size"], c["block_size"]
    dt, write = DTYPE[c["dtype"]], c["op"] == "qk_norm_rope_write"
    # channels of unlike size, as projections have them
    chan = torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))
    rows = h + kvh + (kvh if write else 0)
    x = torch.randn(t, rows, d, generator=g, device=DEV).mul_(chan).to(dt)
    s = dict(case=c, x=x)
    if c["fused_qkv"]:
        # views of one projection's output
        s["q"], s["k"] = x[:, :h], x[:, h:h + kvh]
        s["v"] = x[:, h + kvh:] if write else None
    else:
        s["q"], s["k"] = x[:, :h].contiguous(), x[:, h:h + kvh].contiguous()
        s["v"] = x[:, h + kvh:].contiguous() if write else None
    # tokens of sequences that stand at unlike positions, four in a row each
    first = torch.randint(0, c["max_position"], ((t + 3) // 4,), generator=g, device=DEV)
    s["positions"] = (first.repeat_interleave(4)[:t] + torch.arange(t, device=DEV) % 4).contiguous()
    s["qw"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV) if c["norm"] else None
    s["kw"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV) if c["norm"] else None
    s["eps"] = 1e-6
    freq, s["factor"] = _inv_freq(c)
    s["inv_freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
    s["q_out"] = torch.empty(t, h, d, dtype=dt, device=DEV)
    if write:
        kd = DTYPE[c["kv_dtype"]]
        blocks = -(-t // bs) + 1
        # a block that no token of the call goes to stays as it was
        shape = (blocks, kvh, bs, d)
        s["k_cache"] = _cast(torch.randn(shape, generator=g, device=DEV), kd)
        s["v_cache"] = _cast(torch.randn(shape, generator=g, device=DEV), kd)
        ids = torch.randperm(blocks, generator=g, device=DEV)[:blocks - 1]
        tok = torch.arange(t, device=DEV)
        s["slots"] = ids[tok // bs] * bs + tok % bs
        if t > 8:
            s["slots"][t // 2] = -1  # padding
        s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if c["kv_dtype"] == "e4m3" else (1.0, 1.0)
    else:
        s["k_out"] = torch.empty(t, kvh, d, dtype=dt, device=DEV)
    if own:
        import paged_kv_cache_75_gb300 as pk

        s["transform"] = pk.QKTransform(
            rope=pk.rope_frequencies(c["rotary"], c["base"], scaling=c["scaling"], device=DEV, **SCALING[c["scaling"]]),
            interleaved=c["interleaved"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"])
        if write:
            s["cache"] = pk.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
            s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def _kept(c, L, first):
    """Which blocks of a sequence of L keys hold a position that a query from position `first` on sees."""
    bs = c["block_size"]
    j = np.arange(-(-int(L) // bs))
    return (j * bs < min(c["sinks"], L)) | ((j + 1) * bs > max(0, first - c["window"] + 1))


def _prepare_attn(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    lk, lq = _lengths(c)
    bs, d, dt, kd = c["block_size"], c["head_size"], DTYPE[c["dtype"]], DTYPE[c["kv_dtype"]]
    width = max(1, max(-(-int(x) // bs) for x in lk))
    table = np.full((c["seqs"], width), -1, np.int32)
    rows = []
    for b in range(c["seqs"]):
        n = -(-int(lk[b]) // bs)
        keep = _kept(c, lk[b], int(lk[b] - lq[b])) if c["released"] else np.ones(n, bool)
        rows.append(np.flatnonzero(keep))
    total = sum(len(r) for r in rows)
    ids = rng.permutation(total + 3).astype(np.int32)
    at = 0
    for b, r in enumerate(rows):
        table[b, r] = ids[at:at + len(r)]
        at += len(r)
    shape = (total + 3, c["kv_heads"], bs, d)
    s = dict(case=c, max_k=int(max(1, lk.max())), max_q=int(lq.max()), scale=d ** -0.5)
    s["k_cache"] = _cast(torch.randn(shape, generator=g, device=DEV), kd)
    s["v_cache"] = _cast(torch.randn(shape, generator=g, device=DEV), kd)
    s["q"] = torch.randn(int(lq.sum()), c["heads"], d, generator=g, device=DEV).to(dt)
    s["out"] = torch.empty_like(s["q"])
    s["table"] = torch.from_numpy(table).to(DEV)
    s["lens"] = torch.from_numpy(lk.astype(np.int32)).to(DEV)
    cum = lambda a: torch.from_numpy(np.concatenate([[0], np.cumsum(a)]).astype(np.int32)).to(DEV)  # noqa: E731
    s["cu_q"], s["cu_k"] = cum(lq), cum(lk)
    s["k_scale"] = s["v_scale"] = 1.0
    if own:
        import paged_kv_cache_75_gb300 as pk

        s["cache"] = pk.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if c["op"] == "decode_window":
            n = pk.pa_decode_window_workspace_size(c["seqs"], c["heads"], d, s["max_k"], bs, c["window"], c["sinks"])
            s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    return _prepare_rope(case, seed) if case["op"].startswith("qk") else _prepare_attn(case, seed)


# ----------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------
def _norm_rotate(x, w, s):
    c = s["case"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w
    rot = c["rotary"]
    ang = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = (ang.cos() * s["factor"]).float()[:, None], (ang.sin() * s["factor"]).float()[:, None]
    if c["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _put(cache, x, scale, slots, bs):
    real = slots >= 0
    at = slots[real]
    x = x[real]
    if cache.dtype == torch.float8_e4m3fn:
        x = (x / scale).clamp(-448.0, 448.0)
    bits = torch.uint8 if cache.element_size() == 1 else torch.int16
    cache.view(bits)[at // bs, :, at % bs] = x.to(cache.dtype).view(bits)


def _run_rope(s):
    c = s["case"]
    write = c["op"] == "qk_norm_rope_write"
    if own:
        import paged_kv_cache_75_gb300 as pk

        if not write:
            pk.pa_qk_norm_rope(s["q_out"], s["k_out"], s["q"], s["k"], s["positions"], s["transform"])
            return {"q": s["q_out"], "k": s["k_out"]}
        pk.pa_qk_norm_rope_write(s["q_out"], s["q"], s["k"], s["v"], s["cache"], s["positions"], s["slots"],
                                 s["transform"], s["status"])
    else:
        q, k = _norm_rotate(s["q"], s["qw"], s), _norm_rotate(s["k"], s["kw"], s)
        if not write:
            return {"q": q.to(s["q"].dtype), "k": k.to(s["k"].dtype)}
        s["q_out"].copy_(q.to(s["q"].dtype))
        _put(s["k_cache"], k, s["k_scale"], s["slots"], c["block_size"])
        _put(s["v_cache"], s["v"].float(), s["v_scale"], s["slots"], c["block_size"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gather(cache, table, pos, bs):
    """Rows [B, n, Hkv, D] in 32 bits of the positions pos [B, n] (those in released blocks read block 0)."""
    blk = table.long().gather(1, (pos // bs).clamp(0, table.shape[1] - 1)).clamp(min=0)
    return cache[blk, :, pos % bs].float()


def _run_decode(s):
    c = s["case"]
    if own:
        import paged_kv_cache_75_gb300 as pk

        pk.pa_decode_window(s["out"], s["q"], s["cache"], s["table"], s["lens"], s["max_k"], s["scale"], c["window"],
                            c["sinks"], workspace=s["workspace"], dev_status=s["status"])
        return s["out"]
    lens = s["lens"].long()[:, None]
    lo = (lens - c["window"]).clamp(min=0)
    sink = torch.arange(min(c["sinks"], s["max_k"]), device=DEV)[None].expand(len(lens), -1)
    near = lo + torch.arange(min(c["window"], s["max_k"]), device=DEV)[None]
    pos = torch.cat((sink, near), 1)
    # a first token inside the window counts once
    seen = torch.cat((sink < torch.minimum(lo, lens), near < lens), 1)
    keys = _gather(s["k_cache"], s["table"], pos, c["block_size"])
    vals = _gather(s["v_cache"], s["table"], pos, c["block_size"])
    q = s["q"].float().unflatten(1, (c["kv_heads"], -1))
    w = torch.einsum("bhgd,bnhd->bhgn", q, keys) * (s["scale"] * s["k_scale"])
    w = w.masked_fill(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
    out = torch.einsum("bhgn,bnhd->bhgd", w, vals) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return (out * s["v_scale"]).flatten(1, 2).to(s["q"].dtype)


def _run_prefill(s):
    c = s["case"]
    if own:
        import paged_kv_cache_75_gb300 as pk

        pk.pa_prefill_varlen_window(s["out"], s["q"], s["cache"], s["table"], s["cu_q"], s["cu_k"], s["max_q"],
                                    s["max_k"], s["scale"], c["window"], c["sinks"], dev_status=s["status"])
        return s["out"]
    n, heads = c["seqs"], c["heads"]
    lq, lk = s["cu_q"].diff().long(), s["cu_k"].diff().long()
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), lq, output_size=s["q"].shape[0])
    row = torch.arange(s["q"].shape[0], device=DEV) - s["cu_q"].long()[seq]
    q = torch.zeros(n, s["max_q"], heads, c["head_size"], device=DEV)
    q[seq, row] = s["q"].float()
    pos = torch.arange(s["max_k"], device=DEV)[None].expand(n, -1)
    keys = _gather(s["k_cache"], s["table"], pos, c["block_size"])
    vals = _gather(s["v_cache"], s["table"], pos, c["block_size"])
    q = q.unflatten(2, (c["kv_heads"], -1))
    w = torch.einsum("bqhgd,bnhd->bhgqn", q, keys) * s["scale"]
    at = (lk - lq)[:, None] + torch.arange(s["max_q"], device=DEV)[None]
    seen = (pos[:, None] <= at[..., None]) & ((pos[:, None] > at[..., None] - c["window"]) | (pos[:, None] < c["sinks"]))
    w = w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    out = torch.einsum("bhgqn,bnhd->bqhgd", w, vals)
    out = out / w.sum(-1).permute(0, 3, 1, 2)[..., None].clamp(min=1e-30)
    return out.flatten(2, 3)[seq, row].to(s["q"].dtype)


def run(state):
    op = state["case"]["op"]
    return _run_rope(state) if op.startswith("qk") else _run_decode(state) if op == "decode_window" else _run_prefill(state)


# ----------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------
SIZE = {"f16": 2, "bf16": 2, "e4m3": 1}


def work(case):
    c = case
    d = c["head_size"]
    if c["op"].startswith("qk"):
        write = c["op"] == "qk_norm_rope_write"
        t, h, kvh = c["tokens"], c["heads"], c["kv_heads"]
        moved = t * d * (4 * h + kvh * (2 + (SIZE[c["kv_dtype"]] if write else 2)))
        if write:
            moved += t * d * kvh * (2 + SIZE[c["kv_dtype"]]) + 8 * t
        per = 3 * c["rotary"] + (4 * d if c["norm"] else 0)
        return {"bytes": moved + 8 * t + 8 * (c["rotary"] // 2) + (8 * d if c["norm"] else 0), "flops": t * (h + kvh) * per}
    lk, lq = _lengths(c)
    pairs = rows = pages = 0
    for k, q in zip(lk.tolist(), lq.tolist()):
        at = np.arange(k - q, k)
        at = at[at >= 0]
        lo = np.maximum(at - c["window"] + 1, 0)
        pairs += int((at + 1 - lo).sum() + np.minimum(lo, c["sinks"]).sum())
        if k:
            lo = max(0, k - q - c["window"] + 1)
            rows += k - lo + min(lo, c["sinks"])
            pages += int(_kept(c, k, k - q).sum())
    moved = rows * c["kv_heads"] * d * 2 * SIZE[c["kv_dtype"]] + 4 * int(lq.sum()) * c["heads"] * d + 4 * pages + 8 * len(lk)
    return {"bytes": moved, "flops": 4 * pairs * c["heads"] * d}


# ----------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------
def _exact_rows(x, w, c, pos, freq, factor, eps):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * w.double()
    out = x.clone()
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rotary"] // 2)
        phi = pos.double() * f
        co, si = factor * torch.cos(phi)[:, None], factor * torch.sin(phi)[:, None]
        out[..., a] = x[..., a] * co - x[..., b] * si
        out[..., b] = x[..., a] * si + x[..., b] * co
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"].startswith("qk"):
        freq, factor = _inv_freq(c)
        q = _exact_rows(s["q"], s["qw"], c, s["positions"], freq, factor, s["eps"])
        k = _exact_rows(s["k"], s["kw"], c, s["positions"], freq, factor, s["eps"])
        if c["op"] == "qk_norm_rope":
            return {"q": q, "k": k}
        bs = c["block_size"]
        out = {"q": q}
        for name, x, sc in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
            whole = s[name].double()
            for lo in range(0, c["tokens"], 4096):
                at, y = s["slots"][lo:lo + 4096], x[lo:lo + 4096]
                y, at = y[at >= 0], at[at >= 0]
                if c["kv_dtype"] == "e4m3":
                    y = torch.clamp(y / sc, -448.0, 448.0)
                whole[at // bs, :, at % bs] = y
            out[name] = whole
        return out
    lk, lq = _lengths(c)
    bs, group = c["block_size"], c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    first = 0
    for b in range(c["seqs"]):
        L, n = int(lk[b]), int(lq[b])
        for i0 in range(0, n, 256):
            i1 = min(n, i0 + 256)
            p0, p1 = L - n + i0, L - n + i1  # positions p0 .. p1-1
            lo = max(0, p0 - c["window"] + 1)
            j = np.concatenate([np.arange(min(c["sinks"], lo, max(p1, 0))), np.arange(lo, max(p1, lo))])
            if j.size == 0:
                continue
            j = torch.from_numpy(j.astype(np.int64)).to(DEV)
            blk = s["table"][b][j // bs].long()
            K = s["k_cache"][blk, :, j % bs].double() * s["k_scale"]
            V = s["v_cache"][blk, :, j % bs].double() * s["v_scale"]
            p = torch.arange(p0, p1, device=DEV)[:, None]
            hide = (j[None] > p) | ((p - j[None] >= c["window"]) & (j[None] >= c["sinks"]))
            for h in range(c["heads"]):
                sc = (s["q"][first + i0:first + i1, h].double() @ K[:, h // group].T) * s["scale"]
                sc[hide] = -math.inf
                top = sc.max(-1, keepdim=True).values
                e = torch.exp(sc - torch.nan_to_num(top, neginf=0.0))
                tot = e.sum(-1, keepdim=True)
                out[first + i0:first + i1, h] = (e @ V[:, h // group]) / torch.where(tot == 0, 1.0, tot)
        first += n
    return out
