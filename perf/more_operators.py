"""Measured cases of three operators of beam search over the paged cache.

* ``beam_select``     the best continuations of a request's beams over the vocabulary: log-softmax of each beam's
                      logits, its score added, the K largest of beams and tokens together
* ``beam_reorder``    block tables, lengths and slots of the beams that go on, the partly filled blocks that two
                      of them share copied in every layer's cache
* ``varlen_cascade``  attention over the paged cache of groups of sequences that share a prefix, one query token
                      a sequence or several, the prefix's products computed once for a group

``run`` computes the plain form (elementary torch operations) where ``own`` is false, and makes the library's
calls where it is true.  ``exact`` is the definition in 64 bits, written apart from the plain form.  Sequence
lengths, group sizes and beam counts follow from the case alone; values, tables and parents from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}


# ----------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------
def _select(requests, beams, vocab, dtype, select, **more):
    c = dict(op="beam_select", requests=requests, beams=beams, beams_lo=beams, vocab=vocab, dtype=dtype, select=select,
             allowed=False, ended=False, pad=0, lens_seed=0)
    c.update(more)
    return c


def _reorder(requests, beams, layers, kv_heads, head_size, dtype, **more):
    c = dict(op="beam_reorder", requests=requests, beams=beams, layers=layers, kv_heads=kv_heads, head_size=head_size,
             dtype=dtype, block_size=16, first=False, prompt_lo=16, prompt_hi=64, gen_hi=128, width=0, lens_seed=0)
    c.update(more)
    return c


def _cascade(groups, members, heads, kv_heads, dtype, shared_lo, shared_hi, own_lo, own_hi, q_lo, q_hi, **more):
    c = dict(op="varlen_cascade", groups=groups, members=members, members_lo=members, heads=heads, kv_heads=kv_heads,
             dtype=dtype, shared_lo=shared_lo, shared_hi=shared_hi, own_lo=own_lo, own_hi=own_hi, q_lo=q_lo, q_hi=q_hi,
             block_size=16, lens_seed=0)
    c.update(more)
    return c


def listed():
    return [
        # one request, four beams: the latency of a step's selection
        dict(_select(1, 4, 32000, "bf16", 4), name="select_1x4"),
        # odd vocabulary whose rows start anywhere, beams of unlike count, a grammar's mask over the tokens
        dict(_select(16, 6, 50257, "f16", 12, beams_lo=1, allowed=True, lens_seed=11), name="select_16_mask"),
        # 32-bit logits in a wider buffer, some beams ended
        dict(_select(32, 4, 65024, "f32", 8, ended=True, pad=512), name="select_32x4_f32"),
        # a full serving batch over a large vocabulary
        dict(_select(64, 8, 128256, "bf16", 16), name="select_64x8"),
        # one request's beams, one layer: the latency of the tables' step
        dict(_reorder(1, 4, 1, 8, 128, "bf16", lens_seed=21), name="reorder_1x4"),
        # the first step of 48 requests (one row becomes eight), an E4M3 cache of four layers, long prompts
        dict(_reorder(48, 8, 4, 8, 128, "e4m3", block_size=32, first=True, prompt_lo=64, prompt_hi=4096, width=256,
                      lens_seed=22), name="reorder_first_e4m3"),
        # 64 requests of four beams in the middle of their answers, 16 layers
        dict(_reorder(64, 4, 16, 8, 128, "bf16", lens_seed=23), name="reorder_64x4"),
        # one request of four beams behind a prompt: the latency of a decode step's attention
        dict(_cascade(1, 4, 32, 8, "bf16", 1008, 1008, 1, 64, 1, 1, lens_seed=31), name="cascade_1x4"),
        # beam search of 32 requests, eight beams each, prompts of unlike length
        dict(_cascade(32, 8, 32, 8, "bf16", 256, 8192, 1, 256, 1, 1, lens_seed=32), name="cascade_beams"),
        # 64 answers sampled behind one long document, eight heads to a KV head
        dict(_cascade(1, 64, 64, 8, "f16", 65536, 65536, 16, 1024, 1, 1, block_size=32, lens_seed=33),
             name="cascade_document"),
        # 32 short questions of a few tokens each to one document
        dict(_cascade(1, 32, 32, 8, "bf16", 16384, 16384, 1, 64, 4, 32, lens_seed=34), name="cascade_questions"),
        # prompts behind a few system prompts: ragged chunks of hundreds of tokens
        dict(_cascade(4, 8, 32, 8, "bf16", 1024, 8192, 0, 512, 16, 1024, members_lo=3, lens_seed=35),
             name="cascade_prompts"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["beam_select", "beam_reorder", "varlen_cascade", "varlen_cascade"])
    seed = rng.randrange(1 << 30)
    if op == "beam_select":
        vocab, dtype = _log(rng, 100, 160000), rng.choice(["f16", "bf16", "f32"])
        most = max(1, 60_000_000 // (vocab * (2 if dtype == "f32" else 1)))
        beams = min(_log(rng, 1, 32), most)
        return _select(_log(rng, 1, max(1, min(96, most // beams))), beams, vocab, dtype, rng.randint(1, 64),
                       beams_lo=rng.randint(1, beams), allowed=rng.random() < 0.4, ended=rng.random() < 0.4,
                       pad=rng.choice([0, 0, 1, 8, 200]), lens_seed=seed)
    bs = rng.choice([16, 32, 64])
    kvh = rng.choice([1, 2, 4, 8])
    if op == "beam_reorder":
        return _reorder(_log(rng, 1, 64), rng.randint(1, 8), _log(rng, 1, 6), kvh, rng.choice([64, 128]),
                        rng.choice(["f16", "bf16", "e4m3"]), block_size=bs, first=rng.random() < 0.3,
                        prompt_hi=_log(rng, 16, 96), gen_hi=_log(rng, 1, 96), width=rng.choice([0, 0, 33, 512]),
                        lens_seed=seed)
    groups, members = _log(rng, 1, 12), _log(rng, 1, 24)
    q_hi = rng.choice([1, 1, _log(rng, 1, 24), _log(rng, 2, 256)])
    heads, shared_hi, own_hi = kvh * rng.choice([1, 2, 4, 8]), _log(rng, 16, 8192), _log(rng, 1, 600)
    while q_hi > 1 and groups * members * q_hi * heads * (shared_hi + own_hi) > 3e9:
        q_hi //= 2
    return _cascade(groups, members, heads, kvh, rng.choice(["f16", "bf16"]), 0, shared_hi, 0, own_hi, 1, q_hi,
                    members_lo=rng.randint(1, members), block_size=bs, lens_seed=seed)


def _beam_counts(c):
    g = np.random.default_rng(c["lens_seed"])
    return g.integers(c["beams_lo"], c["beams"] + 1, size=c["requests"])


def _reorder_lengths(c):
    """Prompt and generated tokens of each request (its beams are of one length)."""
    g = np.random.default_rng(c["lens_seed"])
    n = c["requests"]
    prompt = g.integers(min(c["prompt_lo"], c["prompt_hi"]), c["prompt_hi"] + 1, size=n)
    gen = np.zeros(n, np.int64) if c["first"] else g.integers(0, c["gen_hi"] + 1, size=n)
    return prompt, gen


def _cascade_lengths(c):
    """Members and shared tokens of each group; keys past the prefix and queries of each sequence."""
    g = np.random.default_rng(c["lens_seed"])
    bs = c["block_size"]
    size = g.integers(c["members_lo"], c["members"] + 1, size=c["groups"])
    lo, hi = max(c["shared_lo"], 1), max(c["shared_hi"], 1)
    shared = np.exp(g.uniform(math.log(lo), math.log(hi) + 1e-9, size=c["groups"])).astype(np.int64) // bs * bs
    n = int(size.sum())
    lq = g.integers(c["q_lo"], c["q_hi"] + 1, size=n)
    prior = g.integers(c["own_lo"], c["own_hi"] + 1, size=n)
    return size, shared, prior + lq, lq


# ----------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _cum(a):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(a)]).astype(np.int32)).to(DEV)


def _prepare_select(c, seed):
    g = _gen(seed)
    counts = _beam_counts(c)
    rows, v, dt = int(counts.sum()), c["vocab"], DTYPE[c["dtype"]]
    # a broad bulk and a few likely tokens, as a head's outputs have them
    x = torch.randn(rows, v + c["pad"], generator=g, device=DEV).mul_(1.5)
    peaks = torch.randint(0, v, (rows, 12), generator=g, device=DEV)
    x.scatter_(1, peaks, 4.0 + 8.0 * torch.rand(rows, 12, generator=g, device=DEV))
    s = dict(case=c, buffer=x.to(dt), cu_beams=_cum(counts))
    s["logits"] = s["buffer"][:, :v]
    # sums of log-probabilities so far; beams that a request does not have yet stand at -inf
    s["scores"] = -20.0 * torch.rand(rows, generator=g, device=DEV)
    if rows > 8:
        s["scores"][torch.randint(0, rows, (rows // 16 + 1,), generator=g, device=DEV)] = -math.inf
    s["allowed"] = s["ended"] = None
    s["end_token"] = 2 % v
    if c["allowed"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (rows, (v + 31) // 32), generator=g, device=DEV, dtype=torch.int64)
        s["allowed"] = words.to(torch.int32)
        if rows > 4:
            s["allowed"][rows // 2] = 0  # a beam that its grammar leaves nothing
        # what is not allowed may hold anything
        hidden = ~_bits(s["allowed"], v)
        s["logits"][hidden & (torch.rand(rows, v, generator=g, device=DEV) < 0.01)] = math.inf
        s["logits"][hidden & (torch.rand(rows, v, generator=g, device=DEV) < 0.01)] = math.nan
    if c["ended"]:
        s["ended"] = (torch.rand(rows, generator=g, device=DEV) < 0.2).to(torch.uint8)
    k = c["select"]
    s["out"] = (torch.empty(c["requests"], k, dtype=torch.float32, device=DEV),
                torch.empty(c["requests"], k, dtype=torch.int32, device=DEV),
                torch.empty(c["requests"], k, dtype=torch.int32, device=DEV))
    if own:
        import paged_kv_cache_75_gb300 as pk

        n = pk.pa_beam_select_workspace_size(rows, v, k)
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def _prepare_reorder(c, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    prompt, gen = _reorder_lengths(c)
    bs, w = c["block_size"], c["beams"]
    old = 1 if c["first"] else w
    length = prompt + gen
    need = -(-(length + 1) // bs)
    width = max(int(need.max()), c["width"])
    whole = prompt // bs  # shared by a request's beams; what follows is each beam's own
    total = int((whole + old * (-(-length // bs) - whole)).sum())
    n = c["requests"] * w
    blocks = total + n + 3
    ids = rng.permutation(blocks).astype(np.int32)
    table = np.full((c["requests"] * old, width), -1, np.int32)
    at = 0
    for b in range(c["requests"]):
        have = -(-int(length[b]) // bs)
        rows = table[b * old:(b + 1) * old]
        rows[:, :whole[b]] = ids[at:at + whole[b]]
        at += int(whole[b])
        for r in range(old):
            rows[r, whole[b]:have] = ids[at:at + have - whole[b]]
            at += have - int(whole[b])
    spare = ids[at:at + n]
    # the likelier beams go on more than once, others not at all; a request may end with fewer
    pick = (rng.random((c["requests"], w)) ** 2 * old).astype(np.int64)
    parents = (np.arange(c["requests"])[:, None] * old + pick).astype(np.int32)
    if c["requests"] > 2:
        parents[rng.integers(0, c["requests"]), -1] = -1
    s = dict(case=c)
    kd = DTYPE[c["dtype"]]
    shape = (blocks, c["kv_heads"], bs, c["head_size"])
    s["layers"] = []
    for _ in range(c["layers"]):
        s["layers"].append(tuple(torch.randn(shape, generator=g, device=DEV).to(kd) for _ in range(2)))
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    s["table"], s["lens"] = to(table), to(np.repeat(length, old))
    s["parents"], s["spare"] = to(parents.reshape(-1)), to(spare)
    s["table_out"] = torch.empty(n, width, dtype=torch.int32, device=DEV)
    s["lens_out"] = torch.empty(n, dtype=torch.int32, device=DEV)
    s["slots"] = torch.empty(n, dtype=torch.int64, device=DEV)
    s["used"] = torch.empty(n, dtype=torch.int32, device=DEV)
    if own:
        import paged_kv_cache_75_gb300 as pk

        s["caches"] = pk.KVLayers([pk.KVCache(k, v) for k, v in s["layers"]])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def _prepare_cascade(c, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    size, shared, mine, lq = _cascade_lengths(c)
    bs, d, dt = c["block_size"], 128, DTYPE[c["dtype"]]
    group = np.repeat(np.arange(c["groups"]), size)
    lk = shared[group] + mine
    have, pre = -(-lk // bs), shared // bs
    width = int(have.max()) + 1
    total = int(pre.sum() + (have - pre[group]).sum())
    ids = rng.permutation(total + 3).astype(np.int32)
    table = np.full((len(lk), width), -1, np.int32)
    at = 0
    for k in range(c["groups"]):
        rows = np.flatnonzero(group == k)
        table[rows, :pre[k]] = ids[at:at + pre[k]]
        at += int(pre[k])
        for b in rows:
            table[b, pre[k]:have[b]] = ids[at:at + have[b] - pre[k]]
            at += int(have[b] - pre[k])
    shape = (total + 3, c["kv_heads"], bs, d)
    s = dict(case=c, scale=d ** -0.5, max_q=int(lq.max()), max_k=int(lk.max()), max_group=int(size.max()),
             max_shared=int(shared.max()))
    s["k_cache"] = torch.randn(shape, generator=g, device=DEV).to(dt)
    s["v_cache"] = torch.randn(shape, generator=g, device=DEV).to(dt)
    s["q"] = torch.randn(int(lq.sum()), c["heads"], d, generator=g, device=DEV).to(dt)
    s["out"] = torch.empty_like(s["q"])
    s["table"] = torch.from_numpy(table).to(DEV)
    s["cu_q"], s["cu_k"], s["cu_groups"] = _cum(lq), _cum(lk), _cum(size)
    s["shared"] = torch.from_numpy(shared.astype(np.int32)).to(DEV)
    s["host"] = (size, shared, lk, lq)  # lengths that a program's scheduler has beside the device's
    if own:
        import paged_kv_cache_75_gb300 as pk

        s["cache"] = pk.KVCache(s["k_cache"], s["v_cache"])
        n = pk.pa_varlen_cascade_workspace_size(len(lk), int(lq.sum()), c["heads"], c["kv_heads"], d, s["max_q"],
                                                s["max_k"], s["max_shared"], bs)
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    return {"beam_select": _prepare_select, "beam_reorder": _prepare_reorder,
            "varlen_cascade": _prepare_cascade}[case["op"]](case, seed)


# ----------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------
def _bits(words, n):
    on = (words[:, :, None] >> torch.arange(32, dtype=torch.int32, device=words.device)) & 1
    return on.flatten(1)[:, :n].bool()


def _run_select(s):
    c = s["case"]
    scores, rows, tokens = s["out"]
    if own:
        import paged_kv_cache_75_gb300 as pk

        pk.pa_beam_select(scores, rows, tokens, s["logits"], s["scores"], s["cu_beams"], allowed=s["allowed"],
                          ended=s["ended"], end_token=s["end_token"], workspace=s["workspace"], dev_status=s["status"])
        return {"scores": scores, "rows": rows, "tokens": tokens}
    v, k = c["vocab"], c["select"]
    # 64 bits: candidates of two beams may stand closer than 32 bits tell apart
    x = s["logits"].double()
    if s["allowed"] is not None:
        x = x.masked_fill_(~_bits(s["allowed"], v), -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    total = torch.exp(x - top).sum(-1, keepdim=True)
    x = x.sub_(top + torch.log(total)).add_(s["scores"].double()[:, None])
    x = torch.where(torch.isnan(x), -math.inf, x)  # a row that has nothing: -inf less -inf
    if s["ended"] is not None:
        done = s["ended"].bool()
        x = x.masked_fill_(done[:, None], -math.inf)
        x[:, s["end_token"]] = torch.where(done, s["scores"].double(), x[:, s["end_token"]])
    # a request's beams side by side
    cu = s["cu_beams"].long()
    n = cu.diff()
    req = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=x.shape[0])
    at = torch.arange(x.shape[0], device=DEV) - cu[req]
    wide = torch.full((len(n), max(c["beams"], -(-k // v)), v), -math.inf, dtype=torch.float64, device=DEV)
    wide[req, at] = x
    best, idx = torch.sort(wide.flatten(1), dim=1, descending=True, stable=True)
    best, idx = best[:, :k], idx[:, :k]
    real = best > -math.inf
    return {"scores": best.float(), "rows": torch.where(real, cu[:-1, None] + idx // v, -1).int(),
            "tokens": torch.where(real, idx % v, -1).int()}


def _run_reorder(s):
    c = s["case"]
    out = (s["table_out"], s["lens_out"], s["slots"], s["used"])
    if own:
        import paged_kv_cache_75_gb300 as pk

        pk.pa_beam_reorder(s["caches"], s["parents"], s["table"], s["lens"], s["spare"], *out, dev_status=s["status"])
    else:
        bs, parents = c["block_size"], s["parents"].long()
        real, p = parents >= 0, parents.clamp(min=0)
        length = torch.where(real, s["lens"].long()[p], 0)
        last, rest = length // bs, length % bs
        again = torch.tril(parents[:, None] == parents[None], -1).any(1)  # an earlier row has the same parent
        fresh = real & ((rest == 0) | again)
        j = torch.arange(s["table"].shape[1], device=DEV)
        table = torch.where(real[:, None] & (j * bs < length[:, None]), s["table"][p], -1)
        source = s["table"].long()[p, last.clamp(max=len(j) - 1)]
        n = torch.arange(len(p), device=DEV)
        table[n, last] = torch.where(fresh, s["spare"], table[n, last])
        out[0].copy_(table)
        out[1].copy_(torch.where(real, length + 1, 0))
        out[2].copy_(torch.where(real, table[n, last].long() * bs + rest, -1))
        out[3].copy_(fresh)
        # the rows of the blocks that get a copy, token by token
        i, t = torch.nonzero((fresh & (rest > 0))[:, None] & (torch.arange(bs, device=DEV) < rest[:, None]), as_tuple=True)
        for pair in s["layers"]:
            for x in pair:
                x = x.view(torch.uint8) if x.element_size() == 1 else x
                x[s["spare"].long()[i], :, t] = x[source[i], :, t]
    return {"table": out[0], "lens": out[1], "slots": out[2], "used": out[3],
            "caches": [x for pair in s["layers"] for x in pair]}


def _run_cascade(s):
    c = s["case"]
    if own:
        import paged_kv_cache_75_gb300 as pk

        pk.pa_varlen_cascade(s["out"], s["q"], s["cache"], s["table"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"],
                             s["scale"], s["cu_groups"], s["shared"], s["max_group"], s["max_shared"], s["workspace"],
                             dev_status=s["status"])
        return s["out"]
    bs, kvh = c["block_size"], c["kv_heads"]
    first = 0
    _, _, lk, lq = s["host"]
    for b, (n, m) in enumerate(zip(lk.tolist(), lq.tolist())):
        have = -(-n // bs)
        blk = s["table"][b, :have].long()
        keys = s["k_cache"][blk].transpose(1, 2).flatten(0, 1)[:n].float()
        vals = s["v_cache"][blk].transpose(1, 2).flatten(0, 1)[:n].float()
        q = s["q"][first:first + m].float().unflatten(1, (kvh, -1))
        w = torch.einsum("qhgd,nhd->hgqn", q, keys) * s["scale"]
        seen = torch.arange(n, device=DEV)[None] <= n - m + torch.arange(m, device=DEV)[:, None]
        w = w.masked_fill_(~seen, -math.inf)
        w = w.sub_(w.amax(-1, keepdim=True)).exp_()
        o = torch.einsum("hgqn,nhd->qhgd", w, vals) / w.sum(-1).permute(2, 0, 1)[..., None]
        s["out"][first:first + m] = o.flatten(1, 2).to(s["q"].dtype)
        first += m
    return s["out"]


def run(state):
    return {"beam_select": _run_select, "beam_reorder": _run_reorder,
            "varlen_cascade": _run_cascade}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "beam_select":
        rows, v = int(_beam_counts(c).sum()), c["vocab"]
        moved = rows * v * SIZE[c["dtype"]] + (rows * 4 * ((v + 31) // 32) if c["allowed"] else 0)
        return {"bytes": moved + 4 * rows + (rows if c["ended"] else 0) + 12 * c["requests"] * c["select"],
                "flops": 4 * rows * v}
    if c["op"] == "beam_reorder":
        prompt, gen = _reorder_lengths(c)
        bs, w, old = c["block_size"], c["beams"], 1 if c["first"] else c["beams"]
        length = prompt + gen
        width = max(int((-(-(length + 1) // bs)).max()), c["width"])
        # a parent's table row read once, each new row written whole; of a request's beams, those past the
        # likely number of different parents get a copy of the last block's rows
        kept = sum(1.0 - (1.0 - (math.sqrt((i + 1) / old) - math.sqrt(i / old))) ** w for i in range(old))
        rows = float((length % bs).sum()) * max(0.0, w - kept)
        copied = 2 * 2 * rows * c["layers"] * c["kv_heads"] * c["head_size"] * SIZE[c["dtype"]]
        n = c["requests"] * w
        return {"bytes": int(copied + 4 * kept * float((-(-length // bs)).sum()) + 4 * n * width + 24 * n), "flops": 0}
    size, shared, mine, lq = _cascade_lengths(c)
    pre = np.repeat(shared, size)
    pairs = int((pre * lq).sum() + (lq * (mine - lq) + lq * (lq + 1) // 2).sum())
    rows = int(shared.sum() + mine.sum())
    moved = rows * c["kv_heads"] * 128 * 2 * 2 + 2 * 2 * int(lq.sum()) * c["heads"] * 128 + 4 * rows // c["block_size"]
    return {"bytes": moved + 8 * len(lq), "flops": 4 * pairs * c["heads"] * 128}


# ----------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------
def _exact_select(c, s):
    v, k, cu = c["vocab"], c["select"], s["cu_beams"].tolist()
    scores = torch.full((c["requests"], k), -math.inf, dtype=torch.float64, device=DEV)
    rows = torch.full((c["requests"], k), -1, dtype=torch.int32, device=DEV)
    tokens = rows.clone()
    for b in range(c["requests"]):
        found = []
        for r in range(cu[b], cu[b + 1]):
            base = float(s["scores"][r])
            if base == -math.inf:
                continue
            if s["ended"] is not None and int(s["ended"][r]):
                found.append((-base, r, s["end_token"]))
                continue
            tok = torch.arange(v, device=DEV)
            if s["allowed"] is not None:
                tok = tok[(s["allowed"][r][tok // 32].long() >> (tok % 32)) & 1 == 1]
            x = s["logits"][r].double()[tok]
            if x.numel() == 0:
                continue
            lse = torch.logsumexp(x, 0)
            kth = torch.topk(x, min(k, x.numel())).values[-1]
            keep = torch.nonzero(x >= kth)[:, 0]
            found += [(-(base + y), r, t) for y, t in zip((x[keep] - lse).tolist(), tok[keep].tolist())]
        for i, (neg, r, t) in enumerate(sorted(found)[:k]):
            scores[b, i], rows[b, i], tokens[b, i] = -neg, r, t
    return {"scores": scores, "rows": rows, "tokens": tokens}


def _exact_reorder(c, s):
    bs = c["block_size"]
    table, lens, parents = s["table"].cpu().numpy(), s["lens"].cpu().numpy(), s["parents"].cpu().numpy()
    spare = s["spare"].cpu().numpy()
    n, width = len(parents), table.shape[1]
    t2, l2 = np.full((n, width), -1, np.int32), np.zeros(n, np.int32)
    slots, used = np.full(n, -1, np.int64), np.zeros(n, np.int32)
    copies, met = [], set()
    for i, p in enumerate(parents.tolist()):
        if p < 0:
            continue
        full, rest = divmod(int(lens[p]), bs)
        t2[i, :full + (rest > 0)] = table[p, :full + (rest > 0)]
        if rest == 0 or p in met:
            used[i] = 1
            t2[i, full] = spare[i]
            if rest:
                copies.append((int(table[p, full]), int(spare[i]), rest))
        met.add(p)
        l2[i] = lens[p] + 1
        slots[i] = int(t2[i, full]) * bs + rest
    caches = []
    for pair in s["layers"]:
        for x in pair:
            y = x.double()
            for a, b, rest in copies:
                y[b, :, :rest] = y[a, :, :rest].clone()
            caches.append(y)
    to = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return {"table": to(t2), "lens": to(l2), "slots": to(slots), "used": to(used), "caches": caches}


def _exact_cascade(c, s):
    bs, per = c["block_size"], c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cu_q) - 1):
        q0, m, n = cu_q[b], cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        pos = torch.arange(n, device=DEV)
        blk = s["table"][b].long()[pos // bs]
        hide = pos[None] > (n - m) + torch.arange(m, device=DEV)[:, None]
        for h in range(c["kv_heads"]):
            K, V = s["k_cache"][blk, h, pos % bs].double(), s["v_cache"][blk, h, pos % bs].double()
            q = s["q"][q0:q0 + m, h * per:(h + 1) * per].double().transpose(0, 1)
            sc = (q @ K.T) * s["scale"]
            sc[:, hide] = -math.inf
            out[q0:q0 + m, h * per:(h + 1) * per] = (torch.softmax(sc, -1) @ V).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"beam_select": _exact_select, "beam_reorder": _exact_reorder, "varlen_cascade": _exact_cascade}[case["op"]](case, s)
